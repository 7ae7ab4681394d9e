// Buffer resources: bounds-checked loads and stores, exchange between workgroups, direct transfers to LDS.
#pragma once
#include "awq_device.h"

namespace awq {

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)(uint32_t)bytes, 0x00020000);
}
constexpr uint32_t kOutside = 0x80000000u;   // an offset past every resource (all are below 2 GiB)
constexpr int kCpolStream = 2;               // non-temporal: data read once
constexpr int kCpolAgent = 16;               // device-coherent level (the sc1 bit)
__device__ __forceinline__ void store4_agent(__amdgpu_buffer_rsrc_t r, uint32_t off, floatx4 v) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), r, off, 0, kCpolAgent);
}
__device__ __forceinline__ floatx4 load4_agent(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(floatx4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, kCpolAgent));
}

__device__ __forceinline__ i32x4 byte_rsrc(const void* base, uint32_t bytes) {
    const uint64_t a = (uint64_t)(uintptr_t)base;
    return i32x4{(int)__builtin_amdgcn_readfirstlane((uint32_t)a),
                 (int)(__builtin_amdgcn_readfirstlane((uint32_t)(a >> 32)) & 0xffff),
                 (int)__builtin_amdgcn_readfirstlane(bytes), 0x00020000};
}
// 16 bytes per lane from byte voff + soff of the resource to LDS address lds + off + 16 * lane (off a constant); a lane
// whose voff is at or past the resource's end brings zeros.  M0 holds the LDS address: every transfer writes it
// itself, with a wait state before its use, and leaves nothing there for another statement.
__device__ __forceinline__ void dma16(i32x4 rsrc, uint32_t voff, uint32_t soff, uint32_t lds, int off) {
#ifdef __HIP_DEVICE_COMPILE__                   // the host pass does not know the registers
    asm volatile(
        "s_add_u32 m0, %3, %4\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %0, %1, %2 offen lds"
        :
        : "v"(voff), "s"(rsrc), "s"(__builtin_amdgcn_readfirstlane(soff)), "s"(__builtin_amdgcn_readfirstlane(lds)), "i"(off)
        : "memory", "scc");
#endif
}

}  // namespace awq
