// Microscaled (MX) operators: formats shared by their kernels, and the host-side launchers
// (internal; the public ABI is include/awq.h).
//
// A block is 32 consecutive input channels.  Its scale is 2^(E - 127), E one byte, and its elements
// are p / 2^(E - 127) in e4m3 (8 bits) or e2m1 (4 bits), rounded to nearest even and saturated:
//   E = max(biased exponent of max|p| - e_max, 0),  e_max = 8 (e4m3) or 2 (e2m1),
// so that the largest element lands in the format's top binade.  E = 255 marks a block that holds
// an infinity or a NaN (its elements are stored as zeros; every value it stands for is NaN).
#pragma once
#include "awq_device.h"

namespace awq {

constexpr int kMxBlock = 32;     // channels per scale
constexpr int kMxTile = 64;      // output columns per tile of packed weights
constexpr int kMxChunk = 128;    // channels per scaled matrix-core product: packed weights are padded to it

inline int64_t mx_kb(int64_t K) { return (K + kMxChunk - 1) / kMxChunk * (kMxChunk / kMxBlock); }   // blocks, padded
inline int64_t mx_nt(int64_t N) { return (N + kMxTile - 1) / kMxTile; }
inline size_t mx_codes_bytes(int64_t K, int64_t N) { return (size_t)mx_nt(N) * mx_kb(K) * kMxTile * 16; }
inline size_t mx_scales_bytes(int64_t K, int64_t N) { return (size_t)mx_nt(N) * mx_kb(K) * kMxTile; }

// ---- formats on the device
// Scale byte of a block whose largest |p| has the float32 bits `top` (NaN > infinity > finite as
// unsigned integers, so an integer maximum of |p| finds them).
template <int BITS>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t top) {
    const int e = (int)(top >> 23);
    return e == 255 ? 255u : (uint32_t)max(e - (BITS == 8 ? 8 : 2), 0);
}
// The conversions' scale operand: 2^(E - 127) with E in the exponent field (they read that field
// alone: 0 is 2^-127, 255 turns every element into NaN).
__device__ __forceinline__ float mx_scale(uint32_t E) { return __uint_as_float(E << 23); }
// Eight numbers of a block -> packed codes.  e4m3: two words, saturated first (the conversion itself
// turns what rounds beyond 448 into NaN).  e2m1: one word (the conversion saturates).
__device__ __forceinline__ uint2 mx_e4m3x8(const float (&p)[8], uint32_t E) {
    typedef short s16x2 __attribute__((ext_vector_type(2)));
    const float scale = mx_scale(E), lim = E == 0 ? 0x1.cp-119f : 448.f * scale;
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float q[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) q[i] = __builtin_amdgcn_fmed3f(p[4 * h + i], -lim, lim);
        s16x2 r = {0, 0};
        r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, q[0], q[1], scale, false);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, q[2], q[3], scale, true);
        w[h] = __builtin_bit_cast(uint32_t, r);
    }
    return uint2{w[0], w[1]};
}
__device__ __forceinline__ uint32_t mx_e2m1x8(const float (&p)[8], uint32_t E) {
    const float scale = mx_scale(E);
    uint32_t r = 0;
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, p[0], p[1], scale, 0);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, p[2], p[3], scale, 1);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, p[4], p[5], scale, 2);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, p[6], p[7], scale, 3);
    return r;
}
// Division by the input scales, s in [2^-120, 2^120]: x / s rounded to float32.
//
// Activations: (float)(x r) with r = 1 / s to 53 bits (the float32 approximation's error e, below 2^-22, taken out to the
// third order: r (1 + e + e^2)).  r and the product are each off by at most 2^-53 of their size, but a quotient of two
// 24-bit numbers lies either on a border between two float32 numbers, which only subnormal ones can, or at least 2^-49
// of its size away from it: the difference is a whole number over the 24-bit divisor times a 25-bit border.  So the result is the
// rounded quotient, infinite where it overflows, subnormal below 2^-126 (there an exact tie may go to either
// side), with the sign of a zero.
__device__ __forceinline__ double mx_recip64(float s) {
    const double d = s, r = __builtin_amdgcn_rcpf(s), e = fma(-d, r, 1.);
    return fma(r, fma(e, e, e), r);
}
__device__ __forceinline__ float mx_div(float x, double r) { return (float)((double)x * r); }
// Elements of weights (.5 <= |x| <= 6, or 0): float32 alone, which is faster where a divisor serves few elements.  r is 1 / s
// rounded (checked on gfx950 for every mantissa), q = x r at most 1.5 of its steps away from the quotient, and
// its remainder exact: R / S steps, S the 24-bit divisor and R a whole number.  The correction R / S (1 + e), |e| <= 2^-24,
// misses R / S by less than its distance from every border, at least 1 / (2 S), so the result is the rounded
// quotient.  (For other x a remainder below 2^-149 would be lost, and a quotient that overflows would become NaN.)
__device__ __forceinline__ float mx_recip(float s) {
    const float r = __builtin_amdgcn_rcpf(s);
    return fmaf(fmaf(-s, r, 1.f), r, r);
}
__device__ __forceinline__ float mx_div_element(float x, float s, float r) {
    const float q = x * r;
    return fmaf(-fmaf(q, s, -x), r, q);          // signs such that -0 stays -0
}
// The largest |p| (as integer bits) of a block held by four consecutive lanes, eight elements each;
// all four lanes must be active.
__device__ __forceinline__ uint32_t mx_block_top(const float (&p)[8]) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(p[i]) & 0x7fffffffu);
    top = max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0xB1, 0xf, 0xf, true));   // lanes 1 0 3 2
    return max(top, (uint32_t)__builtin_amdgcn_mov_dpp((int)top, 0x4E, 0xf, 0xf, true));  // lanes 2 3 0 1
}
// Quantizes the eight elements of octet `oct` of a row (block oct / 4) and stores codes and scale.
template <int BITS>
__device__ __forceinline__ void mx_store8(const float (&p)[8], uint8_t* codes_row, uint8_t* scales_row, int64_t oct) {
    const uint32_t E = mx_scale_byte<BITS>(mx_block_top(p));
    if constexpr (BITS == 8) {
        const uint2 w = mx_e4m3x8(p, E);
        *(uint2*)(codes_row + oct * 8) = E == 255 ? uint2{0u, 0u} : w;
    } else {
        const uint32_t w = mx_e2m1x8(p, E);
        *(uint32_t*)(codes_row + oct * 4) = E == 255 ? 0u : w;
    }
    if ((oct & 3) == 0) scales_row[oct >> 2] = (uint8_t)E;
}
// 16 bytes of bf16 -> eight floats
__device__ __forceinline__ void bf16x8_to_f32(const u32x4& v, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(v[i]);
        x[2 * i + 1] = bf16_hi(v[i]);
    }
}

// ---- host side
// Records a HIP error for awq_last_hip_error and returns the call's status (awq_api.hip).
int record_hip(hipError_t e);

hipError_t launch_mx_pack(const uint16_t* W, int64_t K, int64_t N, const float* s, uint8_t* codes, uint8_t* scales,
                          hipStream_t st);
hipError_t launch_mx_unpack(const uint8_t* codes, const uint8_t* scales, int64_t K, int64_t N, const float* s,
                            uint16_t* W, hipStream_t st);
hipError_t launch_mx_quantize(const uint16_t* X, const uint16_t* gate, int64_t M, int64_t K, const float* s, int bits,
                              uint8_t* codes, uint8_t* scales, hipStream_t st);
hipError_t launch_rms_norm(const uint16_t* X, const uint16_t* residual, const uint16_t* weight, int64_t M, int64_t K,
                           float eps, uint16_t* residual_out, uint16_t* Y, const float* s, int bits, uint8_t* codes,
                           uint8_t* scales, hipStream_t st);

struct MxGemmPlan {
    int wm;                         // 0: the register kernel; else LDS tiles of 64 wm rows
    int nz;                         // slices of K
    int cstride;                    // arrival counter i at word i * cstride of the counter region
    int64_t col_tiles, row_tiles;   // workgroup tiles
    size_t ws_bytes;
};
MxGemmPlan plan_mx_gemm(int64_t M, int64_t K, int64_t N, int bits);
hipError_t launch_mx_gemm(const uint8_t* xcodes, const uint8_t* xscales, int bits, int64_t M, const uint8_t* codes,
                          const uint8_t* scales, int64_t K, int64_t N, uint16_t* Y, void* ws, const MxGemmPlan& p,
                          hipStream_t st);

}  // namespace awq
