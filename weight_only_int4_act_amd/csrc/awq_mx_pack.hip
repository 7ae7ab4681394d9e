// MX weights: bf16 [K, N] to 4-bit blocks in the product's tile order, and back.
#include <algorithm>

#include "awq_mx.h"

namespace awq {
namespace {

// A thread owns four adjacent columns of one block (32 rows), so that a wavefront reads 512
// contiguous bytes of each row; a workgroup's four wavefronts take the four blocks of one 128-row
// chunk.  Bound by HBM: 2 bytes read and 0.53 written per weight; 8192 x 28672 with scales takes
// 119 us (5.0 TB/s; a copy of 2 GiB reaches 4.9; right behind an unpack, whose output is still being written
// back, 147), 4096 x 4096 11.7 us.  The rows stay packed in
// registers (64 of them, all loads in flight at once): without scales the maximum is taken on packed
// bf16 bits and pairs go straight into the conversion; with scales the products are formed twice,
// for the maximum and for the conversion, which is cheaper than holding them.  Both directions with
// scales, one after the other, took 466 us when each row was converted by itself, 241 us now.
//
// Tile t holds columns 64t .. 64t+63: codes[(t * kb_all + kb) * 64 + c] is the 16-byte block of column
// 64t + c, and scale byte 4i + j of (t, kb) belongs to column 64t + 16j + i, so that one 4-byte load
// gives a lane of the matrix-core product the scales of its four 16-column fragments.  A lane has
// columns 4a .. 4a+3 (a = lane % 16): their bytes go to 16 (a % 4) + 4b + a / 4, b = 0 .. 3.  Between
// the four lanes with equal a % 4 that is a 4 x 4 transposition of bytes, after which lane a holds
// the word at 16 (a % 4) + 4 (a / 4).  It is its own inverse.
__device__ __forceinline__ uint32_t transpose_scales(uint32_t e, int lane) {
    // exchange odd and even bytes between lanes 4 apart, then halves between lanes 8 apart
    const uint32_t o = (uint32_t)__shfl_xor((int)e, 4, kWave);
    e = lane & 4 ? (e & 0xff00ff00u) | ((o >> 8) & 0x00ff00ffu) : (e & 0x00ff00ffu) | ((o << 8) & 0xff00ff00u);
    const uint32_t p = (uint32_t)__shfl_xor((int)e, 8, kWave);
    return lane & 8 ? (e & 0xffff0000u) | (p >> 16) : (e & 0x0000ffffu) | (p << 16);
}
__device__ __forceinline__ uint32_t scale_word(int lane) { return 16 * (lane & 3) + 4 * ((lane >> 2) & 3); }

struct __attribute__((packed, aligned(2))) Quad {   // four columns at a bf16's alignment
    uint2 v;
};
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// halves of two words: (a.lo, b.lo) or (a.hi, b.hi)
__device__ __forceinline__ uint32_t pair_lo(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x05040100); }
__device__ __forceinline__ uint32_t pair_hi(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302); }

// The conversions with a byte index h that the unrolled loops make constant.
#define MX_BYTE(call)            \
    switch (h) {                 \
        case 0: return call(0);  \
        case 1: return call(1);  \
        case 2: return call(2);  \
        default: return call(3); \
    }
__device__ __forceinline__ uint32_t to_fp4(uint32_t old, float a, float b, float scale, int h) {
#define MX_CALL(i) __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, a, b, scale, i)
    MX_BYTE(MX_CALL)
#undef MX_CALL
}
__device__ __forceinline__ uint32_t to_fp4(uint32_t old, bf16x2 p, float scale, int h) {
#define MX_CALL(i) __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, p, scale, i)
    MX_BYTE(MX_CALL)
#undef MX_CALL
}
__device__ __forceinline__ bf16x2 fp4_to_bf16(uint32_t w, float scale, int h) {
#define MX_CALL(i) __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, i)
    MX_BYTE(MX_CALL)
#undef MX_CALL
}
typedef float f32x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ f32x2 fp4_to_f32(uint32_t w, float scale, int h) {
#define MX_CALL(i) __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, i)
    MX_BYTE(MX_CALL)
#undef MX_CALL
}
#undef MX_BYTE

template <bool SCALED>
__global__ __launch_bounds__(256) void k_mx_pack(const uint16_t* __restrict__ W, int64_t K, int64_t N,
                                                 const float* __restrict__ s, uint8_t* __restrict__ codes,
                                                 uint8_t* __restrict__ scales, int64_t kb_all) {
    const int lane = threadIdx.x & 63;
    const int64_t kb = (int64_t)blockIdx.y * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n0 = ((int64_t)blockIdx.x * 64 + lane) * 4, k0 = kb * kMxBlock;
    const bool in_k = k0 < K;                    // K % 32 == 0: a block is inside or outside as a whole
    // The last columns of a row are read as the last four and shifted (what lies outside is zero).
    const int64_t n1 = max((int64_t)0, min(n0, N - 4));
    const uint32_t past = (uint32_t)min(n0 - n1, (int64_t)4);
    uint2 w[32];
    if (in_k && N >= 4) {
#pragma unroll
        for (int r = 0; r < 32; ++r) w[r] = ((const Quad*)(W + (k0 + r) * N + n1))->v;
        if (__any(past != 0)) {
#pragma unroll
            for (int r = 0; r < 32; ++r) {
                const uint64_t q = past > 3 ? 0 : ((uint64_t)w[r].x | ((uint64_t)w[r].y << 32)) >> (16 * past);
                w[r] = uint2{(uint32_t)q, (uint32_t)(q >> 32)};
            }
        }
    } else {
#pragma unroll
        for (int r = 0; r < 32; ++r) {
            uint32_t v[3] = {0, 0, 0};           // fewer than four columns
            if (in_k)
                for (int c = 0; c < 3; ++c)
                    if (n0 + c < N) v[c] = W[(k0 + r) * N + n0 + c];
            w[r] = uint2{v[0] | (v[1] << 16), v[2]};
        }
    }
    uint32_t top[4] = {0, 0, 0, 0};              // largest |p| of each column, as float32 bits
    if constexpr (SCALED) {
#pragma unroll
        for (int r = 0; r < 32; ++r) {
            const float sk = in_k ? s[k0 + r] : 1.f;
            const float p[4] = {bf16_lo(w[r].x) * sk, bf16_hi(w[r].x) * sk, bf16_lo(w[r].y) * sk, bf16_hi(w[r].y) * sk};
#pragma unroll
            for (int c = 0; c < 4; ++c) top[c] = max(top[c], __float_as_uint(p[c]) & 0x7fffffffu);
        }
    } else {
        u16x2 a = {0, 0}, b = {0, 0};
#pragma unroll
        for (int r = 0; r < 32; ++r) {
            a = __builtin_elementwise_max(a, __builtin_bit_cast(u16x2, w[r].x & 0x7fff7fffu));
            b = __builtin_elementwise_max(b, __builtin_bit_cast(u16x2, w[r].y & 0x7fff7fffu));
        }
        top[0] = (uint32_t)a[0] << 16, top[1] = (uint32_t)a[1] << 16;
        top[2] = (uint32_t)b[0] << 16, top[3] = (uint32_t)b[1] << 16;
    }
    uint32_t E[4], word = 0;
    float scale[4];
    u32x4 out[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        E[c] = mx_scale_byte<4>(top[c]);
        word |= E[c] << (8 * c);
        scale[c] = mx_scale(E[c]);
        out[c] = u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int h = 0; h < 4; ++h) {            // byte h of word q: rows 8q + 2h and the next
            const int r = 8 * q + 2 * h;
            if constexpr (SCALED) {
                const float s0 = in_k ? s[k0 + r] : 1.f, s1 = in_k ? s[k0 + r + 1] : 1.f;
                const float a[4] = {bf16_lo(w[r].x) * s0, bf16_hi(w[r].x) * s0, bf16_lo(w[r].y) * s0, bf16_hi(w[r].y) * s0};
                const float b[4] = {bf16_lo(w[r + 1].x) * s1, bf16_hi(w[r + 1].x) * s1, bf16_lo(w[r + 1].y) * s1,
                                    bf16_hi(w[r + 1].y) * s1};
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    out[c][q] = to_fp4(out[c][q], a[c], b[c], scale[c], h);
            } else {
                const uint32_t p[4] = {pair_lo(w[r].x, w[r + 1].x), pair_hi(w[r].x, w[r + 1].x),
                                       pair_lo(w[r].y, w[r + 1].y), pair_hi(w[r].y, w[r + 1].y)};
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    out[c][q] = to_fp4(out[c][q], __builtin_bit_cast(bf16x2, p[c]), scale[c], h);
            }
        }
    word = transpose_scales(word, lane);
    if (n0 >= (N + kMxTile - 1) / kMxTile * kMxTile) return;     // past the last tile: 16 lanes at a time
    const int64_t base = (n0 / kMxTile * kb_all + kb) * kMxTile;
#pragma unroll
    for (int c = 0; c < 4; ++c)
        *(u32x4*)(codes + (base + (n0 % kMxTile) + c) * 16) = E[c] == 255 ? u32x4{0, 0, 0, 0} : out[c];
    *(uint32_t*)(scales + base + scale_word(lane)) = word;
}

// The reverse: a thread reads four adjacent 16-byte blocks and writes four columns of 32 rows.  Bound by
// HBM, too: 8192 x 28672 with scales 124 us (4.8 TB/s), without 118; 4096 x 4096 12.3 and 9.6 us.
template <bool SCALED>
__global__ __launch_bounds__(256) void k_mx_unpack(const uint8_t* __restrict__ codes,
                                                   const uint8_t* __restrict__ scales, int64_t K, int64_t N,
                                                   const float* __restrict__ s, uint16_t* __restrict__ W,
                                                   int64_t kb_all) {
    const int lane = threadIdx.x & 63;
    const int64_t kb = (int64_t)blockIdx.y * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t n0 = ((int64_t)blockIdx.x * 64 + lane) * 4, k0 = kb * kMxBlock;
    if (k0 >= K) return;
    const bool in_n = n0 < (N + kMxTile - 1) / kMxTile * kMxTile;
    const int64_t base = ((in_n ? n0 : 0) / kMxTile * kb_all + kb) * kMxTile;
    u32x4 w[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) w[c] = *(const u32x4*)(codes + (base + (n0 % kMxTile) + c) * 16);
    const uint32_t word = transpose_scales(*(const uint32_t*)(scales + base + scale_word(lane)), lane);
    if (n0 >= N) return;
    float scale[4], power[4];                    // with scales the block's power of two comes after the division
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const uint32_t E = (word >> (8 * c)) & 255u;
        scale[c] = SCALED && E < 255 ? 1.f : mx_scale(E);
        power[c] = E == 0 ? 0x1p-127f : mx_scale(min(E, 254u));
    }
    auto store = [&](int r, uint2 v) {
        uint16_t* row = W + (k0 + r) * N + n0;
        if (n0 + 3 < N) {
            ((Quad*)row)->v = v;
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (n0 + c < N) row[c] = (uint16_t)((c < 2 ? v.x : v.y) >> (16 * (c & 1)));
        }
    };
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const int r = 8 * q + 2 * h;
            if constexpr (SCALED) {
                // .5 <= |element| <= 6: no quotient by s leaves float32, so that only the last product may
                const float s0 = s[k0 + r], s1 = s[k0 + r + 1], r0 = mx_recip(s0), r1 = mx_recip(s1);
                float a[4], b[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const f32x2 v = fp4_to_f32(w[c][q], scale[c], h);
                    a[c] = mx_div_element(v[0], s0, r0) * power[c];
                    b[c] = mx_div_element(v[1], s1, r1) * power[c];
                }
                store(r, uint2{pack_bf16x2(a[0], a[1]), pack_bf16x2(a[2], a[3])});
                store(r + 1, uint2{pack_bf16x2(b[0], b[1]), pack_bf16x2(b[2], b[3])});
            } else {
                uint32_t p[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) p[c] = __builtin_bit_cast(uint32_t, fp4_to_bf16(w[c][q], scale[c], h));
                store(r, uint2{pair_lo(p[0], p[1]), pair_lo(p[2], p[3])});
                store(r + 1, uint2{pair_hi(p[0], p[1]), pair_hi(p[2], p[3])});
            }
        }
}

}  // namespace

hipError_t launch_mx_pack(const uint16_t* W, int64_t K, int64_t N, const float* s, uint8_t* codes, uint8_t* scales,
                          hipStream_t st) {
    const int64_t kb = mx_kb(K);
    const dim3 grid((unsigned)((mx_nt(N) * kMxTile + 255) / 256), (unsigned)(kb / 4));
    if (s) k_mx_pack<true><<<grid, 256, 0, st>>>(W, K, N, s, codes, scales, kb);
    else k_mx_pack<false><<<grid, 256, 0, st>>>(W, K, N, s, codes, scales, kb);
    return hipGetLastError();
}

hipError_t launch_mx_unpack(const uint8_t* codes, const uint8_t* scales, int64_t K, int64_t N, const float* s,
                            uint16_t* W, hipStream_t st) {
    const int64_t kb = mx_kb(K);
    const dim3 grid((unsigned)((N + 255) / 256), (unsigned)(kb / 4));
    if (s) k_mx_unpack<true><<<grid, 256, 0, st>>>(codes, scales, K, N, s, W, kb);
    else k_mx_unpack<false><<<grid, 256, 0, st>>>(codes, scales, K, N, s, W, kb);
    return hipGetLastError();
}

}  // namespace awq
