// 8-bit operators with float32 scales for groups of 128: formats shared by their kernels, and the host-side
// launchers (internal; the public ABI is include/awq.h).
//
// A group is 128 consecutive channels of one row of activations, or 128 channels x 128 columns of weights:
// s = max(max|p|, 448 * 2^-120) / 448, elements p / s in e4m3.  s = NaN marks a group that holds an infinity or a NaN
// (its elements are zero).
#pragma once
#include "awq_device.h"

namespace awq {

constexpr int kFp8Group = 128;   // channels (and columns of weights) per scale
constexpr int kFp8Tile = 64;     // output columns per tile of packed weights: 8 KB for each group of channels

inline int64_t fp8_kc(int64_t K) { return (K + kFp8Group - 1) / kFp8Group; }
inline int64_t fp8_nt(int64_t N) { return (N + kFp8Tile - 1) / kFp8Tile; }
inline int64_t fp8_nb(int64_t N) { return (N + kFp8Group - 1) / kFp8Group; }
inline size_t fp8_codes_bytes(int64_t K, int64_t N) { return (size_t)fp8_nt(N) * fp8_kc(K) * kFp8Tile * kFp8Group; }
inline size_t fp8_scales_count(int64_t K, int64_t N) { return (size_t)fp8_nb(N) * fp8_kc(K); }

// ---- formats on the device
struct Fp8Scale {
    float s, d, r;               // the scale (NaN marks the group), what elements are divided by, and 1 / d
    bool bad;
};
// Scale of a group whose largest |p| has the float32 bits `top` (NaN > infinity > finite as unsigned integers).  The
// floor keeps 1 / s finite: 2^120 at most.
__device__ __forceinline__ Fp8Scale fp8_scale(uint32_t top) {
    Fp8Scale f;
    f.bad = top >= 0x7f800000u;
    f.d = fmaxf(__uint_as_float(f.bad ? 0u : top), 0x1.cp-112f) / 448.f;
    f.r = 1.f / f.d;
    f.s = f.bad ? __uint_as_float(0x7fc00000u) : f.d;
    return f;
}
// Eight elements: e4m3 of the float32 quotient p / s.  With S / 2^23 = t the scale's 24-bit mantissa, r is off by 2^-25 t of
// itself at most, so q = p r, of mantissa m, is less than m t / 4 + 1/2 of its steps away from the quotient: R / S steps, R a whole
// number.  Only quotients next to a border of two codes matter, where m <= 31/16: |R / S| < 1.47, so that q - R / S rounds right
// unless it lies by the border half a step from q.  There R is below 2^24, its remainder in float32 exact, and the correction
// misses R / S by 2^-26 t, less than its distance from the border, which is 0 or at least 1 / (2 S) = 2^-24 / t.  A remainder below
// 2^-149 would be lost: small groups are taken 2^64 times as large (beside them, numbers below 2^-10 scales, whose elements
// are zero either way).  No quotient rounds above 448.  p r alone gave other codes where p / s lies midway between two of them, as
// quotients of bf16 numbers often do (4096 x 8192: 19.8 us, that way 19.4; packing 4096 x 4096: 11.5 and 11.7).
__device__ __forceinline__ uint2 fp8_codes8(const float (&p)[8], const Fp8Scale& f) {
    float x[8], d = f.d, r = f.r;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = p[i];
    if (d < 0x1p-40f) {
        d *= 0x1p64f, r *= 0x1p-64f;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= 0x1p64f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float q = x[i] * r;
        x[i] = fmaf(-fmaf(q, d, -x[i]), r, q);   // signs such that -0 stays -0
    }
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        int v = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * h], x[4 * h + 1], 0, false);
        v = __builtin_amdgcn_cvt_pk_fp8_f32(x[4 * h + 2], x[4 * h + 3], v, true);
        w[h] = f.bad ? 0u : (uint32_t)v;
    }
    return uint2{w[0], w[1]};
}
__device__ __forceinline__ uint32_t fp8_top8(const float (&p)[8]) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(p[i]) & 0x7fffffffu);
    return top;
}
// The maximum over 16 consecutive lanes, in each of them (all must be active).
__device__ __forceinline__ uint32_t max16(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xf, 0xf, true));     // lanes 1 0 3 2
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xf, 0xf, true));     // lanes 2 3 0 1
    v = max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x141, 0xf, 0xf, true));    // mirrored within 8
    return max(v, (uint32_t)__builtin_amdgcn_mov_dpp((int)v, 0x140, 0xf, 0xf, true)); // mirrored within 16
}

// ---- host side
int record_hip(hipError_t e);    // records a HIP error for awq_last_hip_error, returns the call's status (awq_api.hip)

hipError_t launch_fp8_pack(const uint16_t* W, int64_t K, int64_t N, uint8_t* codes, float* scales, hipStream_t st);
hipError_t launch_fp8_quantize(const uint16_t* X, const uint16_t* gate, int64_t M, int64_t K, uint8_t* codes,
                               float* scales, hipStream_t st);

struct Fp8GemmPlan {
    int wm;                         // 0: the register kernel; else LDS tiles of 64 wm rows
    int nz;                         // slices of K
    int cstride;                    // arrival counter i at word i * cstride of the counter region
    int64_t col_tiles, row_tiles;   // workgroup tiles
    size_t ws_bytes;
};
Fp8GemmPlan plan_fp8_gemm(int64_t M, int64_t K, int64_t N);
hipError_t launch_fp8_gemm(const uint8_t* xcodes, const float* xscales, int64_t M, const uint8_t* codes,
                           const float* scales, int64_t K, int64_t N, uint16_t* Y, void* ws, const Fp8GemmPlan& p,
                           hipStream_t st);

}  // namespace awq
