// Activations and weights into e4m3 groups of 128 with float32 scales.
#include "awq_fp8.h"

namespace awq {
namespace {

__device__ __forceinline__ void widen8(const u32x4& v, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(v[i]);
        x[2 * i + 1] = bf16_hi(v[i]);
    }
}

// ---------------------------------------------------------------- quantizer of activations
// p = x, or x g / (1 + e^-g).  Bound by HBM: 2 (4 with a gate) bytes read and 1.03 written per element; 4096 x 8192 in 20 us
// (5.0 TB/s), 16 x 28672 with a gate in 2.4 (a launch and one trip to memory).  Sixteen consecutive lanes hold a group, eight
// channels each, so that its maximum is four lane exchanges and no LDS; a wavefront takes 512 channels of R rows, R > 1
// only where the grid's second dimension would not hold the rows.
template <bool GATE>
__global__ __launch_bounds__(256) void k_fp8_quantize(const uint16_t* __restrict__ X, const uint16_t* __restrict__ gate,
                                                      int64_t M, int64_t K, uint8_t* __restrict__ codes,
                                                      float* __restrict__ scales, int R) {
    const int64_t oct = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63), octs = K / 8, kc = (K + 127) / 128;
    const bool in = oct < octs;                  // a lane past K takes part in its group with zeros
    const int64_t m0 = ((int64_t)blockIdx.y * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * R;
    const int64_t m1 = min(m0 + R, M);
    for (int64_t m = m0; m < m1; ++m) {
        u32x4 xv = {0, 0, 0, 0}, gv = {0, 0, 0, 0};
        if (in) {
            xv = *(const u32x4*)(X + m * K + oct * 8);
            if constexpr (GATE) gv = *(const u32x4*)(gate + m * K + oct * 8);
        }
        float x[8];
        widen8(xv, x);
        if constexpr (GATE) {
            float g[8];
            widen8(gv, g);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // e^-g as a power of two; where it overflows the factor is zero
                const float e = __builtin_amdgcn_exp2f(g[i] * -1.44269504f);
                x[i] *= g[i] * __builtin_amdgcn_rcpf(1.f + e);
            }
        }
        const Fp8Scale f = fp8_scale(max16(fp8_top8(x)));
        const uint2 w = fp8_codes8(x, f);
        if (!in) continue;
        *(uint2*)(codes + m * K + oct * 8) = w;
        if ((oct & 15) == 0) scales[m * kc + (oct >> 4)] = f.s;
    }
}

// ---------------------------------------------------------------- weights
// One workgroup per group of 128 x 128: the numbers stay in registers (thread t: columns 8 (t % 16) .. + 7 of rows
// 8 (t / 16) .. + 7), the codes go through LDS into the packed order, 8 KB for each of the two column tiles.
// Bound by HBM: 2 bytes read and 1 written per weight; 8192 x 28672 in 137 us (5.2 TB/s).  4096 x 4096 takes 14.8 (3.4 TB/s): 1024
// workgroups are one round of four per CU, whose loads, barriers and stores do not overlap each other's.  Weights of other columns
// than a multiple of 8, or not on 16 bytes, are read two bytes at a time: 8192 x 28671 277 us, 4096 x 4096 at an odd address 23.
template <bool VEC>
__global__ __launch_bounds__(256) void k_fp8_pack(const uint16_t* __restrict__ W, int64_t K, int64_t N, int64_t kc,
                                                  uint8_t* __restrict__ codes, float* __restrict__ scales) {
    __shared__ u32x4 out[1024];                  // [2 column tiles][8][64] pieces of 16 bytes
    __shared__ uint32_t tops[4];
    lds_poison_start(&out[0], 1024);
    const int t = threadIdx.x;
    const int64_t c = blockIdx.x % kc, nb = blockIdx.x / kc;
    const int col = 8 * (t & 15), row = 8 * (t >> 4);
    const int64_t k0 = c * 128 + row, n0 = nb * 128 + col;
    u32x4 v[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        v[r] = u32x4{0, 0, 0, 0};
        const int64_t k = k0 + r;
        if (k >= K) continue;
        if constexpr (VEC) {                     // N % 8 == 0 and W on 16 bytes
            if (n0 < N) v[r] = *(const u32x4*)(W + k * N + n0);
        } else {
            uint32_t h[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] = n0 + i < N ? W[k * N + n0 + i] : 0u;
            v[r] = u32x4{h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16};
        }
    }
    uint32_t top = 0;
#pragma unroll
    for (int r = 0; r < 8; ++r) {
        float x[8];
        widen8(v[r], x);
        top = max(top, fp8_top8(x));
    }
    top = max16(top);
    top = max(top, (uint32_t)__shfl_xor((int)top, 16, kWave));
    top = max(top, (uint32_t)__shfl_xor((int)top, 32, kWave));
    if ((t & 63) == 0) tops[t >> 6] = top;
    __syncthreads();
    const Fp8Scale f = fp8_scale(max(max(tops[0], tops[1]), max(tops[2], tops[3])));
    if (t == 0) scales[nb * kc + c] = f.s;
    // column n's eight consecutive channels: bytes (row % 16) .. + 7 of piece 16 g + i of unit 2 f + h
    const int h = row >> 6, g = row >> 4 & 3;
#pragma unroll
    for (int n = 0; n < 8; ++n) {
        float p[8];
#pragma unroll
        for (int r = 0; r < 8; ++r) p[r] = n & 1 ? bf16_hi(v[r][n / 2]) : bf16_lo(v[r][n / 2]);
        const int cn = col + n, tile = cn >> 6, fr = cn >> 4 & 3, i = cn & 15;
        *(uint2*)((uint8_t*)out + ((tile * 8 + 2 * fr + h) * 64 + 16 * g + i) * 16 + (row & 15)) = fp8_codes8(p, f);
    }
    __syncthreads();
    const int64_t nt = (N + 63) / 64;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int piece = q * 256 + t;
        const int64_t tile = nb * 2 + (piece >> 9);
        if (tile < nt) *(u32x4*)(codes + (tile * kc + c) * 8192 + (piece & 511) * 16) = out[piece];
    }
}

}  // namespace

hipError_t launch_fp8_quantize(const uint16_t* X, const uint16_t* gate, int64_t M, int64_t K, uint8_t* codes,
                               float* scales, hipStream_t st) {
    const int64_t cols = (K / 8 + 63) / 64, quads = (M + 3) / 4;
    int R = 1;
    while ((quads + R - 1) / R > 65535) R *= 2;
    const dim3 grid((unsigned)cols, (unsigned)((quads + R - 1) / R));
    if (gate) k_fp8_quantize<true><<<grid, 256, 0, st>>>(X, gate, M, K, codes, scales, R);
    else k_fp8_quantize<false><<<grid, 256, 0, st>>>(X, gate, M, K, codes, scales, R);
    return hipGetLastError();
}

hipError_t launch_fp8_pack(const uint16_t* W, int64_t K, int64_t N, uint8_t* codes, float* scales, hipStream_t st) {
    const int64_t kc = fp8_kc(K);
    const unsigned grid = (unsigned)(kc * fp8_nb(N));
    if (N % 8 == 0 && (uintptr_t)W % 16 == 0) k_fp8_pack<true><<<grid, 256, 0, st>>>(W, K, N, kc, codes, scales);
    else k_fp8_pack<false><<<grid, 256, 0, st>>>(W, K, N, kc, codes, scales);
    return hipGetLastError();
}

}  // namespace awq
