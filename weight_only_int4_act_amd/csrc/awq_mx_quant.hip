// Activations into MX blocks: the quantizer (with an optional gate) and the root-mean-square norm.
#include <algorithm>

#include "awq_mx.h"

namespace awq {
namespace {

// ---------------------------------------------------------------- quantizer
// p = x, or silu(g) x = x g / (1 + e^-g), divided by s per channel.  A thread owns eight channels
// (one 16-byte load) of one row; four consecutive lanes hold a block.
template <int BITS>
__global__ __launch_bounds__(256) void k_mx_quantize(const uint16_t* __restrict__ X,
                                                     const uint16_t* __restrict__ gate, int64_t M, int64_t K,
                                                     const float* __restrict__ s, uint8_t* __restrict__ codes,
                                                     uint8_t* __restrict__ scales) {
    const int64_t octs = K / 8;
    const int64_t oct = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (oct >= octs) return;                     // octs % 4 == 0: a block's four lanes leave together
    for (int64_t m = blockIdx.y; m < M; m += gridDim.y) {
        float x[8];
        bf16x8_to_f32(*(const u32x4*)(X + m * K + oct * 8), x);
        if (gate) {
            float g[8];
            bf16x8_to_f32(*(const u32x4*)(gate + m * K + oct * 8), g);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] *= g[i] / (1.f + expf(-g[i]));
        }
        if (s) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] /= s[oct * 8 + i];
        }
        mx_store8<BITS>(x, codes + m * (BITS == 8 ? K : K / 2), scales + m * (K / kMxBlock), oct);
    }
}

// ---------------------------------------------------------------- root-mean-square norm
// h = x + r, y = h * rsqrt(mean h^2 + eps) * weight.  A workgroup owns a row; the squares are summed
// in float64 (no overflow for any finite row, and one fixed order: lanes, then wavefronts).
__global__ __launch_bounds__(256) void k_rms_norm(const uint16_t* X, const uint16_t* residual,
                                                  const uint16_t* __restrict__ weight, int64_t M, int64_t K,
                                                  float eps, uint16_t* residual_out, uint16_t* Y,
                                                  const float* __restrict__ s, int bits,
                                                  uint8_t* __restrict__ codes, uint8_t* __restrict__ scales) {
    __shared__ double part[4];
    const int64_t octs = K / 8;
    for (int64_t m = blockIdx.x; m < M; m += gridDim.x) {
        auto load = [&](int64_t oct, float (&h)[8]) {
            bf16x8_to_f32(*(const u32x4*)(X + m * K + oct * 8), h);
            if (residual) {
                float r[8];
                bf16x8_to_f32(*(const u32x4*)(residual + m * K + oct * 8), r);
#pragma unroll
                for (int i = 0; i < 8; ++i) h[i] += r[i];
            }
        };
        double sum = 0.;
        for (int64_t oct = threadIdx.x; oct < octs; oct += 256) {
            float h[8];
            load(oct, h);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += (double)h[i] * (double)h[i];
        }
        sum = wave_sum(sum);
        __syncthreads();
        if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
        __syncthreads();
        const float rstd = (float)(1. / sqrt((part[0] + part[1] + part[2] + part[3]) / (double)K + (double)eps));
        for (int64_t oct = threadIdx.x; oct < octs; oct += 256) {
            float h[8], w[8];
            load(oct, h);
            auto store = [&](uint16_t* dst) {
                *(u32x4*)(dst + m * K + oct * 8) = u32x4{pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3]),
                                                         pack_bf16x2(h[4], h[5]), pack_bf16x2(h[6], h[7])};
            };
            if (residual_out) store(residual_out);
            bf16x8_to_f32(*(const u32x4*)(weight + oct * 8), w);
#pragma unroll
            for (int i = 0; i < 8; ++i) h[i] = h[i] * rstd * w[i];
            if (Y) store(Y);
            if (!codes) continue;
            if (s) {
#pragma unroll
                for (int i = 0; i < 8; ++i) h[i] /= s[oct * 8 + i];
            }
            if (bits == 8) mx_store8<8>(h, codes + m * K, scales + m * (K / kMxBlock), oct);
            else mx_store8<4>(h, codes + m * (K / 2), scales + m * (K / kMxBlock), oct);
        }
    }
}

}  // namespace

hipError_t launch_mx_quantize(const uint16_t* X, const uint16_t* gate, int64_t M, int64_t K, const float* s, int bits,
                              uint8_t* codes, uint8_t* scales, hipStream_t st) {
    const dim3 grid((unsigned)((K / 8 + 255) / 256), (unsigned)std::min<int64_t>(M, 65535));
    if (bits == 8) k_mx_quantize<8><<<grid, 256, 0, st>>>(X, gate, M, K, s, codes, scales);
    else k_mx_quantize<4><<<grid, 256, 0, st>>>(X, gate, M, K, s, codes, scales);
    return hipGetLastError();
}

hipError_t launch_rms_norm(const uint16_t* X, const uint16_t* residual, const uint16_t* weight, int64_t M, int64_t K,
                           float eps, uint16_t* residual_out, uint16_t* Y, const float* s, int bits, uint8_t* codes,
                           uint8_t* scales, hipStream_t st) {
    k_rms_norm<<<(unsigned)std::min<int64_t>(M, 1 << 20), 256, 0, st>>>(X, residual, weight, M, K, eps, residual_out,
                                                                        Y, s, bits, codes, scales);
    return hipGetLastError();
}

}  // namespace awq
