// The product of MX activations (e4m3 or e2m1 elements) and MX weights (e2m1) on the scaled matrix
// cores: Y[m, n] = sum over blocks of 2^(Ex + Ew - 254) * sum of 32 element products, float32
// accumulation, one rounding to bf16.
//
// Operands of the 16x16x128 product, lane (i, g) = (lane % 16, lane / 16).  First operand: the
// weights, so that a lane's four results are four adjacent output columns.  4-bit elements: lane
// (i, g) holds the 32 elements of block g (16 bytes).  8-bit elements: bytes 16g .. 16g+15 of the
// 128 and bytes 64+16g .. 64+16g+15.  In both, the scale byte of lane (i, g) applies to block g
// (channels 32g .. 32g+31).  Results: lane (i, g), element r = weight column 4g + r, row i.
#include <algorithm>

#include "awq_mx.h"

namespace awq {
namespace {

typedef int i32x8 __attribute__((ext_vector_type(8)));

// acc += weights x activations; J: the byte of the weights' scale word, in [0, 4).
template <int BITS, int J>
__device__ __forceinline__ floatx4 mx_mfma(const u32x4& w, const i32x8& x, const floatx4& acc, uint32_t wscale,
                                           uint32_t xscale) {
    const i32x8 a = i32x8{(int)w[0], (int)w[1], (int)w[2], (int)w[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, x, acc, 4, BITS == 8 ? 0 : 4, J, (int)wscale, 0,
                                                            (int)xscale);
}

// 16 rows x 64 columns per workgroup; its four wavefronts take every fourth 128-channel chunk and
// their sums meet in LDS in a fixed order.
template <int BITS>
__global__ __launch_bounds__(256) void k_mx_gemm(const uint8_t* __restrict__ xcodes,
                                                 const uint8_t* __restrict__ xscales, int64_t M,
                                                 const uint8_t* __restrict__ codes,
                                                 const uint8_t* __restrict__ scales, int64_t K, int64_t N,
                                                 int64_t kb_all, uint16_t* __restrict__ Y) {
    __shared__ floatx4 red[3][4][64];
    lds_poison_start(&red[0][0][0], 3 * 4 * 64);
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
    const int64_t tile = blockIdx.x, m = (int64_t)blockIdx.y * 16 + i;
    const int64_t row = min(m, M - 1);           // rows past M repeat the last one and are not stored
    const uint8_t* xr = xcodes + row * (BITS == 8 ? K : K / 2);
    const uint8_t* xs = xscales + row * (K / kMxBlock);
    const int64_t blocks = K / kMxBlock;
    floatx4 acc[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] = floatx4{0.f, 0.f, 0.f, 0.f};
    for (int64_t c = wave; c < kb_all / 4; c += 4) {
        const int64_t kb = 4 * c + g;
        i32x8 x = i32x8{0, 0, 0, 0, 0, 0, 0, 0};
        // past K: zero elements with the scale 1 (the weights are padded with zeros there)
        const uint32_t xe = kb < blocks ? xs[kb] : 127u;
        if constexpr (BITS == 8) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t k = c * kMxChunk + 64 * h + 16 * g;
                if (k < K) {
                    const u32x4 v = *(const u32x4*)(xr + k);
#pragma unroll
                    for (int e = 0; e < 4; ++e) x[4 * h + e] = (int)v[e];
                }
            }
        } else if (kb < blocks) {
            const u32x4 v = *(const u32x4*)(xr + kb * 16);
#pragma unroll
            for (int e = 0; e < 4; ++e) x[e] = (int)v[e];
        }
        const int64_t wb = (tile * kb_all + kb) * kMxTile;
        const uint32_t we = *(const uint32_t*)(scales + wb + 4 * i);
        u32x4 w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = *(const u32x4*)(codes + (wb + 16 * j + i) * 16);
        acc[0] = mx_mfma<BITS, 0>(w[0], x, acc[0], we, xe);
        acc[1] = mx_mfma<BITS, 1>(w[1], x, acc[1], we, xe);
        acc[2] = mx_mfma<BITS, 2>(w[2], x, acc[2], we, xe);
        acc[3] = mx_mfma<BITS, 3>(w[3], x, acc[3], we, xe);
    }
    // the products must not move into the branches below: they need every lane's operands
#pragma unroll
    for (int j = 0; j < 4; ++j) asm volatile("" : "+v"(acc[j]));
    if (wave > 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j) red[wave - 1][j][lane] = acc[j];
    }
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const floatx4 v = ((acc[j] + red[0][j][lane]) + red[1][j][lane]) + red[2][j][lane];
        const int64_t n = tile * kMxTile + 16 * j + 4 * g;
        if (m < M && n < N)                      // N % 8 == 0: n < N implies n + 3 < N
            *(uint2*)(Y + m * N + n) = uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    }
}

}  // namespace

MxGemmPlan plan_mx_gemm(int64_t M, int64_t K, int64_t N, int bits) {
    MxGemmPlan p{};
    p.col_tiles = mx_nt(N);
    p.row_tiles = (M + 15) / 16;
    p.ws_bytes = 0;
    return p;
}

hipError_t launch_mx_gemm(const uint8_t* xcodes, const uint8_t* xscales, int bits, int64_t M, const uint8_t* codes,
                          const uint8_t* scales, int64_t K, int64_t N, uint16_t* Y, void* ws, const MxGemmPlan& p,
                          hipStream_t st) {
    const dim3 grid((unsigned)p.col_tiles, (unsigned)p.row_tiles);
    if (bits == 8) k_mx_gemm<8><<<grid, 256, 0, st>>>(xcodes, xscales, M, codes, scales, K, N, mx_kb(K), Y);
    else k_mx_gemm<4><<<grid, 256, 0, st>>>(xcodes, xscales, M, codes, scales, K, N, mx_kb(K), Y);
    return hipGetLastError();
}

}  // namespace awq
