// MX weights: bf16 [K, N] to 4-bit blocks in the product's tile order, and back.
#include <algorithm>

#include "awq_mx.h"

namespace awq {
namespace {

// A thread owns four adjacent columns of one block (32 rows), so that a wavefront reads 512
// contiguous bytes of each row; a workgroup's four wavefronts take the four blocks of one 128-row
// chunk.  Bound by HBM: 2 bytes read and 0.53 written per weight.
// Tile t holds columns 64t .. 64t+63: codes[(t * kb_all + kb) * 64 + c] is the 16-byte block of column
// 64t + c, and scale byte 4i + j of (t, kb) belongs to column 64t + 16j + i, so that one 4-byte load
// gives a lane of the matrix-core product the scales of its four 16-column fragments.
__device__ __forceinline__ int scale_pos(int c) { return 4 * (c & 15) + (c >> 4); }

template <bool VEC>
__global__ __launch_bounds__(256) void k_mx_pack(const uint16_t* __restrict__ W, int64_t K, int64_t N,
                                                 const float* __restrict__ s, uint8_t* __restrict__ codes,
                                                 uint8_t* __restrict__ scales, int64_t kb_all) {
    const int lane = threadIdx.x & 63;
    const int64_t kb = (int64_t)blockIdx.y * 4 + (threadIdx.x >> 6);
    const int64_t n0 = ((int64_t)blockIdx.x * 64 + lane) * 4;
    if (n0 >= (N + kMxTile - 1) / kMxTile * kMxTile) return;
    float p[4][32];
    const bool in_k = kb * kMxBlock < K;         // K % 32 == 0: a block is inside or outside as a whole
#pragma unroll
    for (int r = 0; r < 32; ++r) {
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        if (in_k) {
            const int64_t k = kb * kMxBlock + r;
            const uint16_t* row = W + k * N + n0;
            if (VEC) {                           // N % 4 == 0: n0 < N implies n0 + 3 < N
                if (n0 < N) {
                    const uint2 w = *(const uint2*)row;
                    v[0] = bf16_lo(w.x), v[1] = bf16_hi(w.x), v[2] = bf16_lo(w.y), v[3] = bf16_hi(w.y);
                }
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (n0 + c < N) v[c] = bf16_lo((uint32_t)row[c]);
            }
            if (s) {
                const float sk = s[k];
#pragma unroll
                for (int c = 0; c < 4; ++c) v[c] *= sk;
            }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) p[c][r] = v[c];
    }
    const int64_t base = (n0 / kMxTile * kb_all + kb) * kMxTile;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int col = (int)(n0 % kMxTile) + c;
        const bool in = n0 + c < N;              // a column past N is stored as zeros
        uint32_t top = 0;
#pragma unroll
        for (int r = 0; r < 32; ++r) top = max(top, __float_as_uint(p[c][r]) & 0x7fffffffu);
        const uint32_t E = in ? mx_scale_byte<4>(top) : 0u;
        const bool zero = !in || E == 255;
        const float f = mx_to_stored(E == 255 ? 127 : E);
        u32x4 out;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            float q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = zero ? 0.f : p[c][8 * w + i] * f;
            out[w] = mx_e2m1x8(q);
        }
        *(u32x4*)(codes + (base + col) * 16) = out;
        scales[base + scale_pos(col)] = (uint8_t)E;
    }
}

// The reverse: a thread reads four adjacent 16-byte blocks and writes four columns of 32 rows.
template <bool VEC>
__global__ __launch_bounds__(256) void k_mx_unpack(const uint8_t* __restrict__ codes,
                                                   const uint8_t* __restrict__ scales, int64_t K, int64_t N,
                                                   const float* __restrict__ s, uint16_t* __restrict__ W,
                                                   int64_t kb_all) {
    const int lane = threadIdx.x & 63;
    const int64_t kb = (int64_t)blockIdx.y * 4 + (threadIdx.x >> 6);
    const int64_t n0 = ((int64_t)blockIdx.x * 64 + lane) * 4;
    if (n0 >= N || kb * kMxBlock >= K) return;
    const int64_t base = (n0 / kMxTile * kb_all + kb) * kMxTile;
    u32x4 w[4];
    float f[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int col = (int)(n0 % kMxTile) + c;
        w[c] = *(const u32x4*)(codes + (base + col) * 16);
        f[c] = mx_to_value(scales[base + scale_pos(col)]);
    }
#pragma unroll
    for (int r = 0; r < 32; ++r) {
        const int64_t k = kb * kMxBlock + r;
        float v[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const uint32_t code = (w[c][r / 8] >> (4 * (r % 8))) & 15u;
            const uint32_t e = (code >> 1) & 3u, m = code & 1u;
            const float a = e == 0 ? 0.5f * (float)m : __uint_as_float(((126u + e) << 23) | (m << 22));
            v[c] = (code & 8u ? -a : a) * f[c];
            if (s) v[c] /= s[k];
        }
        uint16_t* row = W + k * N + n0;
        const uint2 out = uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        if (VEC) {
            *(uint2*)row = out;
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c)
                if (n0 + c < N) row[c] = (uint16_t)((c < 2 ? out.x : out.y) >> (16 * (c & 1)));
        }
    }
}

}  // namespace

hipError_t launch_mx_pack(const uint16_t* W, int64_t K, int64_t N, const float* s, uint8_t* codes, uint8_t* scales,
                          hipStream_t st) {
    const int64_t kb = mx_kb(K);
    const dim3 grid((unsigned)((mx_nt(N) * kMxTile + 255) / 256), (unsigned)(kb / 4));
    const bool vec = N % 4 == 0 && (uintptr_t)W % 8 == 0;
    if (vec) k_mx_pack<true><<<grid, 256, 0, st>>>(W, K, N, s, codes, scales, kb);
    else k_mx_pack<false><<<grid, 256, 0, st>>>(W, K, N, s, codes, scales, kb);
    return hipGetLastError();
}

hipError_t launch_mx_unpack(const uint8_t* codes, const uint8_t* scales, int64_t K, int64_t N, const float* s,
                            uint16_t* W, hipStream_t st) {
    const int64_t kb = mx_kb(K);
    const dim3 grid((unsigned)((N + 255) / 256), (unsigned)(kb / 4));
    const bool vec = N % 4 == 0 && (uintptr_t)W % 8 == 0;
    if (vec) k_mx_unpack<true><<<grid, 256, 0, st>>>(codes, scales, K, N, s, W, kb);
    else k_mx_unpack<false><<<grid, 256, 0, st>>>(codes, scales, K, N, s, W, kb);
    return hipGetLastError();
}

}  // namespace awq
