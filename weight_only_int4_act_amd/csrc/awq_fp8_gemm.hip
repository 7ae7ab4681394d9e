// The product of e4m3 activations and e4m3 weights with a float32 scale per group of 128:
//   Y[m, n] = sum over groups c of sx[m, c] sw[n / 128, c] * (sum of 128 element products),
// each group's sum on the matrix cores (16x16x128 products, unscaled, into a zero accumulator), the groups added in float32
// by the vector units, one rounding to bf16.
//
// Operands of the 16x16x128 product, lane (i, g) = (lane % 16, lane / 16): bytes 16g .. 16g+15 of the group's
// 128 and bytes 64+16g .. 64+16g+15.  First operand: the weights.  Results: lane (i, g), element r = weight
// column 4g + r, row i: so the two scales of a result are one factor per lane and row fragment.
#include <algorithm>

#include "awq_buffer.h"
#include "awq_fp8.h"

namespace awq {
namespace {

// A group's sum; scale operands of zero select the unscaled product.
__device__ __forceinline__ floatx4 fp8_mfma(const i32x8& w, const i32x8& x) {
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, floatx4{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ i32x8 join8(const u32x4& a, const u32x4& b) {
    return i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

// ---------------------------------------------------------------- few rows: weights streamed once
// Bound by the weights' bytes.  A workgroup owns 64 columns (one tile of packed weights, contiguous in memory), up to
// 16 RF rows and a slice of K; its NW wavefronts take every NW-th group of channels, one in flight each, in registers: 8 KB
// of codes by non-temporal loads, and the rows' elements and scales (repeated reads that the caches serve).  A load past
// the slice, past K or past the last row lies outside its buffer resource: it brings zeros and costs no
// traffic.  The wavefronts' sums meet in LDS in a fixed order; with several slices the last workgroup to arrive
// adds the float32 partials in slice order.
template <int RF, int NW>
__global__ __launch_bounds__(64 * NW) void k_fp8_gemm_rows(
    const uint8_t* __restrict__ xcodes, const float* __restrict__ xscales, int64_t M,
    const uint8_t* __restrict__ codes, const float* __restrict__ scales, int64_t K, int64_t N, int chunks,
    uint16_t* __restrict__ Y, float* __restrict__ part, uint32_t* __restrict__ cnt, int cstride) {
    __shared__ floatx4 red[NW][RF][4][64];
    __shared__ uint32_t arrival;
    lds_poison_start(&red[0][0][0][0], NW * RF * 4 * 64);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int i = lane & 15, g = lane >> 4;
    const int64_t tile = blockIdx.x, m0 = (int64_t)blockIdx.z * 16 * RF;
    const int rows = (int)min<int64_t>(16 * RF, M - m0);
    const int z = blockIdx.y, nz = gridDim.y, per = (chunks + nz - 1) / nz;
    const int cb = min(z * per, chunks), ce = min(cb + per, chunks);
    const uint32_t xrow = (uint32_t)K;
    const __amdgpu_buffer_rsrc_t wr = rsrc(codes + tile * chunks * 8192, (int64_t)chunks * 8192);
    const __amdgpu_buffer_rsrc_t fr = rsrc(scales + tile / 2 * chunks, (int64_t)chunks * 4);
    const __amdgpu_buffer_rsrc_t xr = rsrc(xcodes + m0 * K, (int64_t)rows * xrow);
    const __amdgpu_buffer_rsrc_t sr = rsrc(xscales + m0 * chunks, (int64_t)rows * chunks * 4);

    struct Buf {
        u32x4 w[8], x[RF][2];
        float sw, sx[RF];
    };
    auto issue = [&](int c, Buf& b) {
        const bool in = c < ce;
        const uint32_t wo = in ? (uint32_t)c * 8192 + lane * 16 : kOutside;
#pragma unroll
        for (int rf = 0; rf < RF; ++rf) {
            const uint32_t r = rf * 16 + i;
            const bool inx = in && (int)r < rows;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t k = (uint32_t)c * 128 + h * 64 + g * 16;
                b.x[rf][h] = __builtin_bit_cast(
                    u32x4, __builtin_amdgcn_raw_buffer_load_b128(xr, inx && k < xrow ? r * xrow + k : kOutside, 0, 0));
            }
            b.sx[rf] = __uint_as_float(
                __builtin_amdgcn_raw_buffer_load_b32(sr, inx ? (r * (uint32_t)chunks + c) * 4 : kOutside, 0, 0));
        }
        b.sw = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(fr, in ? (uint32_t)c * 4 : kOutside, 0, 0));
#pragma unroll
        for (int j = 0; j < 8; ++j)
            b.w[j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(wr, wo, j * 1024, kCpolStream));
    };
    floatx4 acc[RF][4];
#pragma unroll
    for (int rf = 0; rf < RF; ++rf)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[rf][j] = floatx4{0.f, 0.f, 0.f, 0.f};
    auto consume = [&](const Buf& b) {
#pragma unroll
        for (int rf = 0; rf < RF; ++rf) {
            const i32x8 x = join8(b.x[rf][0], b.x[rf][1]);
            const float f = b.sx[rf] * b.sw;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const floatx4 p = fp8_mfma(join8(b.w[2 * j], b.w[2 * j + 1]), x);
#pragma unroll
                for (int r = 0; r < 4; ++r) acc[rf][j][r] = fmaf(p[r], f, acc[rf][j][r]);
            }
        }
    };
    Buf buf;
    issue(cb + wave, buf);
    for (int c = cb + wave; c < ce; c += NW) {
        consume(buf);
        issue(c + NW, buf);
    }
    // the products must not move into the branches below: they need every lane's operands
#pragma unroll
    for (int rf = 0; rf < RF; ++rf)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            asm volatile("" : "+v"(acc[rf][j]));
            red[wave][rf][j][lane] = acc[rf][j];
        }
    __syncthreads();
    // the joins: wavefront w takes fragment w % 4 and, with eight wavefronts, half of the row fragments
    constexpr int P = NW / 4, RP = (RF + P - 1) / P;
    const int frag = wave % 4, rf0 = wave / 4 * RP;
    floatx4 sum[RP];                             // columns 16 frag + 4g .. + 3
#pragma unroll
    for (int q = 0; q < RP; ++q) {
        const int rf = min(rf0 + q, RF - 1);
        sum[q] = red[0][rf][frag][lane];
#pragma unroll
        for (int w = 1; w < NW; ++w) sum[q] += red[w][rf][frag][lane];
    }
    const int64_t n = tile * kFp8Tile + 16 * frag + 4 * g;
    auto write_y = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int q = 0; q < RP; ++q) {
            const int r = (rf0 + q) * 16 + i;
            if (rf0 + q < RF && r < rows && n < N)   // N % 8 == 0: n < N implies n + 3 < N
                *(uint2*)(Y + (m0 + r) * N + n) =
                    uint2{pack_bf16x2(sum[q][0], sum[q][1]), pack_bf16x2(sum[q][2], sum[q][3])};
        }
    };
    if (nz == 1) {
        write_y();
        return;
    }
    constexpr uint32_t kPart = RF * 4 * 1024;
    const int64_t slot = (int64_t)blockIdx.z * gridDim.x + tile;
    const __amdgpu_buffer_rsrc_t pr = rsrc(part + slot * nz * (kPart / 4), (int64_t)nz * kPart);
    uint32_t* const counter = cnt + slot * cstride;
    auto poff = [&](int s, int q) {
        return rf0 + q < RF ? (uint32_t)(s * kPart + ((rf0 + q) * 4 + frag) * 1024 + lane * 16) : kOutside;
    };
#pragma unroll
    for (int q = 0; q < RP; ++q) store4_agent(pr, poff(z, q), sum[q]);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // this wavefront's partial has landed
    __syncthreads();
    if (threadIdx.x == 0) arrival = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (arrival != (uint32_t)(nz - 1)) return;
#pragma unroll
    for (int q = 0; q < RP; ++q) sum[q] = floatx4{0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < nz; s += 8) {            // eight slices' loads in flight; past the last: zeros
        floatx4 v[8][RP];
#pragma unroll
        for (int u = 0; u < 8; ++u)
#pragma unroll
            for (int q = 0; q < RP; ++q) v[u][q] = load4_agent(pr, s + u < nz ? poff(s + u, q) : kOutside);
#pragma unroll
        for (int u = 0; u < 8; ++u)
#pragma unroll
            for (int q = 0; q < RP; ++q) sum[q] += v[u][q];
    }
    write_y();
    if (threadIdx.x == 0) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

}  // namespace

constexpr size_t kCounterBytes = 65536;
constexpr int kCus = kNumXcd * kCusPerXcd;
constexpr int kMaxSlices = 16;

Fp8GemmPlan plan_fp8_gemm(int64_t M, int64_t K, int64_t N) {
    Fp8GemmPlan p{};
    const int64_t chunks = fp8_kc(K);
    p.col_tiles = fp8_nt(N);
    const int rf = M <= 16 ? 1 : M <= 32 ? 2 : 4;
    p.row_tiles = (M + 16 * rf - 1) / (16 * rf);
    const int64_t groups = p.col_tiles * p.row_tiles;
    p.nz = 1;
    if (groups <= (int64_t)(kCounterBytes / 4))
        while (p.nz < kMaxSlices && groups * p.nz * 2 <= kCus && chunks / (p.nz * 2) >= 4) p.nz *= 2;
    p.cstride = (int)std::max<int64_t>(1, std::min<int64_t>(32, kCounterBytes / 4 / groups));
    p.ws_bytes = p.nz > 1 ? kCounterBytes + (size_t)groups * p.nz * rf * 4096 : 0;
    return p;
}

template <int RF, int NW>
static hipError_t launch_rows(const uint8_t* xcodes, const float* xscales, int64_t M, const uint8_t* codes,
                              const float* scales, int64_t K, int64_t N, uint16_t* Y, void* ws, const Fp8GemmPlan& p,
                              hipStream_t st) {
    k_fp8_gemm_rows<RF, NW><<<dim3((unsigned)p.col_tiles, (unsigned)p.nz, (unsigned)p.row_tiles), 64 * NW, 0, st>>>(
        xcodes, xscales, M, codes, scales, K, N, (int)fp8_kc(K), Y, (float*)((char*)ws + kCounterBytes), (uint32_t*)ws,
        p.cstride);
    return hipGetLastError();
}

hipError_t launch_fp8_gemm(const uint8_t* xcodes, const float* xscales, int64_t M, const uint8_t* codes,
                           const float* scales, int64_t K, int64_t N, uint16_t* Y, void* ws, const Fp8GemmPlan& p,
                           hipStream_t st) {
    const auto run = [&](auto f) { return f(xcodes, xscales, M, codes, scales, K, N, Y, ws, p, st); };
    if (M <= 16) return run(launch_rows<1, 8>);
    if (M <= 32) return run(launch_rows<2, 4>);
    return run(launch_rows<4, 4>);
}

}  // namespace awq
