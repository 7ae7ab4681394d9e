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

// ---------------------------------------------------------------- rows by the hundred: tiles in LDS
// 64 WM rows x 256 columns per workgroup, WM x WN wavefronts, each with 64 rows and 256/WN columns in
// registers.  Per 128-channel chunk both operands are copied once per workgroup straight into LDS
// (three stages: while chunk c is multiplied, c+1 has landed or is landing and c+2 is requested), in
// the order in which the matrix core's lanes read them back:
//   activations  1 KB per 16 rows and 64 bytes of each row: slot 4r + (p ^ (r/4 % 4)) holds piece p
//                (16 bytes) of row r, so that the 16 lanes that read one piece of 16 rows hit 64
//                different banks;
//   weights      the packed order: 1 KB per block of 64 columns, read 256 contiguous bytes at a time;
//   scales       weights: 64 bytes per block and 64 columns; activations: the bytes of four chunks at
//                a time, from the 4-byte boundary at or before them (16 bytes and 4 more per row).
// Every transfer is issued from inline asm and waited for with counted vmcnt waits (transfers of a
// wavefront complete in order); the barrier after the wait publishes the stage to all wavefronts, and
// says that nobody reads the stage before any more, which is the next one to be refilled.
typedef int i32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ i32x4 byte_rsrc(const void* base, uint32_t bytes) {
    const uint64_t a = (uint64_t)(uintptr_t)base;
    return i32x4{(int)__builtin_amdgcn_readfirstlane((uint32_t)a),
                 (int)(__builtin_amdgcn_readfirstlane((uint32_t)(a >> 32)) & 0xffff),
                 (int)__builtin_amdgcn_readfirstlane(bytes), 0x00020000};
}
// 16 (4) bytes per lane from byte voff + soff of the resource to LDS address lds + 16 (4) * lane; a lane
// whose voff is at or past the resource's end brings zeros.
__device__ __forceinline__ void dma16(i32x4 rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
    uint32_t saved;
    asm volatile(
        "s_mov_b32 %0, m0\n\t"
        "s_mov_b32 m0, %4\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %1, %2, %3 offen lds\n\t"
        "s_mov_b32 m0, %0"
        : "=&s"(saved)
        : "v"(voff), "s"(rsrc), "s"(__builtin_amdgcn_readfirstlane(soff)), "s"(__builtin_amdgcn_readfirstlane(lds))
        : "memory");
}
__device__ __forceinline__ void dma4(i32x4 rsrc, uint32_t voff, uint32_t soff, uint32_t lds) {
    uint32_t saved;
    asm volatile(
        "s_mov_b32 %0, m0\n\t"
        "s_mov_b32 m0, %4\n\t"
        "s_nop 0\n\t"
        "buffer_load_dword %1, %2, %3 offen lds\n\t"
        "s_mov_b32 m0, %0"
        : "=&s"(saved)
        : "v"(voff), "s"(rsrc), "s"(__builtin_amdgcn_readfirstlane(soff)), "s"(__builtin_amdgcn_readfirstlane(lds))
        : "memory");
}
constexpr uint32_t kOutside = 0x80000000u;   // a voff past every resource (all are below 2 GiB)

__device__ __forceinline__ void store4_agent(__amdgpu_buffer_rsrc_t r, uint32_t off, floatx4 v) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), r, off, 0, 16);
}
__device__ __forceinline__ floatx4 load4_agent(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(floatx4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 16));
}

// The results of four 16-column fragments for 16 rows (lane (i, g): row i, columns 16j + 4g .. + 3 of
// fragment j) as bf16, rearranged so that lane (i, g) holds columns 16g .. 16g + 15 of row i: a 4 x 4
// transposition between fragments and lane groups.
__device__ __forceinline__ void mx_rows16(const floatx4 (&v)[4], u32x4 (&out)[2]) {
    uint32_t p[4][2];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        p[j][0] = pack_bf16x2(v[j][0], v[j][1]);
        p[j][1] = pack_bf16x2(v[j][2], v[j][3]);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const auto a = __builtin_amdgcn_permlane16_swap(p[0][h], p[1][h], false, false);
        const auto b = __builtin_amdgcn_permlane16_swap(p[2][h], p[3][h], false, false);
        const auto c = __builtin_amdgcn_permlane32_swap(a[0], b[0], false, false);
        const auto d = __builtin_amdgcn_permlane32_swap(a[1], b[1], false, false);
        out[0][h] = c[0];
        out[0][2 + h] = d[0];
        out[1][h] = c[1];
        out[1][2 + h] = d[1];
    }
}

template <int BITS, int WM, int WN>
struct TileShape {
    static constexpr int kWaves = WM * WN, kRows = 64 * WM, kCols = 256;
    static constexpr int kHalves = BITS == 8 ? 2 : 1;             // 64-byte pieces of a row's chunk
    static constexpr int kXk = kRows / 16 * kHalves;              // 1 KB units of activations per chunk
    static constexpr int kWk = kCols / 64 * 4;                    // 1 KB units of weights per chunk
    static constexpr int kData = (kXk + kWk) / kWaves;            // transfers per wavefront and chunk
    static_assert(kXk % kWaves == 0 && kWk % kWaves == 0, "even shares");
    static constexpr int kStage = (kXk + kWk + 1) * 1024;         // and 1 KB of weight scales
    static constexpr int kXs = kRows * 20;                        // activation scales of four chunks
    static constexpr int kLds = 3 * kStage + 2 * kXs;
};

template <int BITS, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN) void k_mx_gemm_tile(
    const uint8_t* __restrict__ xcodes, const uint8_t* __restrict__ xscales, int64_t M,
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t K, int64_t N, int64_t kb_all,
    uint16_t* __restrict__ Y, float* __restrict__ part, uint32_t* __restrict__ cnt, int row_tiles, int col_tiles,
    int nz, int total, int per_xcd) {
    using S = TileShape<BITS, WM, WN>;
    constexpr int CF = 16 / WN;                  // 16-column fragments per wavefront
    extern __shared__ u32x4 lds[];
    const int logical = xcd_tile(blockIdx.x, per_xcd);
    if (logical >= total) return;
    const int tiles = row_tiles * col_tiles;
    const int z = logical / tiles, tile = logical % tiles;
    // eight row tiles by four column tiles at a time share an XCD's L2
    const int panel = tile / (8 * col_tiles), in = tile % (8 * col_tiles);
    const int prow = min(8, row_tiles - 8 * panel);
    const int rt = 8 * panel + in % prow, ct = in / prow;

    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int i = lane & 15, g = lane >> 4;
    const int wm = wave / WN, wn = wave % WN;
    const int chunks = (int)(kb_all / 4), per = (chunks + nz - 1) / nz;
    const int cb = min(z * per, chunks), ce = min(cb + per, chunks);
    const int64_t row0 = (int64_t)rt * S::kRows, t0 = (int64_t)ct * 4, nt = (N + 63) / 64;
    const int rows = (int)min<int64_t>(S::kRows, M - row0);       // rows past the last repeat it
    const uint32_t xrow = (uint32_t)(BITS == 8 ? K : K / 2), srow = (uint32_t)(K / kMxBlock);

    const uint32_t base = (uint32_t)(uintptr_t)lds;
    const i32x4 xr = byte_rsrc(xcodes + row0 * xrow, (uint32_t)rows * xrow);
    const i32x4 wr = byte_rsrc(codes + t0 * kb_all * 1024, (uint32_t)(min<int64_t>(4, nt - t0) * kb_all * 1024));
    const i32x4 fr = byte_rsrc(scales + t0 * kb_all * 64, (uint32_t)(min<int64_t>(4, nt - t0) * kb_all * 64));
    const uint8_t* s0 = xscales + row0 * srow;
    const uint32_t mis = (uint32_t)((uintptr_t)s0 & 3);           // read whole aligned words
    const i32x4 sr = byte_rsrc(s0 - mis, ((uint32_t)rows * srow + mis + 3) / 4 * 4);

    uint32_t xoff[S::kXk / S::kWaves], woff[S::kWk / S::kWaves];
    int xk[S::kXk / S::kWaves];                  // first channel of the lane's piece within a chunk
#pragma unroll
    for (int u = 0; u < S::kXk / S::kWaves; ++u) {
        const int e = u * S::kWaves + wave, rf = e / S::kHalves, h = e % S::kHalves;
        const int r = lane >> 2, p = (lane & 3) ^ ((r >> 2) & 3);
        xoff[u] = (uint32_t)min(rf * 16 + r, rows - 1) * xrow + 64 * h + 16 * p;
        xk[u] = BITS == 8 ? 64 * h + 16 * p : 32 * p;
    }
#pragma unroll
    for (int u = 0; u < S::kWk / S::kWaves; ++u) {
        const int e = u * S::kWaves + wave;
        woff[u] = (uint32_t)(min<int64_t>(e / 4, nt - t0 - 1) * kb_all * 1024 + (e % 4) * 1024 + lane * 16);
    }
    const uint32_t foff = (uint32_t)(min<int64_t>(lane / 16, nt - t0 - 1) * kb_all * 64 + (lane % 16) * 16);
    // activation scales of chunks 4q .. 4q+3: the first WM wavefronts bring 16 bytes of 64 rows each, the
    // next WM the 4 bytes after them
    static_assert(2 * WM <= S::kWaves, "a wavefront per part");
    const bool wide = wave < WM;
    const int spart = wide ? wave : wave - WM;
    const uint32_t soff = (((uint32_t)min(spart * 64 + lane, rows - 1) * srow + mis) & ~3u) + (wide ? 0 : 16);
    const uint32_t sdst = wide ? spart * 1024 : S::kRows * 16 + spart * 256;
    auto issue_scales = [&](int q) {
        const uint32_t dst = 3 * S::kStage + (q & 1) * S::kXs + sdst, from = 16u * (uint32_t)min(q, (chunks - 1) >> 2);
        if (wave >= 2 * WM) return;
        if constexpr (kLdsPoison) {              // debug build: scales of about 2^120 where these will land
            if (wide) lds[dst / 16 + lane] = lds_nan16();
            else ((uint32_t*)lds)[dst / 4 + lane] = kLdsNan;
            lds_write_fence();
        }
        if (wide) dma16(sr, soff + from, 0, base + dst);
        else dma4(sr, soff + from, 0, base + dst);
    };
    auto issue = [&](int c, int stage) {
        const uint32_t st = base + stage * S::kStage;
        if constexpr (kLdsPoison) {              // debug build: NaN where this wavefront's transfers will land
            u32x4* l = lds + stage * (S::kStage / 16);
#pragma unroll
            for (int u = 0; u < S::kXk / S::kWaves; ++u) l[(u * S::kWaves + wave) * 64 + lane] = lds_nan16();
#pragma unroll
            for (int u = 0; u < S::kWk / S::kWaves; ++u) l[(S::kXk + u * S::kWaves + wave) * 64 + lane] = lds_nan16();
            if (wave == S::kWaves - 1) l[(S::kXk + S::kWk) * 64 + lane] = lds_nan16();
            lds_write_fence();
        }
        if (wave == S::kWaves - 1) dma16(fr, foff, (uint32_t)c * 256, st + (S::kXk + S::kWk) * 1024);
        const int left = (int)min<int64_t>(K - (int64_t)c * kMxChunk, kMxChunk);
#pragma unroll
        for (int u = 0; u < S::kXk / S::kWaves; ++u)
            dma16(xr, xk[u] < left ? xoff[u] : kOutside, (uint32_t)c * (BITS == 8 ? 128 : 64),
                  st + (u * S::kWaves + wave) * 1024);
#pragma unroll
        for (int u = 0; u < S::kWk / S::kWaves; ++u)
            dma16(wr, woff[u], (uint32_t)c * 4096, st + (S::kXk + u * S::kWaves + wave) * 1024);
    };

    // where this lane's scale byte of each of its four row fragments lies in the group's LDS area
    uint32_t sa[4], sb[4];                       // chunks 0-2 (plus 4 each), chunk 3
#pragma unroll
    for (int rf = 0; rf < 4; ++rf) {
        const int r = wm * 64 + rf * 16 + i;
        const int sh = (int)(((uint32_t)min(r, rows - 1) * srow + mis) & 3);
        sa[rf] = r * 16 + sh + g;
        sb[rf] = sh + g >= 4 ? S::kRows * 16 + r * 4 + sh + g - 4 : r * 16 + 12 + sh + g;
    }

    floatx4 acc[4][CF];
#pragma unroll
    for (int rf = 0; rf < 4; ++rf)
#pragma unroll
        for (int j = 0; j < CF; ++j) acc[rf][j] = floatx4{0.f, 0.f, 0.f, 0.f};

    auto compute = [&](int c, int stage) {
        const u32x4* l = lds + stage * (S::kStage / 16);
        const uint8_t* xs = (const uint8_t*)lds + 3 * S::kStage + ((c >> 2) & 1) * S::kXs;
        const uint32_t* f = (const uint32_t*)(l + (S::kXk + S::kWk) * 64);
        const bool inside = 4 * (int64_t)c + g < K / kMxBlock;    // past K: elements are zero, the scale 1
        uint32_t xe[4], we[CF / 4];
        i32x8 x[4];
        const int slot = i * 4 + (g ^ ((i >> 2) & 3));
#pragma unroll
        for (int rf = 0; rf < 4; ++rf) {
            const uint32_t e = xs[(c & 3) == 3 ? sb[rf] : sa[rf] + 4 * (c & 3)];
            xe[rf] = inside ? e : 127u;
            const u32x4 a = l[((wm * 4 + rf) * S::kHalves) * 64 + slot];
            u32x4 b = u32x4{0, 0, 0, 0};
            if constexpr (BITS == 8) b = l[((wm * 4 + rf) * S::kHalves + 1) * 64 + slot];
            x[rf] = i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
        }
#pragma unroll
        for (int w = 0; w < CF / 4; ++w) we[w] = f[(wn * (CF / 4) + w) * 64 + g * 16 + i];
#pragma unroll
        for (int j = 0; j < CF; j += 4) {
            const int t4 = wn * (CF / 4) + j / 4;
            u32x4 w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) w[q] = l[(S::kXk + t4 * 4 + g) * 64 + 16 * q + i];
#pragma unroll
            for (int rf = 0; rf < 4; ++rf) acc[rf][j] = mx_mfma<BITS, 0>(w[0], x[rf], acc[rf][j], we[j / 4], xe[rf]);
#pragma unroll
            for (int rf = 0; rf < 4; ++rf) acc[rf][j + 1] = mx_mfma<BITS, 1>(w[1], x[rf], acc[rf][j + 1], we[j / 4], xe[rf]);
#pragma unroll
            for (int rf = 0; rf < 4; ++rf) acc[rf][j + 2] = mx_mfma<BITS, 2>(w[2], x[rf], acc[rf][j + 2], we[j / 4], xe[rf]);
#pragma unroll
            for (int rf = 0; rf < 4; ++rf) acc[rf][j + 3] = mx_mfma<BITS, 3>(w[3], x[rf], acc[rf][j + 3], we[j / 4], xe[rf]);
        }
    };

    // Past the last chunk the transfers are issued all the same (the last chunk's, into a stage that
    // nobody reads again), so that the counted waits stay the same.
    const int last = max(ce - 1, 0);
    issue_scales(cb >> 2);
    issue_scales((cb >> 2) + 1);
    issue(min(cb, last), 0);
    issue(min(cb + 1, last), 1);
    int stage = 0, ahead = 2;
    for (int c = cb; c < ce; ++c) {
        asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(S::kData) : "memory");
        if ((c & 3) == 1) issue_scales((c >> 2) + 1);   // read from the next multiple of 4 on
        issue(min(c + 2, last), ahead);
        compute(c, stage);
        stage = stage == 2 ? 0 : stage + 1;
        ahead = ahead == 2 ? 0 : ahead + 1;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    // the products must not move into the branches below: they need every lane's operands
#pragma unroll
    for (int rf = 0; rf < 4; ++rf)
#pragma unroll
        for (int j = 0; j < CF; ++j) asm volatile("" : "+v"(acc[rf][j]));

    auto write_y = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int rf = 0; rf < 4; ++rf) {
            const int r = wm * 64 + rf * 16 + i;
#pragma unroll
            for (int j = 0; j < CF; j += 4) {
                const floatx4 v[4] = {acc[rf][j], acc[rf][j + 1], acc[rf][j + 2], acc[rf][j + 3]};
                u32x4 out[2];
                mx_rows16(v, out);
                const int64_t n = (t0 + wn * (CF / 4) + j / 4) * kMxTile + 16 * g;
                uint16_t* y = Y + (row0 + r) * N + n;
                if (r < rows && n < N) *(u32x4*)y = out[0];          // N % 8 == 0
                if (r < rows && n + 8 < N) *(u32x4*)(y + 8) = out[1];
            }
        }
    };
    if (nz == 1) {
        write_y();
        return;
    }
    // Split over K: float32 partials in fragment order, one per (tile, K slice), written through to the
    // device-coherent level; the workgroup that arrives last adds them in slice order.
    constexpr uint32_t kPart = S::kRows * S::kCols * 4;
    float* tile_part = part + (int64_t)tile * nz * (kPart / 4);
    const __amdgpu_buffer_rsrc_t pr =
        __builtin_amdgcn_make_buffer_rsrc(tile_part, (short)0, (int)(nz * kPart), 0x00020000);
    auto poff = [&](int s, int rf, int j) { return (uint32_t)(s * kPart + ((wave * 4 + rf) * CF + j) * 1024 + lane * 16); };
#pragma unroll
    for (int rf = 0; rf < 4; ++rf)
#pragma unroll
        for (int j = 0; j < CF; ++j) store4_agent(pr, poff(z, rf, j), acc[rf][j]);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // this wavefront's partial has landed
    __syncthreads();
    uint32_t* arrival = (uint32_t*)lds;
    if (threadIdx.x == 0) *arrival = __hip_atomic_fetch_add(cnt + tile, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (*arrival != (uint32_t)(nz - 1)) return;
#pragma unroll
    for (int rf = 0; rf < 4; ++rf)
#pragma unroll
        for (int j = 0; j < CF; ++j) acc[rf][j] = floatx4{0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < nz; ++s)
#pragma unroll
        for (int rf = 0; rf < 4; ++rf) {
#pragma unroll
            for (int j = 0; j < CF; ++j) acc[rf][j] += load4_agent(pr, poff(s, rf, j));
            __builtin_amdgcn_sched_barrier(0);   // one row fragment's loads in registers at a time
        }
    write_y();
    if (threadIdx.x == 0) __hip_atomic_store(cnt + tile, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

}  // namespace

// Rows beyond which the LDS tiles take over from the register kernel.
constexpr int64_t kTileRows = 64;
constexpr size_t kCounterBytes = 65536;
constexpr int kCus = kNumXcd * kCusPerXcd;

MxGemmPlan plan_mx_gemm(int64_t M, int64_t K, int64_t N, int bits) {
    MxGemmPlan p{};
    if (M <= kTileRows) {
        p.wm = 0;
        p.col_tiles = mx_nt(N);
        p.row_tiles = (M + 15) / 16;
        p.nz = 1;
        return p;
    }
    p.wm = M > 128 ? 4 : 2;
    p.row_tiles = (M + 64 * p.wm - 1) / (64 * p.wm);
    p.col_tiles = (N + 255) / 256;
    const int64_t tiles = p.row_tiles * p.col_tiles, chunks = mx_kb(K) / 4;
    int nz = 1;
    if (tiles < kCus) nz = (int)std::max<int64_t>(1, std::min<int64_t>(kCus / tiles, chunks / 4));
    p.nz = nz;
    if (nz > 1) p.ws_bytes = kCounterBytes + (size_t)tiles * nz * 64 * p.wm * 256 * 4;
    return p;
}

template <int BITS, int WM, int WN>
static hipError_t launch_tile(const uint8_t* xcodes, const uint8_t* xscales, int64_t M, const uint8_t* codes,
                              const uint8_t* scales, int64_t K, int64_t N, uint16_t* Y, void* ws, const MxGemmPlan& p,
                              hipStream_t st) {
    using S = TileShape<BITS, WM, WN>;
    const int64_t total = p.row_tiles * p.col_tiles * p.nz, per_xcd = (total + kNumXcd - 1) / kNumXcd;
    const auto kernel = k_mx_gemm_tile<BITS, WM, WN>;
    // the limit is a property of the function on the current device; setting it again is harmless
    const hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, S::kLds);
    if (e != hipSuccess) return e;
    kernel<<<(unsigned)(per_xcd * kNumXcd), 64 * S::kWaves, S::kLds, st>>>(
        xcodes, xscales, M, codes, scales, K, N, mx_kb(K), Y, (float*)((char*)ws + kCounterBytes), (uint32_t*)ws,
        (int)p.row_tiles, (int)p.col_tiles, p.nz, (int)total, (int)per_xcd);
    return hipGetLastError();
}

hipError_t launch_mx_gemm(const uint8_t* xcodes, const uint8_t* xscales, int bits, int64_t M, const uint8_t* codes,
                          const uint8_t* scales, int64_t K, int64_t N, uint16_t* Y, void* ws, const MxGemmPlan& p,
                          hipStream_t st) {
    if (p.wm == 0) {
        const dim3 grid((unsigned)p.col_tiles, (unsigned)p.row_tiles);
        if (bits == 8) k_mx_gemm<8><<<grid, 256, 0, st>>>(xcodes, xscales, M, codes, scales, K, N, mx_kb(K), Y);
        else k_mx_gemm<4><<<grid, 256, 0, st>>>(xcodes, xscales, M, codes, scales, K, N, mx_kb(K), Y);
        return hipGetLastError();
    }
    const auto run = [&](auto f) { return f(xcodes, xscales, M, codes, scales, K, N, Y, ws, p, st); };
    if (p.wm == 4) return run(bits == 8 ? launch_tile<8, 4, 2> : launch_tile<4, 4, 2>);
    return run(bits == 8 ? launch_tile<8, 2, 4> : launch_tile<4, 2, 4>);
}

}  // namespace awq
