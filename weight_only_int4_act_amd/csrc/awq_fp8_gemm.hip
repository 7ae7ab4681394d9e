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

// ---------------------------------------------------------------- few rows or little work: operands in registers
// Bound by the weights' bytes up to 32 rows, by latency beyond.  A workgroup owns 64 columns (one tile of packed weights,
// contiguous in memory), up to 16 RF rows and a slice of K; its NW wavefronts take every NW-th group of channels, one in
// flight each, in registers: 8 KB of codes (by non-temporal loads where they are read once), and the rows' elements and
// scales (repeated reads that the caches serve).  A load past the slice, past K or past the last row lies outside its
// buffer resource: it brings zeros and costs no traffic.  The wavefronts' sums meet in LDS in a fixed order; with several
// slices the last workgroup to arrive adds the float32 partials in slice order.  1 x 8192 x 10240, from HBM: 19.0 us (4.4
// TB/s), 1 x 28672 x 8192 41.8 (5.6, a part from the Infinity Cache); two groups in flight per wavefront are no faster.
// 435 x 800 x 136: 5.9 us, where a launch takes 2.2; 420 x 2256 x 568: 10.5, 11.4 with non-temporal loads.
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

    constexpr int kPolicy = RF == 4 ? 0 : kCpolStream;           // weights that other row tiles read, too, stay in the caches
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
            b.w[j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(wr, wo, j * 1024, kPolicy));
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

// ---------------------------------------------------------------- many rows: tiles in LDS
// 64 WM rows x 256 columns per workgroup, WM x WN wavefronts of 64 rows x 32 CF columns, by 32x32x64 products (half the
// operand reads of 16x16x128 ones for the same work).  Lane (i, h) = (lane % 32, lane / 32).  First operand: column i
// of 32 weights; second: row i of 32; both take pieces (16 bytes) 4y + 2h and 4y + 2h + 1 of the group's eight for half y of
// the channels (any order that both share will do).  Results: row i, column 8 (r / 4) + 4h + r % 4: one factor
// sx sw per lane and row fragment.
//
// Both operands of a group are copied once per workgroup straight into LDS, ST groups deep:
//   activations  1 KB units of 8 rows; piece q of row r lies at slot q ^ (r / 2 % 8), so that the lanes that a
//                16-byte read serves together (0-3, 12-15, 20-27 and 4-11, 16-19, 28-31 of either half) hit different banks;
//   weights      the packed order, read 256 contiguous bytes at a time;
//   scales       of four groups at a time, two such sets deep: 16 bytes per row, and 16 per 128 columns.
// Transfers are issued from inline asm and waited for with counted vmcnt waits (those of a wavefront complete in
// order).  A turn multiplies one group in steps of one result fragment: two products, beside them the float32
// additions of the fragment before, the LDS reads of the next weights, a share of the transfers.  Before the last column
// fragment a barrier says that the group is in every wavefront's registers and the next one has landed; its place
// is then filled with group c + ST.
//
// 4096 x 8192 x 28672: 809-890 us by the clock that the card holds (2.2-2.4 PFLOP/s; the matrix cores busy in 64 % of the cycles).
// On one card, 891 us as it is, 843-865 without the float32 additions, 720 without transfers, 647 without both, 813 with
// transfers that always hit the L2: so what the additions cost (a vector instruction per result and group of 128
// channels, where a scale per row alone needs none) and what the transfers cost is power as much as issue.
// 257 x 5120 x 13824: 32 us with the weights in the caches, 38.6 from HBM: 162 tiles of 128 x 256 on 256 CUs, 40 turns of .83 us.
typedef float floatx16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ u32x4 fp8_poison() { return u32x4{~0u, ~0u, ~0u, ~0u}; }   // NaN in e4m3 and in float32

template <int WM, int WN, int CF, int ST>
struct Fp8Tile {
    static constexpr int kWaves = WM * WN, kRows = 64 * WM, kCols = 32 * CF * WN;
    static_assert(kCols == 256 && CF % 2 == 0, "tile shape");
    static constexpr int kXu = kRows / 8 / kWaves, kWu = 32 / kWaves, kData = kXu + kWu;   // 1 KB units per wavefront
    static_assert(kData % 2 == 0 && kXu % 2 == 0 && kXu * kWaves * 8 == kRows && kWu * kWaves == 32, "even shares");
    static constexpr int kX = kRows * 128, kStage = kX + 32768;
    static constexpr int kScaleSet = kRows * 16 + 1024;           // rows, then columns (32 bytes of a transfer's 1 KB)
    static constexpr int kScales = ST * kStage, kLds = kScales + 2 * kScaleSet;
    static_assert(kLds <= 160 * 1024, "LDS of a CU");
};

template <int WM, int WN, int CF, int ST, bool EDGE>
__global__ __launch_bounds__(64 * WM * WN) void k_fp8_gemm_tile(
    const uint8_t* __restrict__ xcodes, const float* __restrict__ xscales, int64_t M, const uint8_t* __restrict__ codes,
    const float* __restrict__ scales, int64_t K, int64_t N, int chunks, uint16_t* __restrict__ Y,
    float* __restrict__ part, int row_tiles, int col_tiles, int nz, int total, int per_xcd) {
    using S = Fp8Tile<WM, WN, CF, ST>;
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
    const int i = lane & 31, h = lane >> 5;
    const int wm = wave / WN, wn = wave % WN;
    const int per = (chunks + nz - 1) / nz;
    const int cb = min(z * per, chunks), ce = min(cb + per, chunks);
    const int64_t row0 = (int64_t)rt * S::kRows, t0 = (int64_t)ct * 4, nt = (N + 63) / 64, nb = (N + 127) / 128;
    const int rows = (int)min<int64_t>(S::kRows, M - row0);       // past the last row and
    const int cts = (int)min<int64_t>(4, nt - t0);                // column tile: zeros
    const uint32_t xrow = (uint32_t)K, srow = (uint32_t)chunks * 4, wtile = (uint32_t)chunks * 8192;
    const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)lds;
    i32x4 xr[S::kXu / 2];                        // one for 16 rows of the wavefront's each
    const i32x4 wr = byte_rsrc(codes + t0 * wtile, (uint32_t)cts * wtile);
    const i32x4 sr = byte_rsrc(xscales + row0 * chunks, (uint32_t)rows * srow);
    const i32x4 fr = byte_rsrc(scales + t0 / 2 * chunks, (uint32_t)min<int64_t>(2, nb - t0 / 2) * srow);

    // this lane's places in its wavefront's transfers
#pragma unroll
    for (int k = 0; k < S::kXu / 2; ++k) {
        const int first = wave * S::kXu * 8 + 16 * k;
        xr[k] = byte_rsrc(xcodes + (row0 + min(first, rows)) * xrow, (uint32_t)max(rows - first, 0) * xrow);
    }
    const int us = lane & 7;
    uint32_t xoff[2];
    int xk[2];                                   // first channel of the piece, units of either parity
#pragma unroll
    for (int k = 0; k < 2; ++k) xk[k] = 16 * (us ^ ((4 * k + lane / 16) & 7));
#pragma unroll
    for (int k = 0; k < 2; ++k) xoff[k] = (uint32_t)(lane / 8 + 8 * k) * xrow + xk[k];
    static_assert(8 % S::kWu == 0, "a wavefront's units lie in one column tile");
    const uint32_t woff = (uint32_t)(wave * S::kWu / 8) * wtile + wave * S::kWu % 8 * 1024 + lane * 16;
    // the scales of the slice's groups 4q .. 4q + 3: 64 rows per wavefront (the same ones by several where there are
    // fewer), and the columns' by every wavefront alike
    const int part64 = wave % WM;
    const uint32_t soff = (uint32_t)(part64 * 64 + lane) * srow + cb * 4;
    const uint32_t foff = lane < 2 ? (uint32_t)lane * srow + cb * 4 : kOutside;
    auto issue_scales = [&](int q) __attribute__((always_inline)) {
        const uint32_t at = S::kScales + (q & 1) * S::kScaleSet;
        if constexpr (kLdsPoison) {
            lds[at / 16 + part64 * 64 + lane] = fp8_poison();
            lds[at / 16 + S::kRows + lane] = fp8_poison();
            lds_write_fence();
        }
        dma16(sr, soff + q * 16, 0, base + at + part64 * 1024, 0);
        dma16(fr, foff + q * 16, 0, base + at + S::kRows * 16, 0);
    };
    // transfer k of group c's batch; for a group past the slice the resources are empty, which brings zeros
    // (no traffic), so that the counted waits stay the same
    auto issue_op = [&](int c, int stage, int k) __attribute__((always_inline)) {
        const bool on = c < ce;
        const uint32_t st = stage * S::kStage;
        const uint32_t to = k < S::kXu ? st + (wave * S::kXu + k) * 1024 : st + S::kX + (wave * S::kWu + k - S::kXu) * 1024;
        if constexpr (kLdsPoison) {
            lds[to / 16 + lane] = fp8_poison();
            lds_write_fence();
        }
        if (k < S::kXu) {
            const i32x4 r = {xr[k / 2][0], xr[k / 2][1], on ? xr[k / 2][2] : 0, xr[k / 2][3]};
            const uint32_t past = !EDGE || xk[k & 1] < (int)xrow - c * 128 ? 0 : kOutside;   // a piece past K
            dma16(r, xoff[k & 1] | past, (uint32_t)c * 128, base + to, 0);
        } else {
            const i32x4 r = {wr[0], wr[1], on ? wr[2] : 0, wr[3]};
            dma16(r, woff, (uint32_t)c * 8192 + (k - S::kXu) * 1024, base + to, 0);
        }
    };

    const uint8_t* const lb = (const uint8_t*)lds;
    uint32_t xl = (wm * 64 + i) * 128 + ((2 * h) ^ (i / 2 & 7)) * 16;   // piece p of half y: ^ (4 y + p) * 16
    const uint32_t wl = S::kX + wn * CF * 4096 + (i / 16) * 2048 + h * 512 + (i & 15) * 16;
    const uint32_t sl = S::kScales + (wm * 64 + i) * 16, fl = S::kScales + S::kRows * 16 + wn * CF * 32 / 128 * 16;

    floatx16 acc[2][CF];
#pragma unroll
    for (int rf = 0; rf < 2; ++rf)
#pragma unroll
        for (int j = 0; j < CF; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[rf][j][r] = 0.f;

    auto pair = [&](uint32_t a, uint32_t b) __attribute__((always_inline)) {
        return join8(*(const u32x4*)(lb + a), *(const u32x4*)(lb + b));
    };
    i32x8 x[2][2], w[2][2];                      // [row fragment][half], [buffer][half]
    auto fetch_x = [&](int stage, int rf) __attribute__((always_inline)) {
        const uint32_t st = stage * S::kStage + rf * 4096;
        asm volatile("" : "+v"(xl));             // four exclusive ors a turn instead of four registers
#pragma unroll
        for (int y = 0; y < 2; ++y) x[rf][y] = pair(st + (xl ^ (64 * y)), st + (xl ^ (64 * y + 16)));
    };
    auto fetch_w = [&](int stage, int j, int y, i32x8& to) __attribute__((always_inline)) {
        const uint32_t at = stage * S::kStage + wl + j * 4096 + y * 1024;
        to = pair(at, at + 256);
    };

    issue_scales(0);
#pragma unroll
    for (int s = 0; s < ST; ++s)
#pragma unroll
        for (int k = 0; k < S::kData; ++k)
            if (s < ST - 1 || k * 4 / S::kData < 2) issue_op(cb + s, s, k);
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((ST - 2) * S::kData + S::kData / 2) : "memory");
    fetch_x(0, 0);
    fetch_x(0, 1);
    fetch_w(0, 0, 0, w[0][0]);
    fetch_w(0, 0, 1, w[0][1]);
    floatx16 p[2];                               // the fragment before, not yet added, and its factor
    float late = 0.f, sw = 0.f;
#pragma unroll
    for (int r = 0; r < 16; ++r) p[1][r] = 0.f;
    const floatx16 zero = p[1];
    int stage = 0;
    for (int c = cb; c < ce; ++c) {
        const int ahead = stage == ST - 1 ? 0 : stage + 1;
        float factor[2];
#pragma unroll
        for (int n = 0; n < 2 * CF; ++n) {
            const int j = n / 2, rf = n % 2, b = j & 1;
            if (n == 2 * CF - 2) {               // every read of this group has been issued
                asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((ST - 2) * S::kData) : "memory");
                if (((c - cb) & 3) == 0) issue_scales((c - cb) / 4 + 1);
            }
            floatx16& now = p[n & 1];
            floatx16& old = p[(n & 1) ^ 1];
            now = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w[b][0], x[rf][0], zero, 0, 0, 0, 0, 0, 0);
            now = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(w[b][1], x[rf][1], now, 0, 0, 0, 0, 0, 0);
            __builtin_amdgcn_sched_barrier(0);
            if (n == 0) {
                const uint32_t set = ((c - cb) / 4 & 1) * S::kScaleSet + ((c - cb) & 3) * 4;
                factor[0] = *(const float*)(lb + sl + set);
                factor[1] = *(const float*)(lb + sl + set + 512);
                sw = *(const float*)(lb + fl + set);
            }
            if (n == 1) factor[0] *= sw, factor[1] *= sw;
            const float g = n == 0 ? late : factor[(n & 1) ^ 1];
            // the next weights; at the end the next group's rows, each where its last product has been issued
            if (j + 1 < CF) fetch_w(stage, j + 1, rf, w[b ^ 1][rf]);
            else fetch_w(ahead, 0, rf, w[b ^ 1][rf]);
            const int oj = n == 0 ? CF - 1 : (n - 1) / 2, orf = n == 0 ? 1 : (n - 1) % 2;
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[orf][oj][r] = fmaf(old[r], g, acc[orf][oj][r]);
            asm volatile("" : "+v"(acc[orf][oj]));   // here, not behind the next barrier
            if (n >= 2 * CF - 2) fetch_x(ahead, rf);
            // the transfers of a batch over four steps: two behind the barrier, two of the next turn
#pragma unroll
            for (int k = 0; k < S::kData; ++k) {
                if (k * 4 / S::kData == n - (2 * CF - 2)) issue_op(c + ST, stage, k);
                if (k * 4 / S::kData == n + 2) issue_op(c + ST - 1, stage == 0 ? ST - 1 : stage - 1, k);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        late = factor[1];
        stage = ahead;
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[1][CF - 1][r] = fmaf(p[1][r], late, acc[1][CF - 1][r]);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");

    // Results leave through a buffer resource, where a row past M or a column past N lies outside: a branch around the
    // stores would let the compiler move products into it, and those need every lane's operands.
    if (nz == 1) {
        const __amdgpu_buffer_rsrc_t yr = rsrc(Y + row0 * N, (int64_t)rows * N * 2);
#pragma unroll
        for (int rf = 0; rf < 2; ++rf) {
            const int r = wm * 64 + rf * 32 + i;
#pragma unroll
            for (int j = 0; j < CF; ++j)
#pragma unroll
                for (int a = 0; a < 4; a += 2) {
                    // columns 8a .. + 7 to the lanes of h = 0, the next eight to those of h = 1
                    const floatx16& v = acc[rf][j];
                    u32x4 out;
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const auto s = __builtin_amdgcn_permlane32_swap(pack_bf16x2(v[4 * a + 2 * e], v[4 * a + 2 * e + 1]),
                                                                        pack_bf16x2(v[4 * a + 4 + 2 * e], v[4 * a + 5 + 2 * e]),
                                                                        false, false);
                        out[e] = s[0];
                        out[2 + e] = s[1];
                    }
                    const int64_t n = t0 * 64 + (wn * CF + j) * 32 + 8 * a + 8 * h;
                    __builtin_amdgcn_raw_buffer_store_b128(out, yr, r < rows && n < N ? (uint32_t)(r * N + n) * 2 : kOutside,
                                                           0, 0);
                }
        }
        return;
    }
    // Split over K: float32 partials in fragment order, one per (tile, K slice), that k_fp8_join adds.
    constexpr uint32_t kPart = S::kRows * 256 * 4;
    const __amdgpu_buffer_rsrc_t pr = rsrc(part + (int64_t)tile * nz * (kPart / 4), (int64_t)nz * kPart);
#pragma unroll
    for (int rf = 0; rf < 2; ++rf)
#pragma unroll
        for (int j = 0; j < CF; ++j)
#pragma unroll
            for (int a = 0; a < 4; ++a) {
                const floatx16& v = acc[rf][j];
                const floatx4 q = {v[4 * a], v[4 * a + 1], v[4 * a + 2], v[4 * a + 3]};
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, q), pr,
                                                       z * kPart + (((wave * 2 + rf) * CF + j) * 4 + a) * 1024 + lane * 16, 0, 0);
            }
}

// Adds the slices of the tiles above: a wavefront takes a quarter of one fragment of every slice, in slice order, eight
// loads in flight.  Bound by the trip to memory: 3 us, and .35 per MB (a load past the last slice that repeats it instead costs
// 257 x 8192 x 8192 .7 us of 40).
template <int WM, int WN, int CF>
__global__ __launch_bounds__(256) void k_fp8_join(const float* __restrict__ part, int64_t M, int64_t N, int row_tiles,
                                                  int col_tiles, int nz, uint16_t* __restrict__ Y) {
    constexpr int kFrags = WM * WN * 2 * CF * 4, kRows = 64 * WM;
    constexpr uint32_t kPart = kFrags * 1024;
    const int lane = threadIdx.x & 63, i = lane & 31, h = lane >> 5;
    const int f = (blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) % kFrags;
    const int tile = blockIdx.x * 4 / kFrags;
    const int panel = tile / (8 * col_tiles), in = tile % (8 * col_tiles), prow = min(8, row_tiles - 8 * panel);
    const int rt = 8 * panel + in % prow, ct = in / prow;
    const int a = f % 4, j = f / 4 % CF, rf = f / (4 * CF) % 2, wave = f / (8 * CF);
    const __amdgpu_buffer_rsrc_t pr = rsrc(part + (int64_t)tile * nz * (kPart / 4), (int64_t)nz * kPart);   // past the last slice: zeros
    floatx4 sum = floatx4{0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < nz; s += 8) {
        floatx4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u)
            v[u] = __builtin_bit_cast(floatx4, __builtin_amdgcn_raw_buffer_load_b128(pr, (uint32_t)(s + u) * kPart + f * 1024 + lane * 16, 0, 0));
#pragma unroll
        for (int u = 0; u < 8; ++u) sum += v[u];
    }
    const int64_t m = (int64_t)rt * kRows + wave / WN * 64 + rf * 32 + i;
    const int64_t n = (int64_t)ct * 256 + (wave % WN * CF + j) * 32 + 8 * a + 4 * h;
    if (m < M && n < N)                          // N % 8 == 0: n < N implies n + 3 < N
        *(uint2*)(Y + m * N + n) = uint2{pack_bf16x2(sum[0], sum[1]), pack_bf16x2(sum[2], sum[3])};
}

}  // namespace

constexpr size_t kCounterBytes = 65536;
constexpr int kCus = kNumXcd * kCusPerXcd;
constexpr int kMaxSlices = 16;

// Which kernel, and how many slices of K, by the time that each would take: us on this card, fitted to 5200 launches of 33 .. 3000
// rows (K = 128 .. 28672, N = 64 .. 28672):
//   register kernel, 64 rows of 64 columns a workgroup: 4.3 + 1.25 x + steps * 1.44 (1 + 1.8 x rows / 64), where x is the
//     workgroups over 512 and a step a group of channels for each of four wavefronts; for slices 1.7 + .11 for each of them +
//     .17 per MB of partials; not less than the weights' bytes at 3.4 TB/s;
//   tiles of 64 wm rows: start + each * x + turns * turn for each round of one workgroup per CU (crowd more, where every CU
//     has one; x: workgroups over 256), for joining slices join + per MB of partials; not less than the weights' bytes at 4.6.
// What this takes is in the mean 1.3 % slower than the best of all.  92 x 2176 x 4952: 11.5 us by the register kernel, 17.9 by tiles;
// 435 x 800 x 136 6.6 and 10.0; 643 x 7312 x 1104 35.5 and 25.0; 64 x 8192 x 28672 69 and 53; 257 x 5120 x 13824: 37 us with 128 rows a tile,
// 68 with 64, 62 with 256; 2048 x 8192 x 8192: 120 us with 256 rows, 132 with 128; 512 x 8192 x 8192, 128 rows, 1, 2, 4
// slices: 60, 51, 61.
// Up to 32 rows the register kernel alone, cut where that leaves one workgroup per CU, with a group of channels or more
// for every wavefront (1 x 8192 x 1024, 1, 2, 4, 8 slices: 12.9, 9.9, 7.5, 6.6 us; 1 x 1024 x 8192, 1 and 2: 5.1, 6.0; 1 x
// 28672 x 8192, 1, 2, 4: 54.8, 41.8, 42.1).
Fp8GemmPlan plan_fp8_gemm(int64_t M, int64_t K, int64_t N) {
    Fp8GemmPlan p{};                             // wm = 0: the register kernel
    const int64_t chunks = fp8_kc(K), slots = fp8_nt(N) * ((M + 63) / 64);
    const int rf = M <= 16 ? 1 : M <= 32 ? 2 : 4, least = rf == 1 ? 8 : rf == 2 ? 4 : 2;   // groups of channels per slice
    const double bytes = (double)fp8_codes_bytes(K, N), row_part = M < 64 ? (double)M / 64 : 1.;
    double best = 1e300;
    for (int nz = 1; nz <= kMaxSlices; nz *= 2) {
        if (nz > 1 && (slots * nz > kCus || chunks < nz * least)) break;
        const double x = (double)(slots * nz) / 512, steps = (double)((chunks + 4 * nz - 1) / (4 * nz));
        const double total = 4.3 + 1.25 * x + steps * 1.44 * (1 + 1.8 * x * row_part) +
                             (nz == 1 ? 0 : 1.7 + .11 * nz + .17e-6 * (double)(slots * nz * 16384));
        const double us = rf < 4 ? -nz : std::max(2 + bytes / 3.4e6, total) + .02 * total;
        if (us >= best) continue;
        best = us;
        p.nz = nz;
    }
    p.col_tiles = fp8_nt(N);
    p.row_tiles = (M + 63) / 64;
    p.cstride = (int)std::max<int64_t>(1, std::min<int64_t>(32, kCounterBytes / 4 / slots));
    p.ws_bytes = p.nz > 1 ? kCounterBytes + (size_t)slots * p.nz * rf * 4096 : 0;
    if (rf < 4) return p;
    struct Tile {
        double start, each, turn, crowd, join, join_mb;
    };
    static const Tile tiles[3] = {{5.3, 3.4, .75, .04, 2., .31}, {5.9, 5.2, .66, .13, 2.1, .31}, {6.7, 8.9, 1.15, .24, 2.8, .23}};
    for (int k = 0; k < 3; ++k) {
        const Tile& t = tiles[k];
        const int wm = 1 << k;
        const int64_t rt = (M + 64 * wm - 1) / (64 * wm), ct = (N + 255) / 256;
        for (int nz = 1; nz <= kMaxSlices; ++nz) {
            const int64_t turns = (chunks + nz - 1) / nz, groups = rt * ct * nz, full = groups / kCus, rest = groups % kCus;
            if (nz > 1 && (turns < 2 || groups > kCus)) break;
            const double rounds = (double)full * (t.turn + t.crowd) + (rest ? t.turn + t.crowd * (double)rest / kCus : 0);
            const size_t part = (size_t)groups * 64 * wm * 256 * 4;
            const double total = t.start + t.each * (double)groups / kCus + (double)turns * rounds +
                                 (nz == 1 ? 0 : t.join + t.join_mb * 1e-6 * (double)part);
            const double us = std::max(2 + bytes / 4.6e6, total) + .02 * total;
            if (us >= best) continue;
            best = us;
            p.wm = wm;
            p.row_tiles = rt;
            p.col_tiles = ct;
            p.nz = nz;
            p.ws_bytes = nz > 1 ? kCounterBytes + part : 0;
        }
    }
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

template <int WM, int WN, int CF, int ST>
static hipError_t launch_tile(const uint8_t* xcodes, const float* xscales, int64_t M, const uint8_t* codes,
                              const float* scales, int64_t K, int64_t N, uint16_t* Y, void* ws, const Fp8GemmPlan& p,
                              hipStream_t st) {
    using S = Fp8Tile<WM, WN, CF, ST>;
    const int64_t total = p.row_tiles * p.col_tiles * p.nz, per_xcd = (total + kNumXcd - 1) / kNumXcd;
    const auto kernel = K % kFp8Group ? k_fp8_gemm_tile<WM, WN, CF, ST, true> : k_fp8_gemm_tile<WM, WN, CF, ST, false>;
    // the limit is a property of the function on the current device; setting it again is harmless
    const hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, S::kLds);
    if (e != hipSuccess) return e;
    float* const part = (float*)((char*)ws + kCounterBytes);
    kernel<<<(unsigned)(per_xcd * kNumXcd), 64 * S::kWaves, S::kLds, st>>>(
        xcodes, xscales, M, codes, scales, K, N, (int)fp8_kc(K), Y, part, (int)p.row_tiles, (int)p.col_tiles, p.nz,
        (int)total, (int)per_xcd);
    const hipError_t launched = hipGetLastError();
    if (launched != hipSuccess || p.nz == 1) return launched;
    k_fp8_join<WM, WN, CF><<<(unsigned)(p.row_tiles * p.col_tiles * (S::kWaves * 2 * CF)), 256, 0, st>>>(
        part, M, N, (int)p.row_tiles, (int)p.col_tiles, p.nz, Y);
    return hipGetLastError();
}

hipError_t launch_fp8_gemm(const uint8_t* xcodes, const float* xscales, int64_t M, const uint8_t* codes,
                           const float* scales, int64_t K, int64_t N, uint16_t* Y, void* ws, const Fp8GemmPlan& p,
                           hipStream_t st) {
    const auto run = [&](auto f) { return f(xcodes, xscales, M, codes, scales, K, N, Y, ws, p, st); };
    if (p.wm == 0) {
        if (M <= 16) return run(launch_rows<1, 8>);
        if (M <= 32) return run(launch_rows<2, 4>);
        return run(launch_rows<4, 4>);
    }
    if (p.wm == 4) return run(launch_tile<4, 2, 4, 2>);
    if (p.wm == 2) return run(launch_tile<2, 4, 2, 3>);
    return run(launch_tile<1, 4, 2, 3>);
}

}  // namespace awq
