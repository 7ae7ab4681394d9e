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
#include <type_traits>

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

__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* p, int64_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), (short)0, (int)(uint32_t)bytes, 0x00020000);
}
constexpr uint32_t kOutside = 0x80000000u;   // an offset past every resource (all are below 2 GiB)
constexpr int kCpolStream = 2;               // non-temporal: data read once
constexpr int kCpolAgent = 16;               // device-coherent level (the sc1 bit)
__device__ __forceinline__ void store4_agent(__amdgpu_buffer_rsrc_t r, uint32_t off, floatx4 v) {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), r, off, 0, kCpolAgent);
}
__device__ __forceinline__ floatx4 load4_agent(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    return __builtin_bit_cast(floatx4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, kCpolAgent));
}

// ---------------------------------------------------------------- up to 64 rows: weights streamed once
// Bound by the weights' bytes.  A workgroup owns 64 columns (one tile of packed weights, contiguous
// in memory) and a slice of K; its NW wavefronts take every NW-th 128-channel chunk, one in flight each,
// in registers: 4 KB of codes by non-temporal loads, the scale words, and the rows'
// elements and scale bytes (16 RF rows, repeated reads that the caches serve).  (Two chunks in flight were
// slower: 1 x 8192 x 10240 12.2 against 10.0 us, 20 x 9792 x 680 6.4 against 6.0.)  A load past the slice,
// past K or past the last row lies outside its buffer resource: it brings zeros and costs no traffic,
// so the loop needs no branch between a load and its use.  The wavefronts' sums meet in LDS in a fixed
// order; with several slices the last workgroup to arrive adds the float32 partials in slice order.
// 13 x 28672 x 8192: 23 us (5.4 TB/s; with both operands staged in LDS 109 us); 1 x 8192 x 10240: 10 us.
template <int BITS, int RF, int NW>
__global__ __launch_bounds__(64 * NW) void k_mx_gemm_rows(
    const uint8_t* __restrict__ xcodes, const uint8_t* __restrict__ xscales, int rows,
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t K, int64_t N, int64_t kb_all,
    uint16_t* __restrict__ Y, float* __restrict__ part, uint32_t* __restrict__ cnt, int cstride) {
    constexpr int H = BITS == 8 ? 2 : 1;         // 16-byte pieces of a lane's elements
    __shared__ floatx4 red[NW][RF][4][64];
    __shared__ uint32_t arrival;
    lds_poison_start(&red[0][0][0][0], NW * RF * 4 * 64);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int i = lane & 15, g = lane >> 4;
    const int64_t tile = blockIdx.x;
    const int z = blockIdx.y, nz = gridDim.y;
    const int chunks = (int)(kb_all / 4), per = (chunks + nz - 1) / nz;
    const int cb = min(z * per, chunks), ce = min(cb + per, chunks);
    const uint32_t xrow = (uint32_t)(BITS == 8 ? K : K / 2), srow = (uint32_t)(K / kMxBlock);
    const __amdgpu_buffer_rsrc_t wr = rsrc(codes + tile * kb_all * 1024, kb_all * 1024);
    const __amdgpu_buffer_rsrc_t fr = rsrc(scales + tile * kb_all * 64, kb_all * 64);
    const __amdgpu_buffer_rsrc_t xr = rsrc(xcodes, (int64_t)rows * xrow);
    const __amdgpu_buffer_rsrc_t sr = rsrc(xscales, (int64_t)rows * srow);

    struct Buf {
        u32x4 w[4], x[RF][H];
        uint32_t we, xe[RF];
    };
    auto issue = [&](int c, Buf& b) {
        const bool in = c < ce;
        const uint32_t wo = in ? (uint32_t)c * 4096 + g * 1024 + i * 16 : kOutside;
#pragma unroll
        for (int rf = 0; rf < RF; ++rf) {
            const uint32_t r = rf * 16 + i;
            const bool inx = in && (int)r < rows;
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const uint32_t k = (uint32_t)c * (BITS == 8 ? 128 : 64) + h * 64 + g * 16;   // byte of the row
                b.x[rf][h] = __builtin_bit_cast(
                    u32x4, __builtin_amdgcn_raw_buffer_load_b128(xr, inx && k < xrow ? r * xrow + k : kOutside, 0, 0));
            }
            const uint32_t kb = 4 * (uint32_t)c + g;
            b.xe[rf] = __builtin_amdgcn_raw_buffer_load_b8(sr, inx && kb < srow ? r * srow + kb : kOutside, 0, 0);
        }
        b.we = __builtin_amdgcn_raw_buffer_load_b32(fr, in ? (uint32_t)c * 256 + lane * 4 : kOutside, 0, kCpolStream);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            b.w[j] = __builtin_bit_cast(u32x4,
                                        __builtin_amdgcn_raw_buffer_load_b128(wr, wo, j * 256, kCpolStream));
    };
    floatx4 acc[RF][4];
#pragma unroll
    for (int rf = 0; rf < RF; ++rf)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[rf][j] = floatx4{0.f, 0.f, 0.f, 0.f};
    auto consume = [&](const Buf& b) {
        i32x8 x[RF];
#pragma unroll
        for (int rf = 0; rf < RF; ++rf) {
            const u32x4 a = b.x[rf][0], d = H == 2 ? b.x[rf][H - 1] : u32x4{0, 0, 0, 0};
            x[rf] = i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)d[0], (int)d[1], (int)d[2], (int)d[3]};
        }
#pragma unroll
        for (int rf = 0; rf < RF; ++rf) {
            acc[rf][0] = mx_mfma<BITS, 0>(b.w[0], x[rf], acc[rf][0], b.we, b.xe[rf]);
            acc[rf][1] = mx_mfma<BITS, 1>(b.w[1], x[rf], acc[rf][1], b.we, b.xe[rf]);
            acc[rf][2] = mx_mfma<BITS, 2>(b.w[2], x[rf], acc[rf][2], b.we, b.xe[rf]);
            acc[rf][3] = mx_mfma<BITS, 3>(b.w[3], x[rf], acc[rf][3], b.we, b.xe[rf]);
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
    const int64_t n = tile * kMxTile + 16 * frag + 4 * g;
    auto write_y = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int q = 0; q < RP; ++q) {
            const int r = (rf0 + q) * 16 + i;
            if (r < rows && n < N)               // N % 8 == 0: n < N implies n + 3 < N
                *(uint2*)(Y + (int64_t)r * N + n) =
                    uint2{pack_bf16x2(sum[q][0], sum[q][1]), pack_bf16x2(sum[q][2], sum[q][3])};
        }
    };
    if (nz == 1) {
        write_y();
        return;
    }
    constexpr uint32_t kPart = RF * 4 * 1024;
    const __amdgpu_buffer_rsrc_t pr = rsrc(part + tile * nz * (kPart / 4), (int64_t)nz * kPart);
    auto poff = [&](int s, int q) {
        return rf0 + q < RF ? (uint32_t)(s * kPart + ((rf0 + q) * 4 + frag) * 1024 + lane * 16) : kOutside;
    };
#pragma unroll
    for (int q = 0; q < RP; ++q) store4_agent(pr, poff(z, q), sum[q]);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // this wavefront's partial has landed
    __syncthreads();
    if (threadIdx.x == 0)
        arrival = __hip_atomic_fetch_add(cnt + tile * cstride, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
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
    if (threadIdx.x == 0) __hip_atomic_store(cnt + tile * cstride, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// ---------------------------------------------------------------- rows by the hundred: tiles in LDS
// 16 RF WM rows x 256 columns per workgroup, WM x WN wavefronts, each with RF x CF fragments of 16 x 16
// results in registers.  Per 128-channel chunk both operands are copied once per workgroup straight
// into LDS, ST chunks deep, in the order in which the matrix core's lanes read them back:
//   activations  1 KB units.  8 bits: 8 rows of 128 bytes; the two 16-byte pieces g and g + 4 that one lane
//                needs share the 32-byte slot g ^ 2 (row/8 % 2), the first of them at its half row/2 % 2.
//                4 bits: 16 rows of 64 bytes, piece g at 16-byte slot g ^ 2 (row/8 % 2).  So a transfer
//                reads whole lines, and the lanes that a 16-byte read serves together (0-3, 12-15, 20-27
//                and 4-11, 16-19, 28-31 of either half) hit different banks: conflicts per LDS instruction
//                2.36 -> 0.47 (8 bits), 1.33 -> 0.44 (4 bits), against swizzling by row/2 and row/4;
//   weights      the packed order: 1 KB per block of 64 columns, read 256 contiguous bytes at a time;
//   scales       of four chunks at a time, two such groups deep: weights 1 KB per column tile;
//                activations 16 bytes per row, from the 4-byte boundary at or before the group's first
//                byte (ALIGNED: at it), so that a row whose scales do not start on a boundary takes the
//                last bytes of a group's fourth chunk from the next group.  Chunk by chunk the gather of
//                4 bytes a row took a fifth of the transfers' time.
// Every transfer is issued from inline asm and waited for with counted vmcnt waits (transfers of a
// wavefront complete in order).  A turn multiplies one chunk in two halves of CF/2 column fragments,
// each product followed by its share of everything else, because a wavefront issues in order and a
// product keeps its matrix core busy for 32 cycles: during the first half the transfers of chunk
// c + ST - 1 are issued and the second half's weights are read from LDS; then a barrier says that chunk c
// is in every wavefront's registers and chunk c + 1 has landed; during the second half the next chunk's
// activations and first weights are read.  (Both operands of a whole chunk a turn ahead in registers: no
// faster, and too many of them for 256 rows.)  128 rows are four wavefronts, one per SIMD (eight with a
// quarter of the columns each were 2 % slower); 256 rows are eight of 64 rows (four with twice the rows each,
// which leave no register for the four-turn loop, took 643 instead of 640 us for 4096 x 8192 x 28672 with 8 bits,
// 438 instead of 424 for 4096 x 28672 x 8192 with 4).
//
// What bounds it.  256 rows: the clock, which falls from 2.4 to 1.6-1.95 GHz under this load, and, within the cycles left,
// how far LDS reads, transfers and barriers hide behind products.  4096 x 8192 x 28672, 8 bits: 640 to 700 us (2.8 to 3.0
// PFLOP/s), the matrix cores busy in 0.72 of the cycles; the products alone, on operands that stay in registers, 490 to 512.
// 4096 x 28672 x 8192, 4 bits: 424 to 459 us (4.2 to 4.5 PFLOP/s), busy in 0.57 (a product takes half the cycles,
// its LDS reads do not); products alone 302 to 316.  64 and 128 rows: one wavefront per SIMD issues everything, and
// products, transfers and LDS reads overlap in part (257 x 5120 x 13824, 4 bits, 23 us where a cache holds the
// weights, 25.8 where none does: products alone 10, transfers alone 10, LDS reads 4, prologue and epilogue 6).
typedef int i32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ i32x4 byte_rsrc(const void* base, uint32_t bytes) {
    const uint64_t a = (uint64_t)(uintptr_t)base;
    return i32x4{(int)__builtin_amdgcn_readfirstlane((uint32_t)a),
                 (int)(__builtin_amdgcn_readfirstlane((uint32_t)(a >> 32)) & 0xffff),
                 (int)__builtin_amdgcn_readfirstlane(bytes), 0x00020000};
}
// 16 bytes per lane from byte voff + soff of the resource to LDS address lds + off + 16 * lane (off a constant); a lane
// whose voff is at or past the resource's end brings zeros.  M0 holds the LDS address: every transfer writes it
// itself, with a wait state before its use, and leaves nothing there for another statement.
__device__ __forceinline__ void dma16(i32x4 rsrc, uint32_t voff, uint32_t soff, uint32_t lds, int off) {
#ifdef __HIP_DEVICE_COMPILE__                   // the host pass does not know the registers
    asm volatile(
        "s_add_u32 m0, %3, %4\n\t"
        "s_nop 0\n\t"
        "buffer_load_dwordx4 %0, %1, %2 offen lds"
        :
        : "v"(voff), "s"(rsrc), "s"(__builtin_amdgcn_readfirstlane(soff)), "s"(__builtin_amdgcn_readfirstlane(lds)), "i"(off)
        : "memory", "scc");
#endif
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

// acc += weights x activations in place, in accumulation registers; J: the byte of the weights' scale
// word.  (From the builtin the compiler makes products that write other registers than they read, and
// copies the accumulators around every turn.)  The compiler does not see a product in this: what the
// operands come from must be two instructions away, and results are read after mx_settle.
template <int BITS>
using XFrag = std::conditional_t<BITS == 8, i32x8, u32x4>;      // a lane's elements of a row fragment
template <int BITS, int J>
__device__ __forceinline__ void mx_mfma_acc(floatx4& acc, const u32x4& w, const XFrag<BITS>& x, uint32_t wscale,
                                            uint32_t xscale) {
#ifdef __HIP_DEVICE_COMPILE__                   // the host pass does not know these register classes
#define MX_MFMA(OPSEL)                                                                                            \
    if constexpr (BITS == 8)                                                                                      \
        asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 " OPSEL " cbsz:4"                  \
                     : "+a"(acc) : "v"(w), "v"(x), "v"(wscale), "v"(xscale));                                     \
    else                                                                                                          \
        asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 " OPSEL " cbsz:4 blgp:4"           \
                     : "+a"(acc) : "v"(w), "v"(x), "v"(wscale), "v"(xscale))
    if constexpr (J == 0) { MX_MFMA("op_sel_hi:[0,0,0]"); }
    if constexpr (J == 1) { MX_MFMA("op_sel:[1,0,0] op_sel_hi:[0,0,0]"); }
    if constexpr (J == 2) { MX_MFMA("op_sel_hi:[1,0,0]"); }
    if constexpr (J == 3) { MX_MFMA("op_sel:[1,0,0] op_sel_hi:[1,0,0]"); }
#undef MX_MFMA
#endif
}
__device__ __forceinline__ void mx_pin(floatx4& acc) {
#ifdef __HIP_DEVICE_COMPILE__
    asm volatile("" : "+a"(acc));
#endif
}
// No result of mx_mfma_acc is read before this (the compiler puts 12 and 8 wait states after its own products).
template <int BITS>
__device__ __forceinline__ void mx_settle() { asm volatile("s_nop %0" ::"n"(BITS == 8 ? 13 : 9)); }

// What the debug build fills LDS with before a transfer: scale bytes of 255 and e4m3 elements of 0xff are NaN, e2m1 elements
// of 0xf are -6, far from any data's sums.
__device__ __forceinline__ u32x4 mx_poison() { return u32x4{~0u, ~0u, ~0u, ~0u}; }

template <int BITS, int WM, int WN, int RF, int CF, int ST>
struct TileShape {
    static constexpr int kWaves = WM * WN, kRows = 16 * RF * WM, kCols = 16 * CF * WN;
    static_assert(kCols == 256 && kRows % 64 == 0 && CF % 4 == 0, "tile shape");
    static constexpr int kXk = kRows * BITS / 64;                 // 1 KB units of activations per chunk
    static constexpr int kWk = kCols / 64 * 4;                    // 1 KB units of weights per chunk
    static constexpr int kXu = kXk / kWaves, kWu = kWk / kWaves;  // per wavefront
    static constexpr int kData = kXu + kWu;
    static_assert(kXk % kWaves == 0 && kWk % kWaves == 0 && kWaves % 4 == 0, "even shares");
    static constexpr int kStage = (kXk + kWk) * 1024;
    static constexpr int kFs = 4096, kXs = kRows * 16;            // scales of a group: weights, activations
    static constexpr int kScales = ST * kStage, kLds = kScales + 2 * (kFs + kXs);
    static_assert(kLds <= 160 * 1024, "LDS of a CU");
    static_assert((ST == 3 || ST == 4) && (ST - 1) * kData + 4 < 64, "counted waits; a group is requested 3 turns early");
};

template <int BITS, int WM, int WN, int RF, int CF, int ST, bool ALIGNED>
__global__ __launch_bounds__(64 * WM * WN) void k_mx_gemm_tile(
    const uint8_t* __restrict__ xcodes, const uint8_t* __restrict__ xscales, int64_t M,
    const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t K, int64_t N, int64_t kb_all,
    uint16_t* __restrict__ Y, float* __restrict__ part, int row_tiles, int col_tiles,
    int nz, int total, int per_xcd) {
    using S = TileShape<BITS, WM, WN, RF, CF, ST>;
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
    const int chunks = (int)(kb_all / 4), per = ((chunks + nz - 1) / nz + 1) / 2 * 2;
    const int cb = min(z * per, chunks), ce = min(cb + per, chunks);
    const int64_t row0 = (int64_t)rt * S::kRows, t0 = (int64_t)ct * 4, nt = (N + 63) / 64;
    const int rows = (int)min<int64_t>(S::kRows, M - row0);       // past the last row and
    const int cts = (int)min<int64_t>(4, nt - t0);                // column tile: zeros
    const uint32_t xrow = (uint32_t)(BITS == 8 ? K : K / 2), srow = (uint32_t)(K / kMxBlock);
    const uint32_t wtile = (uint32_t)kb_all * 1024, ftile = (uint32_t)kb_all * 64;
    const int Kc = (int)K;

    const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) void*)lds;
    const i32x4 xr = byte_rsrc(xcodes + row0 * xrow, (uint32_t)rows * xrow);
    const i32x4 wr = byte_rsrc(codes + t0 * wtile, (uint32_t)cts * wtile);
    const i32x4 fr = byte_rsrc(scales + t0 * ftile, (uint32_t)cts * ftile);
    const uint8_t* s0 = xscales + row0 * srow;
    const uint32_t mis = (uint32_t)((uintptr_t)s0 & 3);           // read whole aligned words
    const i32x4 sr = byte_rsrc(s0 - mis, ((uint32_t)rows * srow + mis + 3) / 4 * 4);

    // A wavefront's units lie together in a stage: kXu of activations, kWu of weights.  This lane's piece of
    // its first activation unit (the next one is the next rows, with the same piece), and the piece's first
    // channel within a chunk.  Rows past `rows` and column tiles past `cts` lie outside the resources: zeros.
    constexpr int kUnitRows = BITS == 8 ? 8 : 16, kPieces = BITS == 8 ? 8 : 4;
    const int ur = wave * S::kXu * kUnitRows + lane / kPieces;
    const int us = lane % kPieces;               // 16-byte slot of the row
    const int ub = wave * S::kXu & 1;            // 8 bits: bit 3 of the first unit's rows
    auto piece = [&](int k) {                    // at slot us of unit k's rows
        if constexpr (BITS == 4) return us ^ (2 * (ur >> 3 & 1));
        else return ((us >> 1) ^ (2 * ((ub + k) & 1))) + 4 * ((us ^ (ur >> 1)) & 1);
    };
    int xk[2];                                   // first channel of the piece, units of either parity
#pragma unroll
    for (int k = 0; k < 2; ++k) xk[k] = piece(k) * (BITS == 8 ? 16 : 32);
    constexpr uint32_t kOwn = (S::kXu + S::kWu) * 1024;
    uint32_t xoff[S::kXu], woff[S::kWu];
#pragma unroll
    for (int k = 0; k < S::kXu; ++k) xoff[k] = (uint32_t)(ur + k * kUnitRows) * xrow + 16 * piece(k);
#pragma unroll
    for (int k = 0; k < S::kWu; ++k) woff[k] = (wave & 3) * 1024 + lane * 16 + (wave / 4 * S::kWu + k) * wtile;   // block wave % 4 of kWu column tiles
    // The scales of the slice's chunks 4q .. 4q+3: one column tile, and 64 rows (the same ones by several wavefronts
    // where there are fewer), per wavefront.  Past K: whatever lies there, or zeros; not used.
    constexpr int kParts = S::kRows / 64;
    const int part64 = wave % kParts;
    const uint32_t foff = (wave & 3) * ftile + lane * 16 + cb * 256;
    const uint32_t soff = (((uint32_t)(part64 * 64 + lane) * srow + mis) & ~3u) + cb * 4;
    auto issue_scales = [&](int q) __attribute__((always_inline)) {
        const uint32_t f = S::kScales + (q & 1) * S::kFs + (wave & 3) * 1024;
        const uint32_t x = S::kScales + 2 * S::kFs + (q & 1) * S::kXs + part64 * 1024;
        if constexpr (kLdsPoison) {              // debug build: where these will land, scales that make every value NaN
            lds[f / 16 + lane] = mx_poison();
            lds[x / 16 + lane] = mx_poison();
            lds_write_fence();
        }
        dma16(fr, foff + q * 1024, 0, base + f, 0);
        dma16(sr, soff + q * 16, 0, base + x, 0);
    };
    // transfer k of chunk c's batch; for a chunk past the slice the resources are empty, which brings zeros
    // (no traffic), so that the counted waits stay the same
    auto issue_op = [&](int c, int stage, int k) __attribute__((always_inline)) {
        const bool in = c < ce;
        const uint32_t st = stage * S::kStage + wave * kOwn;
        if constexpr (kLdsPoison) {              // debug build: e4m3 NaN, or e2m1's -6 in every element (it has no NaN)
            lds[st / 16 + k * 64 + lane] = mx_poison();
            lds_write_fence();
        }
        const i32x4 xc = {xr[0], xr[1], in ? xr[2] : 0, xr[3]}, wc = {wr[0], wr[1], in ? wr[2] : 0, wr[3]};
        const uint32_t past = ALIGNED || xk[k & 1] < Kc - c * kMxChunk ? 0 : kOutside;   // a piece past K
        const uint32_t sx = c * (BITS == 8 ? 128 : 64);
        const uint32_t to = base + (ST == 4 ? wave * kOwn : st);
        const int off = (ST == 4 ? stage * S::kStage : 0) + k * 1024;
        if (k < S::kXu) dma16(xc, xoff[k] | past, sx, to, off);
        else dma16(wc, woff[k - S::kXu], c * 4096, to, off);
    };

    // LDS byte offsets of this lane's operands within a stage; of its weight scales and of its scale byte of
    // each row fragment within a group
    constexpr int kFragUnits = BITS == 8 ? 2 : 1;                 // units of a row fragment
    auto unit_at = [](int e) { return (uint32_t)(e / S::kXu) * kOwn + (uint32_t)(e % S::kXu) * 1024; };
    static_assert(RF * kFragUnits % S::kXu == 0, "a wavefront's rows are whole wavefronts' units");
    const uint32_t xl = unit_at(wm * RF * kFragUnits) +
                        (BITS == 8 ? (i >> 3) * 1024 + (i & 7) * 128 + (g ^ (2 * (i >> 3))) * 32 + (i >> 1 & 1) * 16
                                   : i * 64 + (g ^ (2 * (i >> 3))) * 16);
    const uint32_t xh = xl ^ 16;                 // 8 bits: the second piece
    const uint32_t wl = g * kOwn + S::kXu * 1024 + i * 16, fl = g * 64 + i * 4;
    auto tile_at = [](int c) { return (uint32_t)(c / S::kWu) * 4 * kOwn + (uint32_t)(c % S::kWu) * 1024; };   // column tile
    uint32_t sl[ALIGNED ? 1 : RF];
#pragma unroll
    for (int rf = 0; rf < (ALIGNED ? 1 : RF); ++rf) {
        const int r = (wm * RF + rf) * 16 + i;
        sl[rf] = r * 16 + (ALIGNED ? 0 : (((uint32_t)r * srow + mis) & 3)) + g;
    }
    uint32_t slot = 0;                           // of the group that is read

    floatx4 acc[RF][CF];
#pragma unroll
    for (int rf = 0; rf < RF; ++rf)
#pragma unroll
        for (int j = 0; j < CF; ++j) acc[rf][j] = floatx4{0.f, 0.f, 0.f, 0.f};

    struct Acts {
        XFrag<BITS> x[RF];
        uint32_t e[RF];
    };
    struct Half {
        u32x4 w[CF / 2];
        uint32_t e;
    };
    constexpr int H = CF / 2, kFetchX = RF * 2, kFetchW = H + 1, kMul = RF * H;
    const uint8_t* const lb = (const uint8_t*)lds;
    // LDS reads of the slice's chunk u modulo 4, one at a time
    auto fetch_x_op = [&](int u, int stage, int k, Acts& a) __attribute__((always_inline)) {
        const int rf = k / 2;
        if (k % 2 == 1) {
            const uint32_t xs = S::kScales + 2 * S::kFs + 4 * u;
            if constexpr (ALIGNED) {
                a.e[rf] = lb[xs + slot * S::kXs + sl[0] + rf * 256];
            } else {                             // 16 bytes a row; past them the next group's first ones
                const bool over = u == 3 && (sl[rf] & 15) >= 4;
                a.e[rf] = lb[xs + (over ? (slot ^ 1) * S::kXs - 16 : slot * S::kXs) + sl[rf]];
            }
        } else if constexpr (BITS == 8) {
            const u32x4 p = *(const u32x4*)(lb + stage * S::kStage + xl + unit_at(2 * rf));
            const u32x4 q = *(const u32x4*)(lb + stage * S::kStage + xh + unit_at(2 * rf));
            a.x[rf] = i32x8{(int)p[0], (int)p[1], (int)p[2], (int)p[3], (int)q[0], (int)q[1], (int)q[2], (int)q[3]};
        } else {
            a.x[rf] = *(const u32x4*)(lb + stage * S::kStage + xl + unit_at(rf));
        }
    };
    auto fetch_w_op = [&](int u, int stage, int half, int k, Half& h) __attribute__((always_inline)) {
        const int j = wn * CF + half * H + (k > 0 ? k - 1 : 0);   // fragment among the tile's 16
        if (k == 0) h.e = *(const uint32_t*)(lb + S::kScales + slot * S::kFs + u * 256 + fl + j / 4 * 1024);
        else h.w[k - 1] = *(const u32x4*)(lb + stage * S::kStage + wl + tile_at(j / 4) + j % 4 * 256);
    };
    auto product = [&](const Acts& a, const uint32_t (&e)[RF], const Half& h, int half, int n) __attribute__((always_inline)) {
        const int q = n / RF, rf = n % RF, j = half * H + q;
        if (j % 4 == 0) mx_mfma_acc<BITS, 0>(acc[rf][j], h.w[q], a.x[rf], h.e, e[rf]);
        if (j % 4 == 1) mx_mfma_acc<BITS, 1>(acc[rf][j], h.w[q], a.x[rf], h.e, e[rf]);
        if (j % 4 == 2) mx_mfma_acc<BITS, 2>(acc[rf][j], h.w[q], a.x[rf], h.e, e[rf]);
        if (j % 4 == 3) mx_mfma_acc<BITS, 3>(acc[rf][j], h.w[q], a.x[rf], h.e, e[rf]);
    };

    issue_scales(0);
#pragma unroll
    for (int s = 0; s < ST - 1; ++s)
#pragma unroll
        for (int k = 0; k < S::kData; ++k) issue_op(cb + s, s, k);
    Acts xa, xb;
    Half lo, hi;
    asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"((ST - 2) * S::kData) : "memory");
#pragma unroll
    for (int k = 0; k < kFetchX; ++k) fetch_x_op(0, 0, k, xa);
#pragma unroll
    for (int k = 0; k < kFetchW; ++k) fetch_w_op(0, 0, 0, k, lo);
    int stage3 = 0;                              // of chunk c, with three stages
    // Chunk c, the slice's chunk u modulo 4; EDGE: it may reach past K.
    auto turn = [&](auto EDGE, int u, int c, const Acts& now, Acts& next) __attribute__((always_inline)) {
        constexpr bool edge = decltype(EDGE)::value;
        const int v = (u + 1) % 4, stage = ST == 4 ? u : stage3;
        const int behind = ST == 4 ? (u + 3) % 4 : stage == 0 ? ST - 1 : stage - 1;
        const int ahead = ST == 4 ? v : stage == ST - 1 ? 0 : stage + 1;
        // The next group takes the place of the one before, whose last bytes were in registers before the last
        // barrier.  Before the batch's kData transfers, so that the counted waits cover it.
        if (u == 0) issue_scales((c - cb) / 4 + 1);
        uint32_t e[RF];
        if constexpr (edge) {                    // past K: elements are zero, the scales 1 (what was read may say NaN)
            const bool inside = 4 * c + g < (int)srow;
#pragma unroll
            for (int rf = 0; rf < RF; ++rf) {
                e[rf] = inside ? now.e[rf] : 127u;
                asm volatile("" : "+v"(e[rf]));  // in registers here, not next to their use
            }
            lo.e = c < chunks ? lo.e : 0x7f7f7f7fu;
            asm volatile("" : "+v"(lo.e));
        } else {
#pragma unroll
            for (int rf = 0; rf < RF; ++rf) e[rf] = now.e[rf];
        }
        asm volatile("s_nop 1");
        constexpr int ops1 = kFetchW + S::kData;
#pragma unroll
        for (int n = 0; n < kMul; ++n) {
            product(now, e, lo, 0, n);
#pragma unroll
            for (int k = 0; k < ops1; ++k) {
                if (k * kMul / ops1 != n) continue;
                if (k < kFetchW) fetch_w_op(u, stage, 1, k, hi);
                else issue_op(c + ST - 1, behind, k - kFetchW);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((ST - 2) * S::kData) : "memory");
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (edge) {
            hi.e = c < chunks ? hi.e : 0x7f7f7f7fu;
            asm volatile("" : "+v"(hi.e));
        }
        asm volatile("s_nop 1");
        if (u == 3) slot ^= 1;
        constexpr int ops2 = kFetchW + kFetchX;
#pragma unroll
        for (int n = 0; n < kMul; ++n) {
            product(now, e, hi, 1, n);
#pragma unroll
            for (int k = 0; k < ops2; ++k) {
                if (k * kMul / ops2 != n) continue;
                if (k < kFetchW) fetch_w_op(v, ahead, 0, k, lo);
                else fetch_x_op(v, ahead, k - kFetchW, next);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        stage3 = ahead;
    };
    // On both sides of every place where the compiler may copy or read accumulators, the ways into and out of
    // a loop or branch: no product is in flight before, and none starts right after.  (A product keeps its
    // matrix core for most of this wait anyway.)
    auto join = [&]() __attribute__((always_inline)) {
        mx_settle<BITS>();
#pragma unroll
        for (int rf = 0; rf < RF; ++rf)
#pragma unroll
            for (int j = 0; j < CF; ++j) mx_pin(acc[rf][j]);
    };
    constexpr std::false_type kWhole{};
    constexpr std::true_type kEdge{};
    int c = cb;
    // Four turns at a time, so that the LDS addresses are constants (60 instructions a turn beside the
    // products instead of 168: 257 x 5120 x 13824, 4 bits, 28.5 -> 23.0 us); then the last one to four chunks.
    for (; c + 4 < ce; c += 4) {
        turn(kWhole, 0, c, xa, xb);
        turn(kWhole, 1, c + 1, xb, xa);
        turn(kWhole, 2, c + 2, xa, xb);
        turn(kWhole, 3, c + 3, xb, xa);
        join();
    }
    join();
    turn(kEdge, 0, c, xa, xb);
    turn(kEdge, 1, c + 1, xb, xa);
    join();
    if (c + 2 < ce) {
        join();
        turn(kEdge, 2, c + 2, xa, xb);
        turn(kEdge, 3, c + 3, xb, xa);
        join();
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    auto settled = [&](int rf) __attribute__((always_inline)) {   // one row fragment's results at a time
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < CF; ++j) mx_pin(acc[rf][j]);
    };

    // Results leave through a buffer resource, where a row past M or a column past N lies outside: a
    // branch around the stores would let the compiler move products into it, and those need every
    // lane's operands.
    const __amdgpu_buffer_rsrc_t yr = rsrc(Y + row0 * N, (int64_t)rows * N * 2);
    auto write_rows = [&](int rf, const floatx4 (&v)[CF]) __attribute__((always_inline)) {
        const int r = (wm * RF + rf) * 16 + i;
#pragma unroll
        for (int j = 0; j < CF; j += 4) {
            const floatx4 q[4] = {v[j], v[j + 1], v[j + 2], v[j + 3]};
            u32x4 out[2];
            mx_rows16(q, out);
            const int64_t n = t0 * kMxTile + (wn * CF + j) * 16 + 16 * g;
#pragma unroll
            for (int h = 0; h < 2; ++h)                              // N % 8 == 0
                __builtin_amdgcn_raw_buffer_store_b128(
                    out[h], yr, r < rows && n + 8 * h < N ? (uint32_t)(r * N + n + 8 * h) * 2 : kOutside, 0, 0);
        }
    };
    if (nz == 1) {
#pragma unroll
        for (int rf = 0; rf < RF; ++rf) {
            settled(rf);
            write_rows(rf, acc[rf]);
        }
        return;
    }
    // Split over K: float32 partials in fragment order, one per (tile, K slice), that k_mx_join adds.
    constexpr uint32_t kPart = S::kRows * S::kCols * 4;
    const __amdgpu_buffer_rsrc_t pr = rsrc(part + (int64_t)tile * nz * (kPart / 4), (int64_t)nz * kPart);
#pragma unroll
    for (int rf = 0; rf < RF; ++rf) {
        settled(rf);
#pragma unroll
        for (int j = 0; j < CF; ++j)
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, acc[rf][j]), pr,
                                                   z * kPart + ((wave * RF + rf) * CF + j) * 1024 + lane * 16, 0, 0);
    }
}

// Adds the slices of the tiles above: a wavefront takes one fragment (stored by wavefront, row fragment, column
// fragment) of every slice, in slice order, eight loads in flight.  Bound by the partials' bytes, which the
// caches hold.  A launch of its own, because the last workgroup of a tile alone reads a slice of it in
// 1.15 WM us: 128 x 4096 x 4096, 3 slices of 64 x 256, 15.5 -> 14.4 us; 99 x 22432 x 832, 8 slices, 23.4 -> 16.9.
template <int WM, int WN, int RF, int CF>
__global__ __launch_bounds__(256) void k_mx_join(const float* __restrict__ part, int64_t M, int64_t N, int row_tiles,
                                                 int col_tiles, int nz, uint16_t* __restrict__ Y) {
    constexpr int kFrags = WM * WN * RF * CF, kRows = 16 * RF * WM;
    constexpr uint32_t kPart = kFrags * 1024;
    const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
    const int f = (blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) % kFrags;
    const int tile = blockIdx.x * 4 / kFrags;
    const int panel = tile / (8 * col_tiles), in = tile % (8 * col_tiles), prow = min(8, row_tiles - 8 * panel);
    const int rt = 8 * panel + in % prow, ct = in / prow;
    const int wave = f / (RF * CF), rf = f / CF % RF, j = f % CF;
    const float* p = part + (int64_t)tile * nz * (kPart / 4) + f * 256 + lane * 4;
    floatx4 sum = floatx4{0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < nz; s += 8) {
        floatx4 v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = *(const floatx4*)(p + (int64_t)min(s + u, nz - 1) * (kPart / 4));
#pragma unroll
        for (int u = 0; u < 8; ++u)
            if (s + u < nz) sum += v[u];
    }
    const int64_t m = (int64_t)rt * kRows + (wave / WN * RF + rf) * 16 + i;
    const int64_t n = (int64_t)ct * 256 + (wave % WN * CF + j) * 16 + 4 * g;
    if (m < M && n < N)                          // N % 8 == 0: n < N implies n + 3 < N
        *(uint2*)(Y + m * N + n) = uint2{pack_bf16x2(sum[0], sum[1]), pack_bf16x2(sum[2], sum[3])};
}

}  // namespace

constexpr size_t kCounterBytes = 65536;
constexpr int kCus = kNumXcd * kCusPerXcd;
constexpr int kMaxSlices = 16;

// Which kernel, and how many slices of K, by the time that each would take: us on this card, fitted to
// measured launches (K = 4096 .. 28672, N = 1024 .. 28672):
//   register kernel: 2.3 + .045 + .0037 M for each 128-channel chunk that a CU takes (64 columns), the
//     weights at 8 TB/s (the caches hold a part of them) and the rows, read by every column tile, at 14,
//     and for joining slices .9 + .035 M + nz (.08 + .003 M); no more workgroups than CUs once K is cut.
//     E.g. 1 x 8192 x 1024, 1, 2, 4, 8 slices: 5.6, 5.5, 4.8, 4.4 us; 1 x 8192 x 10240, 1 and 2: 10.1, 13.4;
//     50 x 9792 x 680, 1, 4, 8, 16: 20.1, 10.4, 8.9, 10.6 (tiles 9.5);
//   tiles of 64 wm rows: 1.5 + rounds of one workgroup per CU * (start_us + turns * turn_us), and for joining
//     slices 2 + .35 per MB of partials; the rounds not below the time in which these kernels stream the
//     weights (4 TB/s).  E.g. 257 x 5120 x 13824, 4 bits: 23 us with 128 rows a tile, 30 with 64, 41 with 256;
//     2048 x 8192 x 8192, 8 bits, 101 us with 256 rows, 116 with 128;
//     128 x 4096 x 4096, 8 bits, 64-row tiles: 14.7, 14.0, 13.4, 13.9 us with 1, 2, 3, 4 slices.
MxGemmPlan plan_mx_gemm(int64_t M, int64_t K, int64_t N, int bits) {
    MxGemmPlan p{};                              // wm = 0: the register kernel
    const int64_t chunks = mx_kb(K) / 4;
    double best = 1e30;
    if (M <= 64) {
        p.col_tiles = mx_nt(N);
        p.row_tiles = (M + 15) / 16;             // fragments of the one workgroup row
        p.cstride = (int)std::max<int64_t>(1, std::min<int64_t>(32, kCounterBytes / 4 / p.col_tiles));
        const int64_t most = p.col_tiles > (int64_t)(kCounterBytes / 4) ? 1 : std::min<int64_t>(kMaxSlices, chunks);
        const double stream = (double)mx_codes_bytes(K, N) / 8e6 + (double)(p.col_tiles * M) * (double)(K * bits / 8) / 14e6;
        for (int nz = 1; nz <= most && (nz == 1 || p.col_tiles * nz <= kCus); ++nz) {
            const double per_cu = std::max((double)((chunks + nz - 1) / nz), (double)(p.col_tiles * chunks) / kCus);
            const double us = 2.3 + per_cu * (.045 + .0037 * (double)M) + stream +
                              (nz == 1 ? 0 : .9 + .035 * (double)M + nz * (.08 + .003 * (double)M));
            if (us >= best) continue;
            best = us;
            p.nz = nz;
            p.ws_bytes = nz > 1 ? kCounterBytes + (size_t)p.col_tiles * nz * p.row_tiles * 4096 : 0;
        }
        if (M <= 16) return p;
    }
    static const double start_us[3] = {4, 6, 8.5}, turn_us[2][3] = {{.31, .45, .72}, {.39, .63, 1.10}};   // 4, 8 bits
    const double stream = 2 + (double)mx_codes_bytes(K, N) / 4e6;
    for (int k = 0; k < 3; ++k) {
        const int wm = 1 << k;
        const int64_t rt = (M + 64 * wm - 1) / (64 * wm), ct = (N + 255) / 256, tiles = rt * ct;
        for (int nz = 1; nz <= kMaxSlices; ++nz) {
            const int64_t turns = ((chunks + nz - 1) / nz + 1) / 2 * 2, groups = tiles * nz;
            if (nz > 1 && (turns < 4 || groups > kCus)) break;
            const double rounds = (double)((groups + kCus - 1) / kCus);
            const double us = std::max(stream, 1.5 + rounds * (start_us[k] + turns * turn_us[bits == 8][k])) +
                              (nz == 1 ? 0 : 2 + .35e-6 * (double)(groups * 64 * wm * 256 * 4));
            if (us >= best) continue;
            best = us;
            p.wm = wm;
            p.row_tiles = rt;
            p.col_tiles = ct;
            p.nz = nz;
            p.ws_bytes = nz > 1 ? kCounterBytes + (size_t)groups * 64 * wm * 256 * 4 : 0;
        }
    }
    return p;
}

template <int BITS, int RF, int NW>
static hipError_t launch_rows(const uint8_t* xcodes, const uint8_t* xscales, int64_t M, const uint8_t* codes,
                              const uint8_t* scales, int64_t K, int64_t N, uint16_t* Y, void* ws, const MxGemmPlan& p,
                              hipStream_t st) {
    k_mx_gemm_rows<BITS, RF, NW><<<dim3((unsigned)p.col_tiles, (unsigned)p.nz), 64 * NW, 0, st>>>(
        xcodes, xscales, (int)M, codes, scales, K, N, mx_kb(K), Y, (float*)((char*)ws + kCounterBytes), (uint32_t*)ws,
        p.cstride);
    return hipGetLastError();
}

template <int BITS, int WM, int WN, int RF, int CF, int ST>
static hipError_t launch_tile(const uint8_t* xcodes, const uint8_t* xscales, int64_t M, const uint8_t* codes,
                              const uint8_t* scales, int64_t K, int64_t N, uint16_t* Y, void* ws, const MxGemmPlan& p,
                              hipStream_t st) {
    using S = TileShape<BITS, WM, WN, RF, CF, ST>;
    const int64_t total = p.row_tiles * p.col_tiles * p.nz, per_xcd = (total + kNumXcd - 1) / kNumXcd;
    const bool aligned = K % kMxChunk == 0 && (uintptr_t)xscales % 4 == 0;
    const auto kernel = aligned ? k_mx_gemm_tile<BITS, WM, WN, RF, CF, ST, true>
                                : k_mx_gemm_tile<BITS, WM, WN, RF, CF, ST, false>;
    // the limit is a property of the function on the current device; setting it again is harmless
    const hipError_t e = hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, S::kLds);
    if (e != hipSuccess) return e;
    kernel<<<(unsigned)(per_xcd * kNumXcd), 64 * S::kWaves, S::kLds, st>>>(
        xcodes, xscales, M, codes, scales, K, N, mx_kb(K), Y, (float*)((char*)ws + kCounterBytes),
        (int)p.row_tiles, (int)p.col_tiles, p.nz, (int)total, (int)per_xcd);
    const hipError_t launched = hipGetLastError();
    if (launched != hipSuccess || p.nz == 1) return launched;
    k_mx_join<WM, WN, RF, CF><<<(unsigned)(p.row_tiles * p.col_tiles * (S::kWaves * RF * CF / 4)), 256, 0, st>>>(
        (const float*)((char*)ws + kCounterBytes), M, N, (int)p.row_tiles, (int)p.col_tiles, p.nz, Y);
    return hipGetLastError();
}

hipError_t launch_mx_gemm(const uint8_t* xcodes, const uint8_t* xscales, int bits, int64_t M, const uint8_t* codes,
                          const uint8_t* scales, int64_t K, int64_t N, uint16_t* Y, void* ws, const MxGemmPlan& p,
                          hipStream_t st) {
    const auto run = [&](auto f) { return f(xcodes, xscales, M, codes, scales, K, N, Y, ws, p, st); };
    if (p.wm == 0) {
        switch (p.row_tiles) {
            case 1: return run(bits == 8 ? launch_rows<8, 1, 8> : launch_rows<4, 1, 8>);
            case 2: return run(bits == 8 ? launch_rows<8, 2, 4> : launch_rows<4, 2, 4>);
            case 3: return run(bits == 8 ? launch_rows<8, 3, 4> : launch_rows<4, 3, 4>);
            default: return run(bits == 8 ? launch_rows<8, 4, 4> : launch_rows<4, 4, 4>);
        }
    }
    if (p.wm == 4) return run(bits == 8 ? launch_tile<8, 4, 2, 4, 8, 3> : launch_tile<4, 4, 2, 4, 8, 4>);
    if (p.wm == 2) return run(bits == 8 ? launch_tile<8, 2, 2, 4, 8, 4> : launch_tile<4, 2, 2, 4, 8, 4>);
    return run(bits == 8 ? launch_tile<8, 1, 4, 4, 4, 4> : launch_tile<4, 1, 4, 4, 4, 4>);
}

}  // namespace awq
