// Attention over the 8-bit cache: out = sum_t p_t v_t / sum_t p_t, p_t = exp(scale q . k_t), in one pass over the tokens
// with the running maximum and sum.
//
// The rows of a sequence for one head of the cache are its new tokens times the G heads of q that read it:
// row r is token r / G, head r % G.  A key or value that one workgroup has loaded serves all of them.
#include <algorithm>

#include "awq_buffer.h"
#include "awq_cache.h"

namespace awq {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
constexpr int kTile = 64;                        // tokens that a wavefront takes at a time
constexpr int kSliceTokens = 256;                // least tokens of a slice
constexpr size_t kCounterBytes = 65536;          // left alone: the products' arrival counters, in a workspace that they share

// Eight e4m3 codes (two words) times 2^(E - 127), the scale's exponent field, in bf16: exact, but for E < 3, whose smallest
// numbers lie below bf16's least step, 2^-133.
__device__ __forceinline__ bf16x8 widen_codes(uint32_t a, uint32_t b, float scale) {
    const bf16x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, false);
    const bf16x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, scale, true);
    const bf16x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, false);
    const bf16x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, scale, true);
    return bf16x8{v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
}
// The maximum and the sum over the four lanes of equal lane % 16.
__device__ __forceinline__ float max_g(float v) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float sum_g(float v) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(a[0]) + __uint_as_float(a[1]);
    const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

struct Args {
    const uint16_t* q;
    uint16_t* out;
    float* part;
    int M, Hq, G, causal, tiles, split;
    float scale;                 // times log2 e
};

// What a tile of R rows is: its sequence, its rows, the tokens that they see, and the slices of tiles of TOKENS tokens
// that these make.
template <int R, int TOKENS>
struct TileRows {
    int b, rt, rows, row0, start, length, G, cap, most, tiles, used;
    __device__ __forceinline__ TileRows(const Args& a, const Sequences& s, const Cache& c, int b_, int rt_) : b(b_), rt(rt_) {
        const NewTokens t = new_tokens(s, b, a.M);
        rows = min(t.count, s.max_q) * a.G;
        row0 = t.row0, start = t.start, length = t.length, G = a.G;
        cap = s.width << c.logT;                 // what the table covers
        most = reach(R * rt + R - 1, a);
        tiles = (most + TOKENS - 1) / TOKENS;
        used = max(min(a.split, (most + kSliceTokens - 1) / kSliceTokens), 1);
    }
    // tokens that a row sees (of one past the last: what the last sees; never fewer than a row before it; none from a
    // position below zero), and where its numbers are
    __device__ __forceinline__ int reach(int row, const Args& a) const {
        const int upto = start + max(min(row, rows - 1), 0) / G + 1;
        return upto <= 0 ? 0 : min(a.causal ? upto : length, cap);
    }
    __device__ __forceinline__ int64_t at(int row, int head, const Args& a, int D) const {
        const int r = max(min(row, rows - 1), 0);
        return ((int64_t)(row0 + r / G) * a.Hq + head * G + r % G) * D;
    }
};
// ---------------------------------------------------------------- few rows: the cache streamed once
// Bound by the cache's bytes.  A workgroup takes 16 rows and a slice of the tokens; its four wavefronts take every
// fourth tile of 64 tokens of it.  A lane (i, g) = (lane % 16, lane / 16) works for tokens 16g .. 16g + 15 of the tile in
// both products, so that what belongs to those tokens (their block, its scales, the mask) is the lane's own:
//   first product   S^T = K Q^T, four 16 x 16 results: row 4g + r of result t is token 16g + 4t + r, so lane
//                   (i, g) gives K's row of token 16 (i / 4) + 4t + i % 4, and takes 16 results of query row i;
//   second product  O^T = V^T P^T: lane (i, g) gives the 16 bytes of number i of V's 16 tokens, and its own
//                   results, in the order in which they are.
// K and V become bf16 in registers (exact); p goes into the second product as two bf16 numbers, whose cost the loads
// hide.  The running maximum and sum are per row; every wavefront has its own,
// joined in LDS at the end, and those of several slices by k_attention_join_rows.
// 64 sequences of up to 8192 tokens, 64 heads on 8, D = 128 (554 MB): 114-134 us by the boxes' memory (4.1-4.8 TB/s, a copy 4.75); one
// of 4097 tokens 7.8 us and 2.9 for the join: lengths, blocks, codes, the join in LDS and the partials are trips to memory
// one after the other, on 96 workgroups.
template <int D>
__global__ __launch_bounds__(256) void k_attention_rows(Args a, Sequences s, Cache c) {
    constexpr int ND = D / 16, NH = D / 64;
    __shared__ floatx4 red[4][ND][64];
    __shared__ float stat[4][2][16];
    lds_poison_start(&red[0][0][0], 4 * ND * 64);
    lds_poison_start(&stat[0][0][0], 128);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int i = lane & 15, g = lane >> 4;
    const int h = blockIdx.x % c.Hk, rest = blockIdx.x / c.Hk;
    const int z = rest % a.split, rt = rest / a.split % a.tiles, b = rest / a.split / a.tiles;
    const TileRows<16, kTile> t(a, s, c, b, rt);
    if (16 * rt >= t.rows || z >= t.used) return;                // the whole workgroup
    const int row = 16 * rt + i, seen = t.reach(row, a), most = t.most, used = t.used;
    const int64_t qat = t.at(row, h, a, D);
    const int per = (t.tiles + used - 1) / used, tb = min(z * per, t.tiles), te = min(tb + per, t.tiles);

    bf16x8 q[NH][2];
#pragma unroll
    for (int n = 0; n < NH; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) q[n][e] = __builtin_bit_cast(bf16x8, *(const u32x4*)(a.q + qat + 64 * n + 16 * g + 8 * e));

    floatx4 o[ND];
#pragma unroll
    for (int n = 0; n < ND; ++n) o[n] = floatx4{0.f, 0.f, 0.f, 0.f};
    float m = -INFINITY, sum = 0.f;

    const int32_t* const table = s.table + (int64_t)b * s.width;
    // the block of tokens first .. first + 15 (a multiple of 16), or -1
    auto block_of = [&](int first) __attribute__((always_inline)) {
        const int j = first >> c.logT;
        const int v = first < most && j < s.width ? table[j] : -1;
        return v >= 0 && v < c.blocks ? v : -1;
    };
    u32x4 k[4][NH], v[ND];
    uint32_t e;
    const int kg = i >> 2;                       // the 16 tokens whose K this lane gives; V's are 16 g ..
    auto load_k = [&](int first, int bk) __attribute__((always_inline)) {
        const uint8_t* const p = c.k + (((int64_t)max(bk, 0) * c.Hk + h) * c.T + ((first + 16 * kg) & (c.T - 1)) + (i & 3)) * D + 16 * g;
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int n = 0; n < NH; ++n) k[u][n] = *(const u32x4*)(p + 4 * u * D + 64 * n);
    };
    auto load_v = [&](int first, int bv) __attribute__((always_inline)) {
        const uint8_t* const p = c.v + (((int64_t)max(bv, 0) * c.Hk + h) * c.T + ((first + 16 * g) & (c.T - 1))) * D + 16 * i;
#pragma unroll
        for (int n = 0; n < ND; ++n) v[n] = *(const u32x4*)(p + 256 * n);
    };
    auto load_scales = [&](int bv) __attribute__((always_inline)) {
        return (uint32_t)*(const uint16_t*)(c.scales + ((int64_t)max(bv, 0) * c.Hk + h) * 2);
    };
    // Blocks are looked up two tiles ahead; a tile's K is requested where the one before has left its registers, its V
    // likewise, so that one tile is on its way all the time.
    int first = (tb + wave) * kTile;
    const int end = te * kTile;
    int bk = block_of(first + 16 * kg), bv = block_of(first + 16 * g);
    int bk1 = block_of(first + 4 * kTile + 16 * kg), bv1 = block_of(first + 4 * kTile + 16 * g);
    if (first < end) {
        e = load_scales(bv);
        load_k(first, bk);
        load_v(first, bv);
    }
    for (; first < end; first += 4 * kTile) {
        const bool more = first + 4 * kTile < end;
        const int bk2 = block_of(first + 8 * kTile + 16 * kg), bv2 = block_of(first + 8 * kTile + 16 * g);
        const bool poisoned = (e & 255) == 255 || e >> 8 == 255;
        // a marked block makes what is seen of it NaN; V's own scale then is any finite one.  (K's times a.scale may pass
        // float32's range where no score does: the two are applied one after the other.)
        const float f = poisoned ? NAN : __uint_as_float((e & 255) == 0 ? 0x00400000u : (e & 255) << 23);
        const float fv = __uint_as_float(poisoned ? 127u << 23 : (e >> 8) << 23);

        floatx4 p[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            p[u] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int n = 0; n < NH; ++n) {
                p[u] = mfma16x16x32(widen_codes(k[u][n][0], k[u][n][1], 1.f), q[n][0], p[u]);
                p[u] = mfma16x16x32(widen_codes(k[u][n][2], k[u][n][3], 1.f), q[n][1], p[u]);
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        if (more) {
            e = load_scales(bv1);
            load_k(first + 4 * kTile, bk1);
        }
        // token 16g + 4u + r of the tile is seen when it lies below `limit`
        const int limit = bv < 0 ? 0 : seen - first - 16 * g;
        float top = -INFINITY;
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                p[u][r] = 4 * u + r < limit ? p[u][r] * f * a.scale : -INFINITY;
                top = fmaxf(top, p[u][r]);
            }
        const float next = fmaxf(m, max_g(top));
        const float base = next == -INFINITY ? 0.f : next;       // nothing seen yet: exponents of -inf, not of NaN
        const float keep = __builtin_amdgcn_exp2f(m - base);
        m = next;
        sum *= keep;
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                p[u][r] = __builtin_amdgcn_exp2f(p[u][r] - base);
                sum += p[u][r];
            }
        bf16x8 w[2], rest[2];                    // p and what its rounding to bf16 leaves: 16 bits of it
#pragma unroll
        for (int y = 0; y < 2; ++y) {
            u32x4 hi, lo;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float v0 = p[2 * y + e / 2][2 * (e & 1)], v1 = p[2 * y + e / 2][2 * (e & 1) + 1];
                hi[e] = pack_bf16x2(v0, v1);
                lo[e] = pack_bf16x2(v0 - bf16_lo(hi[e]), v1 - bf16_hi(hi[e]));
            }
            w[y] = __builtin_bit_cast(bf16x8, hi);
            rest[y] = __builtin_bit_cast(bf16x8, lo);
        }
        // what lies behind the sequence's last token may be anything, NaN among it: zeros
        const int live = bv < 0 ? 0 : t.length - first - 16 * g;
        const uint64_t lo = live >= 8 ? ~0ull : (1ull << 8 * max(live, 0)) - 1;
        const uint64_t hi = live >= 16 ? ~0ull : live <= 8 ? 0ull : (1ull << 8 * (live - 8)) - 1;
        const u32x4 mask = {(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
#pragma unroll
        for (int n = 0; n < ND; ++n) {
#pragma unroll
            for (int r = 0; r < 4; ++r) o[n][r] *= keep;
            const u32x4 x = v[n] & mask;
            const bf16x8 x0 = widen_codes(x[0], x[1], fv), x1 = widen_codes(x[2], x[3], fv);
            o[n] = mfma16x16x32(x0, rest[0], o[n]);
            o[n] = mfma16x16x32(x1, rest[1], o[n]);
            o[n] = mfma16x16x32(x0, w[0], o[n]);
            o[n] = mfma16x16x32(x1, w[1], o[n]);
        }
        __builtin_amdgcn_sched_barrier(0);
        if (more) load_v(first + 4 * kTile, bv1);
        bv = bv1;
        bk1 = bk2;
        bv1 = bv2;
    }
    // the wavefronts' parts: lane (i, g) holds numbers 16n + 4g .. + 3 of row i
    sum = sum_g(sum);
#pragma unroll
    for (int n = 0; n < ND; ++n) {
        asm volatile("" : "+v"(o[n]));
        red[wave][n][lane] = o[n];
    }
    if (g == 0) stat[wave][0][i] = m, stat[wave][1][i] = sum;
    __syncthreads();
    constexpr int NP = ND / 4;                   // wavefront w joins numbers 16 n of n = NP w ..
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < 4; ++w) top = fmaxf(top, stat[w][0][i]);
    const float base = top == -INFINITY ? 0.f : top;
    float total = 0.f;
    floatx4 x[NP];
#pragma unroll
    for (int n = 0; n < NP; ++n) x[n] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const float f = __builtin_amdgcn_exp2f(stat[w][0][i] - base);
        total += f * stat[w][1][i];
#pragma unroll
        for (int n = 0; n < NP; ++n) x[n] += f * red[w][wave * NP + n][lane];
    }
    if (row >= t.rows) return;
    if (used > 1) {                              // several slices: k_attention_join_rows adds them
        float* const to = a.part + ((int64_t)((b * a.tiles + rt) * c.Hk + h) * a.split + z) * (16 * (2 + D));
        if (wave == 0 && g == 0) *(float2*)(to + 2 * i) = float2{top, total};
#pragma unroll
        for (int n = 0; n < NP; ++n) *(floatx4*)(to + 32 + i * D + (wave * NP + n) * 16 + 4 * g) = x[n];
        return;
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;          // nothing seen: zeros
#pragma unroll
    for (int n = 0; n < NP; ++n)
        *(uint2*)(a.out + qat + (wave * NP + n) * 16 + 4 * g) =
            uint2{pack_bf16x2(x[n][0] * inv, x[n][1] * inv), pack_bf16x2(x[n][2] * inv, x[n][3] * inv)};
}

// Adds the slices, in slice order: a wavefront takes 256 / D rows, eight slices' loads in flight.  A launch of its
// own: the last workgroup of a row tile to arrive read 8 KB slices that other dies had written at .4 us each (one sequence of 4097
// tokens 13.5 us, of 8192 20).
template <int D>
__global__ __launch_bounds__(64) void k_attention_join_rows(Args a, Sequences s, Cache c) {
    constexpr int L = D / 4, R = 64 / L, kFlight = 8;            // lanes of a row, rows
    const int part = blockIdx.x % (16 / R), h = blockIdx.x / (16 / R) % c.Hk, rest = blockIdx.x / (16 / R) / c.Hk;
    const TileRows<16, kTile> t(a, s, c, rest / a.tiles, rest % a.tiles);
    const int i = part * R + threadIdx.x / L, d = threadIdx.x % L * 4, row = 16 * t.rt + i;
    if (row >= t.rows || t.used == 1) return;
    constexpr uint32_t kPart = 16 * (2 + D) * 4;
    const float* const from = a.part + (int64_t)((t.b * a.tiles + t.rt) * c.Hk + h) * a.split * (kPart / 4);
    // a slice past the last lies outside: it brings zeros and costs nothing (the last one again, instead, cost 4 us)
    const __amdgpu_buffer_rsrc_t pr = rsrc(from, (int64_t)t.used * kPart);
    float m = -INFINITY, sum = 0.f;
    floatx4 x = {0.f, 0.f, 0.f, 0.f};
    for (int z0 = 0; z0 < t.used; z0 += kFlight) {
        float top[kFlight], part_sum[kFlight];
        floatx4 v[kFlight];
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            const uint32_t p = (uint32_t)(z0 + u) * kPart;
            const auto st = __builtin_amdgcn_raw_buffer_load_b64(pr, p + 8 * i, 0, 0);
            top[u] = __uint_as_float(st[0]), part_sum[u] = __uint_as_float(st[1]);
            v[u] = __builtin_bit_cast(floatx4, __builtin_amdgcn_raw_buffer_load_b128(pr, p + 128 + (i * D + d) * 4, 0, 0));
        }
        // every load is on its way before the first is waited for (a branch around their use would take them along)
#pragma unroll
        for (int u = 0; u < kFlight; ++u) asm volatile("" : "+v"(top[u]), "+v"(part_sum[u]), "+v"(v[u]));
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
            if (z0 + u >= t.used) top[u] = -INFINITY;            // past the last slice: nothing
            const float now = fmaxf(m, top[u]), base = now == -INFINITY ? 0.f : now;
            const float keep = __builtin_amdgcn_exp2f(m - base), f = __builtin_amdgcn_exp2f(top[u] - base);
            m = now;
            sum = sum * keep + part_sum[u] * f;
            x = x * keep + v[u] * f;
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    *(uint2*)(a.out + t.at(row, h, a, D) + d) = uint2{pack_bf16x2(x[0] * inv, x[1] * inv), pack_bf16x2(x[2] * inv, x[3] * inv)};
}

// ---------------------------------------------------------------- many rows: tiles in LDS
// Bound by the matrix cores and, beside them, the exponentials.  A workgroup takes 128 rows, 32 for each of four
// wavefronts, and a slice of the tokens, 64 at a time.  K and V of a tile are loaded once for all rows, a tile ahead, widened
// to bf16 with their scales on the way into LDS (exact), two tiles deep, one barrier a tile.
//   first product   S^T = K Q^T by 32x32x16 products: lane (i, h) = (lane % 32, lane / 32) gives row i of K and of Q, and takes,
//                   of query row i, token 8 (r / 4) + 4h + r % 4 of 32;
//   second product  O^T = V^T P^T: the lane's own results are its operand, if V's tokens 16s .. 16s + 15 lie in the order
//                   0-3, 8-11 (h = 0), 4-7, 12-15 (h = 1): the order in which they go into LDS.
// So a row's maximum and sum cross two lanes only.  The running maximum is taken over when a tile passes it by more
// than 2^8 (any reference gives the same quotient, and p up to 2^8 loses nothing), so that the sums are seldom rescaled.
// LDS rows (K: a token, V: a number of the head) keep 16-byte piece q at slot q ^ (row % 16) where a row is 256 bytes, at
// q ^ (row / 2 % 8) where it is 128: lanes that a read serves together hit different banks.
// 256 rows by eight wavefronts and 128 tokens at a time halve what is widened and stored for each product: the faster
// one where there are rows enough (the plan below).
//
// 4096 tokens behind 4096, 64 heads on 8, D = 128: 730-810 us (1.02-1.13 PFLOP/s; a large bf16 product reaches 1.38), 830 with
// 128 rows.  D = 64 by 128 rows, and by 256: 32 heads on 8 298 and 294 us, 32 heads 277 and 265, 4 sequences of 2048 behind 2048 182
// and 170, but one prompt of 2048 43 and 49 (the plan takes 128).  Matrix cores busy in 48 % of the cycles, vector units in about as many: a product on
// one wavefront of a SIMD slows another's additions to two thirds (measured alone), so that exponentials, maxima,
// roundings and widening are not hidden behind it but added.  On one card, 751 us without the products, 713 without
// loads and widening, 530 without the softmax, in a form with the wavefronts' phases set against each other (itself
// 970; the one kept lets the hardware choose).
typedef float floatx16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ floatx16 mfma32x32x16(const bf16x8& a, const bf16x8& b, const floatx16& c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}
// c + the eight numbers
__device__ __forceinline__ float add_pairs(const bf16x8& v, float c) {
    const u32x4 w = __builtin_bit_cast(u32x4, v);
    const bf16x2 one = {(__bf16)1.f, (__bf16)1.f};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t two = w[e];               // (a vector's element itself would be cast from its first bytes)
        c = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, two), one, c, false);
    }
    return c;
}

// A slice's part: maximum and sum of the rows, then the numbers as the lanes hold them.
template <int D, int NW>
struct Partial {
    static constexpr int kRows = 32 * NW, kFloats = kRows * 2 + kRows * D;
    float* base;
    __device__ __forceinline__ Partial(const Args& a, int slot) : base(a.part + (int64_t)slot * a.split * kFloats) {}
    // offsets in floats: of a slice's row's maximum and sum, of four of its numbers
    static __device__ __forceinline__ uint32_t stats_at(int z, int row) { return (uint32_t)z * kFloats + row * 2; }
    static __device__ __forceinline__ uint32_t numbers_at(int z, int wave, int n, int y, int lane) {
        return (uint32_t)z * kFloats + kRows * 2 + (((wave * (D / 32) + n) * 4 + y) * 64 + lane) * 4;
    }
};
// 32 numbers of a row, of which lane (i, h) holds 8y + 4h .. + 3: as bf16, 16 bytes a lane.
__device__ __forceinline__ void write_row32(uint16_t* to, const floatx16& o, float inv, int h, bool on) {
#pragma unroll
    for (int y = 0; y < 4; y += 2) {             // numbers 8y .. + 7 to the lanes of h = 0, the next eight to those of h = 1
        u32x4 out;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const auto w = __builtin_amdgcn_permlane32_swap(pack_bf16x2(o[4 * y + 2 * e] * inv, o[4 * y + 2 * e + 1] * inv),
                                                            pack_bf16x2(o[4 * y + 4 + 2 * e] * inv, o[4 * y + 5 + 2 * e] * inv),
                                                            false, false);
            out[e] = w[0];
            out[2 + e] = w[1];
        }
        if (on) *(u32x4*)(to + 8 * y + 8 * h) = out;
    }
}

// NW wavefronts; 16 NW tokens are staged at a time.
template <int D, int NW>
__global__ __launch_bounds__(64 * NW, 2) void k_attention_tile(Args a, Sequences s, Cache c) {
    constexpr int NP = D / 64, NB = D / 32;      // 16-byte pieces of K and of V per thread; blocks of 32 numbers
    constexpr int kTileRows = 32 * NW, NG = NW, kTokens = 16 * NG;   // groups of 16 tokens of a stage
    constexpr int kVRow = kTokens * 2, kK = kTokens * D * 2, kStage = 2 * kK;
    __shared__ u32x4 lds[2 * kStage / 16];
    lds_poison_start(&lds[0], 2 * kStage / 16);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int i = lane & 31, h = lane >> 5;
    const int head = blockIdx.x % c.Hk, rest = blockIdx.x / c.Hk;
    const int z = rest % a.split, rt = a.tiles - 1 - rest / a.split % a.tiles, b = rest / a.split / a.tiles;
    const TileRows<32 * NW, 16 * NW> g(a, s, c, b, rt);
    const int rows = g.rows, most = g.most, used = g.used;
    if (kTileRows * rt >= rows || z >= used) return;             // the whole workgroup
    const int row = kTileRows * rt + 32 * wave + i, base_row = kTileRows * rt + 32 * wave;
    const int64_t qat = g.at(row, head, a, D);
    // tokens that this lane's row sees, that every row of the wavefront sees, and that any of its rows does
    const int seen = g.reach(row, a), all = g.reach(base_row, a), wave_most = base_row < rows ? g.reach(base_row + 31, a) : 0;
    const int per = (g.tiles + used - 1) / used, tb = min(z * per, g.tiles), te = min(tb + per, g.tiles);

    // scores are f times the products with f > 0: a negative scale's sign goes into q, and so does a zero scale (0 times an
    // infinity or a NaN stays NaN)
    const float f = a.scale == 0.f ? 1.f : fabsf(a.scale);
    const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
    bf16x8 q[D / 16];
#pragma unroll
    for (int n = 0; n < D / 16; ++n) {
        u32x4 v = *(const u32x4*)(a.q + qat + 16 * n + 8 * h);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = a.scale == 0.f ? pack_bf16x2(bf16_lo(v[e]) * 0.f, bf16_hi(v[e]) * 0.f) : v[e] ^ flip;
        q[n] = __builtin_bit_cast(bf16x8, v);
    }

    const int32_t* const table = s.table + (int64_t)b * s.width;
    // of stage `tile`, by lane % NG: the block of 16 tokens, or -1
    auto blocks_of = [&](int tile) __attribute__((always_inline)) {
        const int first = tile * kTokens + 16 * (lane & (NG - 1)), j = first >> c.logT;
        const int v = first < most && j < s.width ? table[j] : -1;
        return v >= 0 && v < c.blocks ? v : -1;
    };
    auto scales_of = [&](int blk) __attribute__((always_inline)) {
        return (uint32_t)*(const uint16_t*)(c.scales + ((int64_t)max(blk, 0) * c.Hk + head) * 2);
    };
    // piece n of this thread: K of one token, V of 16 tokens and one number; both belong to 16 tokens that are the
    // wavefront's
    auto group_of = [&](int n) { return D == 128 ? NG / 2 * n + (wave >> 1) : wave; };
    constexpr int kPieces = D / 16;              // of a K row
    const int token = threadIdx.x / kPieces, piece = threadIdx.x % kPieces, number = threadIdx.x % D;
    // What belongs to 16 tokens is worked out by the lane of that number, for all groups at once, and handed to the
    // wavefront from there: addresses in scalar arithmetic cost more than the products waited.
    const uint32_t k_off = (uint32_t)((token & 15) * D + 16 * piece), v_off = (uint32_t)(16 * number);
    const uint32_t block_bytes = (uint32_t)(c.Hk * c.T * D);
    const uint64_t head_bytes = (uint64_t)(head * c.T) * D;
    auto handed = [&](uint64_t v, int grp) __attribute__((always_inline)) {
        return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, grp) |
                         (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), grp) << 32);
    };
    u32x4 kn[NP], vn[NP];
    auto load = [&](int tile, int blk) __attribute__((always_inline)) {
        const int first = tile * kTokens + 16 * (lane & (NG - 1));
        const uint64_t base = (uint64_t)(uint32_t)max(blk, 0) * block_bytes + head_bytes + (uint32_t)((first & (c.T - 1)) * D);
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            const int64_t at = handed(base, group_of(n));
            kn[n] = *(const u32x4*)(c.k + at + k_off);
            vn[n] = *(const u32x4*)(c.v + at + v_off);
        }
    };
    uint8_t* const lb = (uint8_t*)lds;
    auto k_slot = [](int r, int p) { return D == 128 ? p ^ (r & 15) : p ^ (r / 2 & 7); };
    auto v_slot = [](int r, int p) { return kVRow == 256 ? p ^ (r & 15) : p ^ (r / 2 & 7); };
    auto store = [&](int tile, int stage, int blk, uint32_t e, bool whole) __attribute__((always_inline)) {
        const bool marked = (e & 255) == 255 || e >> 8 == 255;   // K becomes NaN, V finite
        const uint32_t ks = marked ? 0x7f800000u : (e & 255) << 23, vs = marked ? 127u << 23 : (e >> 8) << 23;
        const int live = blk < 0 ? 0 : g.length - tile * kTokens - 16 * (lane & (NG - 1));
#pragma unroll
        for (int n = 0; n < NP; ++n) {
            const int grp = group_of(n), r = 16 * grp + (token & 15);
            const float k_scale = __uint_as_float(__builtin_amdgcn_readlane(ks, grp));
            const float v_scale = __uint_as_float(__builtin_amdgcn_readlane(vs, grp));
            uint8_t* const kr = lb + stage * kStage + r * D * 2;
            *(bf16x8*)(kr + 16 * k_slot(r, 2 * piece)) = widen_codes(kn[n][0], kn[n][1], k_scale);
            *(bf16x8*)(kr + 16 * k_slot(r, 2 * piece + 1)) = widen_codes(kn[n][2], kn[n][3], k_scale);
            u32x4 x = vn[n];
            if (!whole) {
                // what lies behind the sequence's last token, or in no block, may be anything, NaN among it: zeros
                const int left = __builtin_amdgcn_readlane(live, grp);
                const uint64_t lo = left >= 8 ? ~0ull : (1ull << 8 * max(left, 0)) - 1;
                const uint64_t hi = left >= 16 ? ~0ull : left <= 8 ? 0ull : (1ull << 8 * (left - 8)) - 1;
                x &= u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
            }
            uint8_t* const vr = lb + stage * kStage + kK + number * kVRow;
            *(bf16x8*)(vr + 16 * v_slot(number, 2 * grp)) = widen_codes(x[0], x[2], v_scale);
            *(bf16x8*)(vr + 16 * v_slot(number, 2 * grp + 1)) = widen_codes(x[1], x[3], v_scale);
        }
    };

    floatx16 o[NB];
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[n][r] = 0.f;
    float m = -INFINITY, sum = 0.f;

    int blk = blocks_of(tb), next = blocks_of(tb + 1);
    uint32_t sc = scales_of(blk);
    constexpr uint32_t kAll = (1u << NG) - 1;
    uint32_t holes = (uint32_t)__ballot(blk >= 0) & kAll;        // 16-token groups that are there
    load(tb, blk);
    store(tb, 0, blk, sc, false);
    __syncthreads();
    for (int tile = tb; tile < te; ++tile) {
        const int stage = (tile - tb) & 1, base_token = tile * kTokens;
        const uint32_t there = holes;
        if constexpr (kLdsPoison) {              // the other stage, between its last reader and its next writer
            for (int e = threadIdx.x; e < kStage / 16; e += 64 * NW) lds[(stage ^ 1) * (kStage / 16) + e] = lds_nan16();
            __syncthreads();
        }
        blk = next;
        next = blocks_of(tile + 2);
        if (tile + 1 < te) {
            sc = scales_of(blk);
            holes = (uint32_t)__ballot(blk >= 0) & kAll;
            load(tile + 1, blk);
        }
#pragma unroll
        for (int part = 0; part < NG / 4; ++part) {              // 64 tokens at a time
            const int first = base_token + 64 * part;
            if (first >= wave_most) break;
            const uint32_t groups = there >> 4 * part & 15;
            const uint8_t* const kb = lb + stage * kStage + 64 * part * D * 2;
            floatx16 p[2];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int r = 0; r < 16; ++r) p[u][r] = 0.f;
#pragma unroll
            for (int n = 0; n < D / 16; ++n)
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    p[u] = mfma32x32x16(*(const bf16x8*)(kb + (32 * u + i) * D * 2 + 16 * k_slot(i, 2 * n + h)), q[n], p[u]);
            if (first + kTile > all || groups != 15) {            // a token that some row does not see
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const int at = 32 * u + 8 * (r / 4) + 4 * h + r % 4;
                        if (!(first + at < seen && groups >> (2 * u + r / 8) & 1)) p[u][r] = -INFINITY;
                    }
            }
            // (a maximum that hands on NaN, which makes the row NaN anyway: one instruction for two numbers, in two chains:
            // pairs first would be half as many instructions again)
            float tops[2] = {p[0][0], p[1][0]};
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
                for (int r = 1; r < 15; r += 2) {
                    tops[u] = __builtin_elementwise_maximum(__builtin_elementwise_maximum(tops[u], p[u][r]), p[u][r + 1]);
                }
            }
            float top = __builtin_elementwise_maximum(__builtin_elementwise_maximum(tops[0], p[0][15]), __builtin_elementwise_maximum(tops[1], p[1][15]));
            const auto both = __builtin_amdgcn_permlane32_swap(__float_as_uint(top), __float_as_uint(top), false, false);
            top = __builtin_elementwise_maximum(__uint_as_float(both[0]), __uint_as_float(both[1])) * f;
            const bool passed = top > m + 8.f;   // the first numbers are, beside minus infinity
            if (__any(passed)) {                 // each row by itself: its result does not depend on its neighbours'
                const float now = passed ? top : m, base = now == -INFINITY ? 0.f : now;
                const float keep = __builtin_amdgcn_exp2f(m - base);
                m = now;
                sum *= keep;
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int r = 0; r < 16; ++r) o[n][r] *= keep;
            }
            const float base = m == -INFINITY ? 0.f : m;
            float by = f;
            const bool far = fabsf(base) > 0x1p24f;
            if (__any(far)) {                    // the products rounded before the difference, as the maximum was: half a step
                by = far ? 1.f : f;              // of such a maximum would be a power of two of its own
                const float to = far ? f : 1.f;
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int r = 0; r < 16; ++r) p[u][r] *= to;
            }
            bf16x8 w[4];                         // 16 tokens each
#pragma unroll
            for (int u = 0; u < 2; ++u) {
#pragma unroll
                for (int r = 0; r < 16; ++r) p[u][r] = __builtin_amdgcn_exp2f(fmaf(p[u][r], by, -base));
#pragma unroll
                for (int y = 0; y < 2; ++y)
                    w[2 * u + y] = __builtin_bit_cast(
                        bf16x8, u32x4{pack_bf16x2(p[u][8 * y], p[u][8 * y + 1]), pack_bf16x2(p[u][8 * y + 2], p[u][8 * y + 3]),
                                      pack_bf16x2(p[u][8 * y + 4], p[u][8 * y + 5]), pack_bf16x2(p[u][8 * y + 6], p[u][8 * y + 7])});
            }
            // the sum of the rounded p, two in an instruction, in float32: what the second product weighs V with
#pragma unroll
            for (int y = 0; y < 4; ++y) sum = add_pairs(w[y], sum);
            const uint8_t* const vb = lb + stage * kStage + kK;
#pragma unroll
            for (int y = 0; y < 4; ++y)
#pragma unroll
                for (int n = 0; n < NB; ++n)
                    o[n] = mfma32x32x16(*(const bf16x8*)(vb + (32 * n + i) * kVRow + 16 * v_slot(i, 8 * part + 2 * y + h)), w[y], o[n]);
        }
        if (tile + 1 < te) store(tile + 1, stage ^ 1, blk, sc, holes == kAll && (tile + 2) * kTokens <= g.length);
        __syncthreads();
    }
    const auto halves = __builtin_amdgcn_permlane32_swap(__float_as_uint(sum), __float_as_uint(sum), false, false);
    sum = __uint_as_float(halves[0]) + __uint_as_float(halves[1]);
#pragma unroll
    for (int n = 0; n < NB; ++n) asm volatile("" : "+v"(o[n]));  // the products stay before the branches
    if (used > 1) {                              // several slices: k_attention_join adds them
        using P = Partial<D, NW>;
        const P to(a, (b * a.tiles + rt) * c.Hk + head);
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int y = 0; y < 4; ++y)
                *(floatx4*)(to.base + P::numbers_at(z, wave, n, y, lane)) = floatx4{o[n][4 * y], o[n][4 * y + 1], o[n][4 * y + 2], o[n][4 * y + 3]};
        to.base[P::stats_at(z, 32 * wave + i) + h] = h ? sum : m;
        return;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;              // nothing seen: zeros
#pragma unroll
    for (int n = 0; n < NB; ++n) write_row32(a.out + qat + 32 * n, o[n], inv, h, row < rows);
}

// Adds the slices of the tiles above, in slice order: a workgroup takes 32 rows, a wavefront 32 numbers of each.
// (By the last workgroup to arrive the join of 16 slices of 128 rows took longer than the slices.)
template <int D, int NW>
__global__ __launch_bounds__(2 * D) void k_attention_join(Args a, Sequences s, Cache c) {
    const int n = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, i = lane & 31, h = lane >> 5;
    const int wave = blockIdx.x % NW, head = blockIdx.x / NW % c.Hk, rest = blockIdx.x / NW / c.Hk;
    const TileRows<32 * NW, 16 * NW> r(a, s, c, rest / a.tiles, rest % a.tiles);
    const int row = 32 * NW * r.rt + 32 * wave + i;
    if (32 * NW * r.rt + 32 * wave >= r.rows || r.used == 1) return;
    using P = Partial<D, NW>;
    const P from(a, (r.b * a.tiles + r.rt) * c.Hk + head);
    const __amdgpu_buffer_rsrc_t pr = rsrc(from.base, (int64_t)r.used * P::kFloats * 4);   // past the last slice: zeros
    float m = -INFINITY, sum = 0.f;
    floatx16 o;
#pragma unroll
    for (int e = 0; e < 16; ++e) o[e] = 0.f;
    for (int z0 = 0; z0 < r.used; z0 += 4) {     // four slices' loads in flight
        float top[4], part_sum[4];
        floatx4 v[4][4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const auto st = __builtin_amdgcn_raw_buffer_load_b64(pr, P::stats_at(z0 + u, 32 * wave + i) * 4, 0, 0);
            top[u] = __uint_as_float(st[0]), part_sum[u] = __uint_as_float(st[1]);
#pragma unroll
            for (int y = 0; y < 4; ++y)
                v[u][y] = __builtin_bit_cast(floatx4, __builtin_amdgcn_raw_buffer_load_b128(pr, P::numbers_at(z0 + u, wave, n, y, lane) * 4, 0, 0));
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)              // on their way together
            asm volatile("" : "+v"(top[u]), "+v"(part_sum[u]), "+v"(v[u][0]), "+v"(v[u][1]), "+v"(v[u][2]), "+v"(v[u][3]));
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (z0 + u >= r.used) top[u] = -INFINITY;            // past the last slice: nothing
            const float now = fmaxf(m, top[u]), base = now == -INFINITY ? 0.f : now;
            const float keep = __builtin_amdgcn_exp2f(m - base), g = __builtin_amdgcn_exp2f(top[u] - base);
            m = now;
            sum = sum * keep + part_sum[u] * g;
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = o[e] * keep + v[u][e / 4][e % 4] * g;
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    write_row32(a.out + r.at(row, head, a, D) + 32 * n, o, inv, h, row < r.rows);
}

}  // namespace

// Which kernel, and how many slices of the tokens, by the time that each would take: us on this card, fitted to 7000
// launches (1 .. 256 sequences of 1 .. 8192 new tokens and up to 16384, 1 .. 40 heads; a kernel in the mean within 17 %):
//   start + each * x + turns * turn * (1 + crowd * seen * x), where x is the workgroups over those that the card holds at a
//   time, a turn the kernel's tokens at a time (256 of the rows kernel's four wavefronts), seen the part of the tokens that
//   causal rows see, and for joining slices join + per MB of partials.
// What this takes is in the mean 1.6 % slower than the best of all, where 32 rows and 1024 rows as bounds between the kernels
// and slices for 512 workgroups took 10 %: 2 sequences of 85 tokens, 32 heads: 16 rows 9.2 us, 128 rows 15.8; 42 of 109 tokens,
// 16 heads of q on one: 16, 128, 256 rows 36, 17, 20; 38 of 103 tokens behind 8400, 32 heads on 8: 633, 448, 393.
// (The fit puts D = 64's 256 rows a few percent too high: long prompts lose up to 6 % by it, short ones would lose 14.)
// Where there are 512 workgroups or more without slices there are none (64 sequences of up to 8192, 64 heads on 8: 1 slice
// 118 us, 2 130), and never more than 1024 with them (up to 2048: the same in the mean).
// `tokens`: what the table covers, the only bound of the lengths that the host has.  One kernel and one number of slices
// serve all sequences of a call: one of 65536 tokens among 63 of 1000 takes 422 us (alone 30), a prompt of 2048 beside 63
// single tokens behind 8000 1354 (apart 97 and 189).
AttentionPlan plan_attention(int64_t M, int n_seq, int max_q, int Hq, int Hk, int D, int64_t tokens) {
    struct Kernel {
        int rows, turn_tokens, held;
        double start[2], each[2], turn[2], crowd[2], join[2], join_mb;   // for D = 64 and 128
    };
    static const Kernel kernels[3] = {
        {16, 256, 512, {4.9, 4.8}, {1.17, 2.08}, {1.04, 1.47}, {.83, 1.05}, {1.9, 2.}, .6},
        {128, 64, 512, {5.9, 7.1}, {1.4, 1.5}, {.95, 1.28}, {.6, .77}, {2.3, 1.6}, .25},
        {256, 128, 256, {6.3, 9.2}, {1.9, 1.9}, {2.05, 2.7}, {.585, .657}, {2.5, 1.}, .25}};
    AttentionPlan p{};
    const int64_t rows = std::min<int64_t>(max_q, M) * (Hq / Hk), slices = (tokens + kSliceTokens - 1) / kSliceTokens;
    const double seen = 1 - .5 * std::min((double)max_q / (double)tokens, 1.);
    const int d = D == 128;
    double best = 1e300;
    int before = 0;
    for (const Kernel& k : kernels) {
        if (rows <= before) break;               // the kernel before holds them in one tile
        before = k.rows;
        const int64_t tiles = (rows + k.rows - 1) / k.rows, slots = n_seq * tiles * Hk, turns = (tokens + k.turn_tokens - 1) / k.turn_tokens;
        const int most = slots >= 512 ? 1 : (int)std::min<int64_t>(32, 1024 / slots);
        const size_t part = k.rows * (8 + 4 * (size_t)D);
        // whatever the table covers: the size that a caller asks for does not know it
        if (most > 1) p.ws_bytes = std::max(p.ws_bytes, kCounterBytes + (size_t)slots * most * part);
        for (int z = 1; z <= most && (z == 1 || z <= slices); z += z < 4 ? 1 : (z & (z - 1)) == 0 ? z / 2 : z / 3) {
            const double x = (double)(slots * z) / k.held, mb = 1e-6 * (double)(slots * z) * (double)part;
            const double us = k.start[d] + k.each[d] * x + (double)((turns + z - 1) / z) * k.turn[d] * (1 + k.crowd[d] * seen * x) +
                              (z == 1 ? 0 : k.join[d] + k.join_mb * mb);
            if (us >= best) continue;
            best = us;
            p.rows = k.rows;
            p.tiles = (int)tiles;
            p.split = z;
        }
    }
    return p;
}

hipError_t launch_attention(const uint16_t* q, int64_t M, int Hq, const Sequences& s, const Cache& c, float scale,
                            int causal, uint16_t* out, void* ws, const AttentionPlan& p, hipStream_t st) {
    const Args a{q, out, (float*)((char*)ws + kCounterBytes), (int)M, Hq, Hq / c.Hk, causal, p.tiles, p.split,
                 scale * kLog2e};
    const unsigned grid = (unsigned)((int64_t)s.n * p.tiles * p.split * c.Hk);
    const auto go = [&](auto kernel) {
        kernel<<<grid, attention_threads(p), 0, st>>>(a, s, c);
        return hipGetLastError();
    };
    const auto both = [&](auto kernel, auto join, int per_slot, int threads) {
        const hipError_t e = go(kernel);
        if (e != hipSuccess || p.split == 1) return e;
        join<<<(unsigned)((int64_t)s.n * p.tiles * c.Hk * per_slot), threads, 0, st>>>(a, s, c);
        return hipGetLastError();
    };
    const auto tiles = [&](auto kernel, auto join) { return both(kernel, join, p.rows / 32, 2 * c.D); };
    if (p.rows == 16)
        return c.D == 128 ? both(k_attention_rows<128>, k_attention_join_rows<128>, 8, 64)
                          : both(k_attention_rows<64>, k_attention_join_rows<64>, 4, 64);
    if (p.rows == 128)
        return c.D == 128 ? tiles(k_attention_tile<128, 4>, k_attention_join<128, 4>)
                          : tiles(k_attention_tile<64, 4>, k_attention_join<64, 4>);
    return c.D == 128 ? tiles(k_attention_tile<128, 8>, k_attention_join<128, 8>)
                      : tiles(k_attention_tile<64, 8>, k_attention_join<64, 8>);
}

}  // namespace awq
