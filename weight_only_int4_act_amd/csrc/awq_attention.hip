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
constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kTile = 64;                        // tokens that a wavefront takes at a time
constexpr size_t kCounterBytes = 65536;

// Eight e4m3 codes (two words) times 2^(E - 127), the scale's exponent field, in bf16: exact.
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
    uint32_t* cnt;
    int M, Hq, G, causal, tiles, split, cstride;
    float scale;                 // times log2 e
};

// ---------------------------------------------------------------- few rows: the cache streamed once
// Bound by the cache's bytes.  A workgroup takes 16 rows and a slice of the tokens; its four wavefronts take every
// fourth tile of 64 tokens of it.  A lane (i, g) = (lane % 16, lane / 16) works for tokens 16g .. 16g + 15 of the tile in
// both products, so that what belongs to those tokens (their block, its scales, the mask) is the lane's own:
//   first product   S^T = K Q^T, four 16 x 16 results: row 4g + r of result t is token 16g + 4t + r, so lane
//                   (i, g) gives K's row of token 16 (i / 4) + 4t + i % 4, and takes 16 results of query row i;
//   second product  O^T = V^T P^T: lane (i, g) gives the 16 bytes of number i of V's 16 tokens, and its own
//                   results, in the order in which they are.
// K and V become bf16 in registers (exact).  The running maximum and sum are per row; every wavefront has its own,
// joined in LDS at the end, and those of several slices by the last workgroup to arrive, in slice order.
template <int D>
__global__ __launch_bounds__(256) void k_attention_rows(Args a, Sequences s, Cache c) {
    constexpr int ND = D / 16, NH = D / 64;
    __shared__ floatx4 red[4][ND][64];
    __shared__ float stat[4][2][16];
    __shared__ uint32_t arrival;
    lds_poison_start(&red[0][0][0], 4 * ND * 64);
    lds_poison_start(&stat[0][0][0], 128);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int i = lane & 15, g = lane >> 4;
    const int h = blockIdx.x % c.Hk, rest = blockIdx.x / c.Hk;
    const int z = rest % a.split, rt = rest / a.split % a.tiles, b = rest / a.split / a.tiles;
    const NewTokens t = new_tokens(s, b, a.M);
    const int rows = min(t.count, s.max_q) * a.G;
    if (16 * rt >= rows) return;                 // the whole workgroup
    const int row = 16 * rt + i, tok = min(row, rows - 1) / a.G, head = h * a.G + min(row, rows - 1) % a.G;
    const int64_t qat = ((int64_t)(t.row0 + tok) * a.Hq + head) * D;
    // tokens that this lane's row sees, and that any row of the workgroup sees
    const int last_tok = min(16 * rt + 15, rows - 1) / a.G;
    const int cap = s.width << c.logT;           // what the table covers
    const int seen = min(a.causal ? max(t.start + tok + 1, 0) : t.length, cap);
    const int most = min(a.causal ? max(t.start + last_tok + 1, 0) : t.length, cap);
    const int tiles = (most + kTile - 1) / kTile;
    const int used = max(min(a.split, (tiles + 3) / 4), 1);      // slices of this sequence: four tiles each or more
    if (z >= used) return;
    const int per = (tiles + used - 1) / used, tb = min(z * per, tiles), te = min(tb + per, tiles);

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
    auto block_of = [&](int first) {
        const int j = first >> c.logT;
        const int v = first < most && j < s.width ? table[j] : -1;
        return v >= 0 && v < c.blocks ? v : -1;
    };
    for (int tile = tb + wave; tile < te; tile += 4) {
        const int first = tile * kTile;
        const int kg = i >> 2;                   // the 16 tokens whose K this lane gives
        const int bk = block_of(first + 16 * kg), bv = block_of(first + 16 * g);
        u32x4 k[4][NH], v[ND];
        const uint8_t* const kp = c.k + (((int64_t)max(bk, 0) * c.Hk + h) * c.T + ((first + 16 * kg) & (c.T - 1)) + (i & 3)) * D + 16 * g;
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int n = 0; n < NH; ++n) k[u][n] = *(const u32x4*)(kp + 4 * u * D + 64 * n);
        const uint8_t* const vp = c.v + (((int64_t)max(bv, 0) * c.Hk + h) * c.T + ((first + 16 * g) & (c.T - 1))) * D + 16 * i;
#pragma unroll
        for (int n = 0; n < ND; ++n) v[n] = *(const u32x4*)(vp + 256 * n);
        const uint32_t e = *(const uint16_t*)(c.scales + ((int64_t)max(bv, 0) * c.Hk + h) * 2);
        const bool poisoned = (e & 255) == 255 || e >> 8 == 255;
        // a marked block makes what is seen of it NaN; V's own scale then is any finite one
        const float f = poisoned ? NAN : __uint_as_float((e & 255) == 0 ? 0x00400000u : (e & 255) << 23) * a.scale;
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
        // token 16g + 4u + r of the tile is seen when it lies below `limit`
        const int limit = bv < 0 ? 0 : seen - first - 16 * g;
        float top = -INFINITY;
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                p[u][r] = 4 * u + r < limit ? p[u][r] * f : -INFINITY;
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
        bf16x8 w[2];
#pragma unroll
        for (int y = 0; y < 2; ++y)
            w[y] = __builtin_bit_cast(bf16x8, u32x4{pack_bf16x2(p[2 * y][0], p[2 * y][1]), pack_bf16x2(p[2 * y][2], p[2 * y][3]),
                                                    pack_bf16x2(p[2 * y + 1][0], p[2 * y + 1][1]),
                                                    pack_bf16x2(p[2 * y + 1][2], p[2 * y + 1][3])});
        // what lies behind the sequence's last token may be anything, NaN among it: zeros
        const int live = bv < 0 ? 0 : t.length - first - 16 * g;
#pragma unroll
        for (int n = 0; n < ND; ++n) {
#pragma unroll
            for (int r = 0; r < 4; ++r) o[n][r] *= keep;
            u32x4 x = v[n];
            if (live < 16) {
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int left = min(max(live - 4 * y, 0), 4);
                    x[y] = left == 4 ? x[y] : x[y] & ((1u << 8 * left) - 1);
                }
            }
            o[n] = mfma16x16x32(widen_codes(x[0], x[1], fv), w[0], o[n]);
            o[n] = mfma16x16x32(widen_codes(x[2], x[3], fv), w[1], o[n]);
        }
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
    auto write = [&]() __attribute__((always_inline)) {
        const float inv = total == 0.f ? 0.f : 1.f / total;      // nothing seen: zeros
        if (row >= rows) return;
#pragma unroll
        for (int n = 0; n < NP; ++n)
            *(uint2*)(a.out + qat + (wave * NP + n) * 16 + 4 * g) =
                uint2{pack_bf16x2(x[n][0] * inv, x[n][1] * inv), pack_bf16x2(x[n][2] * inv, x[n][3] * inv)};
    };
    if (used == 1) {
        write();
        return;
    }
    // several slices: maximum and sum of the 16 rows, then the numbers, per slice
    constexpr uint32_t kPart = 16 * 2 * 4 + 16 * D * 4;
    const int slot = (b * a.tiles + rt) * c.Hk + h;
    const __amdgpu_buffer_rsrc_t pr = rsrc((const char*)a.part + (int64_t)slot * a.split * kPart, (int64_t)a.split * kPart);
    auto pat = [&](int z, int n) { return z * kPart + 128 + (uint32_t)((wave * NP + n) * 64 + lane) * 16; };
#pragma unroll
    for (int n = 0; n < NP; ++n) store4_agent(pr, pat(z, n), x[n]);
    if (wave == 0 && g == 0) {
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(top), pr, z * kPart + i * 4, 0, kCpolAgent);
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(total), pr, z * kPart + 64 + i * 4, 0, kCpolAgent);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // this wavefront's part has landed
    __syncthreads();
    uint32_t* const counter = a.cnt + (int64_t)slot * a.cstride;
    if (threadIdx.x == 0) arrival = __hip_atomic_fetch_add(counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    if (arrival != (uint32_t)(used - 1)) return;
    float ms = -INFINITY, ts = 0.f;
#pragma unroll
    for (int n = 0; n < NP; ++n) x[n] = floatx4{0.f, 0.f, 0.f, 0.f};
    for (int z0 = 0; z0 < used; z0 += 4) {       // four slices' loads in flight
        float mz[4], tz[4];
        floatx4 v[4][NP];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int zz = min(z0 + u, used - 1);
            mz[u] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(pr, zz * kPart + i * 4, 0, kCpolAgent));
            tz[u] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(pr, zz * kPart + 64 + i * 4, 0, kCpolAgent));
#pragma unroll
            for (int n = 0; n < NP; ++n) v[u][n] = load4_agent(pr, pat(zz, n));
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (z0 + u >= used) break;
            const float next = fmaxf(ms, mz[u]), base = next == -INFINITY ? 0.f : next;
            const float keep = __builtin_amdgcn_exp2f(ms - base), f = __builtin_amdgcn_exp2f(mz[u] - base);
            ms = next;
            ts = ts * keep + tz[u] * f;
#pragma unroll
            for (int n = 0; n < NP; ++n) x[n] = x[n] * keep + v[u][n] * f;
        }
    }
    total = ts;
    write();
    if (threadIdx.x == 0) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

}  // namespace

AttentionPlan plan_attention(int64_t M, int n_seq, int max_q, int Hq, int Hk, int D) {
    AttentionPlan p{};
    const int64_t rows = std::min<int64_t>(max_q, M) * (Hq / Hk);
    p.tiles = (int)((rows + 15) / 16);
    const int64_t slots = (int64_t)n_seq * p.tiles * Hk;
    p.split = 1;
    if (slots <= (int64_t)(kCounterBytes / 4))
        while (p.split < 64 && slots * p.split < 1024) p.split *= 2;
    p.cstride = (int)std::max<int64_t>(1, std::min<int64_t>(32, kCounterBytes / 4 / slots));
    p.ws_bytes = p.split > 1 ? kCounterBytes + (size_t)slots * p.split * (128 + 64 * (size_t)D) : 0;
    return p;
}

hipError_t launch_attention(const uint16_t* q, int64_t M, int Hq, const Sequences& s, const Cache& c, float scale,
                            int causal, uint16_t* out, void* ws, const AttentionPlan& p, hipStream_t st) {
    const Args a{q, out, (float*)((char*)ws + kCounterBytes), (uint32_t*)ws, (int)M, Hq, Hq / c.Hk, causal, p.tiles,
                 p.split, p.cstride, scale * kLog2e};
    const unsigned grid = (unsigned)((int64_t)s.n * p.tiles * p.split * c.Hk);
    if (c.D == 128) k_attention_rows<128><<<grid, 256, 0, st>>>(a, s, c);
    else k_attention_rows<64><<<grid, 256, 0, st>>>(a, s, c);
    return hipGetLastError();
}

}  // namespace awq
