// q|k|v of new tokens: norms of queries and keys per head, rotation, and the append of keys and values to the 8-bit
// cache.
#include <type_traits>

#include "awq_cache.h"

namespace awq {
namespace {

// The scale byte of a block whose largest number has the float32 bits `top`.  From 1.9375 2^127 on the element would be 256 under
// E = 247, which stands for 2^128 and no finite float32 or bf16 number: an infinity as well.  (Elements of 240 at most in its
// place, by a clamp of every number, cost a long prompt 1 us of 89.)
__device__ __forceinline__ uint32_t cache_scale_byte(uint32_t top) {
    return top >= 0x7f780000u ? 255u : (uint32_t)max((int)(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u), 0);
}
// The conversions' scale operand: they read the exponent field alone (0 is 2^-127).
__device__ __forceinline__ float cache_scale(uint32_t E) { return __uint_as_float(E << 23); }

typedef short s16x2 __attribute__((ext_vector_type(2)));
typedef float floatx2 __attribute__((ext_vector_type(2)));

// Eight numbers over their block's scale; none is beyond 448 times it.
__device__ __forceinline__ uint2 cache_codes8(const float (&p)[8], uint32_t E) {
    const float scale = cache_scale(E);
    uint32_t w[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        s16x2 r = {0, 0};
        r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, p[4 * h], p[4 * h + 1], scale, false);
        r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, p[4 * h + 2], p[4 * h + 3], scale, true);
        w[h] = E == 255 ? 0u : __builtin_bit_cast(uint32_t, r);
    }
    return uint2{w[0], w[1]};
}
// Four codes over 2^d: what an older scale wrote, to a larger one.  Past 2^-30 every code becomes zero.
__device__ __forceinline__ uint32_t cache_rescale4(uint32_t w, uint32_t d) {
    const float scale = cache_scale(127u + min(d, 40u));
    const floatx2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
    s16x2 r = {0, 0};
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, a[0], a[1], scale, false);
    r = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r, b[0], b[1], scale, true);
    return __builtin_bit_cast(uint32_t, r);
}

__device__ __forceinline__ void widen8(const u32x4& v, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(v[i]);
        x[2 * i + 1] = bf16_hi(v[i]);
    }
}

// One head of D numbers is held by D / 8 consecutive lanes, eight numbers each.
template <int D>
struct Head {
    static constexpr int L = D / 8;              // lanes
    // the sum of squares over the head's lanes
    static __device__ __forceinline__ double sum(double v) {
        auto add = [&](auto move) {
            const uint64_t b = __builtin_bit_cast(uint64_t, v);
            const uint64_t o = (uint64_t)(uint32_t)move((int)(uint32_t)b) | ((uint64_t)(uint32_t)move((int)(uint32_t)(b >> 32)) << 32);
            v += __builtin_bit_cast(double, o);
        };
        add([](int x) { return __builtin_amdgcn_mov_dpp(x, 0xB1, 0xf, 0xf, true); });    // lanes 1 0 3 2
        add([](int x) { return __builtin_amdgcn_mov_dpp(x, 0x4E, 0xf, 0xf, true); });    // lanes 2 3 0 1
        add([](int x) { return __builtin_amdgcn_mov_dpp(x, 0x141, 0xf, 0xf, true); });   // mirrored within 8
        if constexpr (L == 16) add([](int x) { return __builtin_amdgcn_mov_dpp(x, 0x140, 0xf, 0xf, true); });   // within 16
        return v;
    }
    // lane l's number from lane l + L/2 modulo L
    static __device__ __forceinline__ float across(float x) {
        int v = __float_as_int(x);
        if constexpr (L == 16) {
            v = __builtin_amdgcn_mov_dpp(v, 0x128, 0xf, 0xf, true);                          // turned by 8 within 16
        } else {
            v = __builtin_amdgcn_mov_dpp(v, 0x141, 0xf, 0xf, true);                          // mirrored within 8 ..
            v = __builtin_amdgcn_mov_dpp(v, 0x1B, 0xf, 0xf, true);                           // .. and within 4
        }
        return __int_as_float(v);
    }
    static __device__ __forceinline__ void norm(float (&x)[8], const uint16_t* weight, int l, double eps) {
        double s = 0.;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += (double)x[i] * (double)x[i];
        const double m = sum(s) * (1. / D) + eps, y = __builtin_amdgcn_rsq(m);
        const float r = (float)(m < __builtin_inf() ? y * (1.5 - 0.5 * m * y * y) : y);   // infinity: 0; NaN: NaN
        float w[8];
        widen8(*(const u32x4*)(weight + l * 8), w);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
    }
    // pairs (i, i + R/2) or (2i, 2i + 1); turn: the row of the rotation's table
    static __device__ __forceinline__ void rotate(float (&x)[8], const float* turn, int R, int interleaved, int l) {
        const int half = R / 16;                 // lanes of the cosines
        const bool in = l < 2 * half;
        if (interleaved) {
            const int at = in ? 4 * l : 0;
            const floatx4 c = *(const floatx4*)(turn + at), s = *(const floatx4*)(turn + R / 2 + at);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = x[2 * i], b = x[2 * i + 1];
                if (in) x[2 * i] = a * c[i] - b * s[i], x[2 * i + 1] = b * c[i] + a * s[i];
            }
            return;
        }
        const bool low = l < half;
        const int at = in ? 8 * (low ? l : l - half) : 0, lane = threadIdx.x & 63;
        const int other = in ? (low ? lane + half : lane - half) : lane;
        const floatx4 c[2] = {*(const floatx4*)(turn + at), *(const floatx4*)(turn + at + 4)};
        const floatx4 s[2] = {*(const floatx4*)(turn + R / 2 + at), *(const floatx4*)(turn + R / 2 + at + 4)};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float o = R == D ? across(x[i]) : __shfl(x[i], other, kWave), t = o * s[i / 4][i % 4];
            if (in) x[i] = x[i] * c[i / 4][i % 4] + (low ? -t : t);
        }
    }
};

// Codes of four tokens, eight numbers each in the two words of lanes l, l + 16, l + 32, l + 48 (token lane / 16): after it
// lane l + 16 g holds numbers 2g and 2g + 1 of its eight, a word of the four tokens each.
__device__ __forceinline__ uint2 four_tokens(const uint2& w) {
    const auto a = __builtin_amdgcn_permlane32_swap(w.x, w.y, false, false);     // tokens 0, 1 and 2, 3 of one word
    const uint32_t even = __builtin_amdgcn_perm(a[1], a[0], 0x05040100u), odd = __builtin_amdgcn_perm(a[1], a[0], 0x07060302u);
    const auto b = __builtin_amdgcn_permlane16_swap(even, odd, false, false);    // two numbers of tokens 0, 2 and of 1, 3
    return uint2{__builtin_amdgcn_perm(b[1], b[0], 0x06020400u), __builtin_amdgcn_perm(b[1], b[0], 0x07030501u)};
}

// The new tokens of one block of the cache for one head of K and V are one workgroup's work, those of the heads of q that
// read it another `parts` workgroups', or its own (OWN) where they are no more heads than a block has of K.  Bound by HBM for
// many tokens (per number of q 4 bytes, of K and V 3), by the chain of dependent reads for few (lengths, blocks, rows).
// Two kernels rather than one with both ways: its registers left half the wavefronts (12000 tokens of 64 heads on 8
// 160 us, now 109).  The numbers of K (float32, normed and rotated) and V (bf16) stay in registers until the block's
// largest are known.  V's codes go through LDS into their order: sixteen tokens of a number in one store where all of
// them are new, else bytes.  6100 tokens of 40 heads, T = 16: 89 us (3.9 TB/s); one token of 64 sequences, 64 heads on 8, with
// norms: 6.8 us, of which the launch takes 2.2 and three trips to memory one after the other the rest.
template <int D, int T, bool OWN>
__global__ __launch_bounds__(256) void k_qkv_append(AppendArgs a, Sequences s, Cache c, int per_seq, int most_parts) {
    const int parts = OWN ? 0 : most_parts;
    using H = Head<D>;
    constexpr int L = H::L, W = 256 / L, U = (T + W - 1) / W;   // lanes of a head, heads at a time, rounds of a block
    __shared__ uint32_t tops[4][2];
    __shared__ u32x4 vt[T / 16 * D];
    lds_poison_start(&tops[0][0], 8);
    lds_poison_start(&vt[0], T / 16 * D);
    const int h = blockIdx.x % c.Hk, part = blockIdx.x / c.Hk % (parts + 1), rest = blockIdx.x / c.Hk / (parts + 1);
    const int j = rest % per_seq, b = rest / per_seq;
    const NewTokens t = new_tokens(s, b, (int)a.M);
    const int lane = threadIdx.x & 63, l = threadIdx.x % L;
    // which head of the W: those of lanes 16 apart are neighbours, for four_tokens
    const int w = (threadIdx.x >> 6) * (64 / L) + (lane >> 4) + (L == 8 ? 4 * (lane >> 3 & 1) : 0);
    const int G = a.Hq / c.Hk;
    const int64_t row_size = (int64_t)(a.Hq + 2 * c.Hk) * D;

    // positions below zero: no block; the first workgroup of a head writes zeros
    if (j == 0 && part == parts && t.start < 0) {
        const int none = min(min(t.count, -t.start), s.max_q);
        for (int i = w; i < none * G; i += W)
            *(u32x4*)(a.q + (((int64_t)t.row0 + i / G) * a.Hq + h * G + i % G) * D + l * 8) = u32x4{0, 0, 0, 0};
    }
    const int64_t index = max(t.start, 0) / T + j;               // the block's, of the sequence
    const int64_t p0 = max((int64_t)t.start, index * T);
    const int64_t p1 = min(min((int64_t)t.length, (index + 1) * T), (int64_t)t.start + s.max_q);
    if (t.count <= 0 || p0 >= p1) return;        // the whole workgroup
    const int n = (int)(p1 - p0), slot0 = (int)(p0 - index * T);
    const int row0 = t.row0 + (int)(p0 - t.start);
    const int turned = a.rope ? (int)min(max((int64_t)a.P - p0, (int64_t)0), (int64_t)n) : n;   // tokens that the rotation covers
    // q: a head's eight numbers of this lane, of token tok
    const int items = n * G;
    struct Item {                                // a head of q: its token, where it is in q|k|v's row, whether it is one
        int tok, col;
        bool in;
        u32x4 raw;
    };
    auto q_load = [&](int i, Item& q) __attribute__((always_inline)) {
        q.in = i < items;                        // past the last: it again, not stored
        q.tok = min(i, items - 1) / G;
        q.col = (h * G + min(i, items - 1) - q.tok * G) * D + l * 8;
        q.raw = *(const u32x4*)(a.qkv + (int64_t)(row0 + q.tok) * row_size + q.col);
    };
    auto q_do = [&](const Item& q) __attribute__((always_inline)) {
        float x[8];
        widen8(q.raw, x);
        if (a.q_weight) H::norm(x, a.q_weight, l, a.eps);
        if (a.rope) {
            H::rotate(x, a.rope + min(p0 + q.tok, (int64_t)a.P - 1) * a.R, a.R, a.interleaved, l);
            if (q.tok >= turned) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = 0.f;
            }
        }
        if (q.in)
            *(u32x4*)(a.q + (int64_t)(row0 + q.tok) * a.Hq * D + q.col) =
                u32x4{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])};
    };
    if (part < parts) {                          // the tokens' G heads, four at a time
        for (int i0 = part * 4 * W; i0 < items; i0 += 4 * W * parts) {
            Item x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (i0 + e * W < items) q_load(i0 + e * W + w, x[e]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (i0 + e * W < items) q_do(x[e]);
        }
        return;
    }
    const int64_t block = index < s.width ? s.table[(int64_t)b * s.width + index] : -1;
    const bool stored = block >= 0 && block < c.blocks && turned > 0;
    const int64_t at = block * c.Hk + h;
    const int slot1 = slot0 + turned;            // slots slot0 .. slot1 - 1 get tokens; head w of round u has slot u W + w

    u32x4 kr[U], v[U];
    Item qr[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (OWN && u * W < items) q_load(u * W + w, qr[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int i = min(max(u * W + w - slot0, 0), n - 1);
        const uint16_t* const row = a.qkv + (int64_t)(row0 + i) * row_size + (int64_t)(a.Hq + h) * D + l * 8;
        if (u * W + W <= slot0 || u * W >= slot1) continue;      // the whole workgroup
        kr[u] = *(const u32x4*)row;
        v[u] = *(const u32x4*)(row + (int64_t)c.Hk * D);
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (OWN && u * W < items) q_do(qr[u]);
    if (!stored) return;                         // the whole workgroup
    const uint32_t before = *(const uint16_t*)(c.scales + at * 2);

    float k[U][8];
    uint32_t kt = 0, vmax = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (u * W + W <= slot0 || u * W >= slot1) continue;      // the whole workgroup
        const int slot = u * W + w, i = min(max(slot - slot0, 0), n - 1);
        widen8(kr[u], k[u]);
        if (a.k_weight) H::norm(k[u], a.k_weight, l, a.eps);
        if (a.rope) H::rotate(k[u], a.rope + min(p0 + i, (int64_t)a.P - 1) * a.R, a.R, a.interleaved, l);
        if (slot < slot0 || slot >= slot1) continue;
#pragma unroll
        for (int e = 0; e < 8; ++e) kt = max(kt, __float_as_uint(k[u][e]) & 0x7fffffffu);
#pragma unroll
        for (int e = 0; e < 4; ++e) vmax = max(vmax, max(v[u][e] << 16 & 0x7fffffffu, v[u][e] & 0x7fff0000u));
    }
#pragma unroll
    for (int off = 1; off < 64; off *= 2) {
        kt = max(kt, (uint32_t)__shfl_xor((int)kt, off, kWave));
        vmax = max(vmax, (uint32_t)__shfl_xor((int)vmax, off, kWave));
    }
    if (lane == 0) tops[threadIdx.x >> 6][0] = kt, tops[threadIdx.x >> 6][1] = vmax;
    __syncthreads();
    kt = max(max(tops[0][0], tops[1][0]), max(tops[2][0], tops[3][0]));
    vmax = max(max(tops[0][1], tops[1][1]), max(tops[2][1], tops[3][1]));
    // a block that holds older tokens keeps the larger scale
    const uint32_t ke0 = slot0 ? before & 255 : 0, ve0 = slot0 ? before >> 8 : 0;
    const uint32_t ke = max(cache_scale_byte(kt), ke0), ve = max(cache_scale_byte(vmax), ve0);
    uint8_t* const kc = c.k + at * T * D;
    uint8_t* const vc = c.v + at * T * D;
    if (slot0 && ke > ke0 && ke != 255)          // older codes to the new scale
        for (int i = threadIdx.x; i < slot0 * D / 4; i += 256) {
            uint32_t* p = (uint32_t*)kc + i;
            *p = cache_rescale4(*p, ke - ke0);
        }
    if (slot0 && ve > ve0 && ve != 255)
        for (int i = threadIdx.x; i < (slot0 + 15) / 16 * D * 4; i += 256) {   // four tokens of a group
            const int first = i / (4 * D) * 16 + i % 4 * 4, older = min(max(slot0 - first, 0), 4);
            const uint32_t mask = older == 4 ? ~0u : (1u << 8 * older) - 1;
            uint32_t* p = (uint32_t*)vc + i;
            if (older) *p = (cache_rescale4(*p, ve - ve0) & mask) | (*p & ~mask);
        }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (u * W + W <= slot0 || u * W >= slot1) continue;      // the whole workgroup
        const int slot = u * W + w;
        if (slot >= slot0 && slot < slot1) *(uint2*)(kc + (int64_t)slot * D + l * 8) = cache_codes8(k[u], ke);
        float x[8];
        widen8(v[u], x);
        const uint2 four = four_tokens(cache_codes8(x, ve));
        if (U * W > T && slot >= T) continue;
        uint32_t* const to = (uint32_t*)vt + ((slot >> 4) * D + l * 8 + 2 * (lane >> 4)) * 4 + (slot >> 2 & 3);
        to[0] = four.x;
        to[4] = four.y;
    }
    __syncthreads();                             // also: the older tokens' bytes before the new ones of the same words
    for (int i = threadIdx.x; i < T / 16 * D; i += 256) {
        const int lo = max(slot0 - (i / D) * 16, 0), hi = min(slot1 - (i / D) * 16, 16);   // new tokens of the sixteen
        if (lo >= hi) continue;
        if (hi - lo == 16) {
            *(u32x4*)(vc + (int64_t)i * 16) = vt[i];
        } else {
            for (int e = lo; e < hi; ++e) vc[(int64_t)i * 16 + e] = ((const uint8_t*)vt)[i * 16 + e];
        }
    }
    if (threadIdx.x == 0) *(uint16_t*)(c.scales + at * 2) = (uint16_t)(ke | ve << 8);
}

}  // namespace

hipError_t launch_qkv_append(const AppendArgs& a, const Sequences& s, const Cache& c, hipStream_t st) {
    const int64_t per_seq = append_per_seq(s.max_q, c.T);
    const int parts = append_parts(s.n, s.max_q, a.Hq / c.Hk, c.Hk, c.T, c.D);
    const unsigned grid = (unsigned)(s.n * per_seq * c.Hk * (parts + 1));
    const auto go = [&](auto kernel) {
        kernel<<<grid, 256, 0, st>>>(a, s, c, (int)per_seq, parts);
        return hipGetLastError();
    };
    const auto blocks = [&](auto d) {
        constexpr int D = decltype(d)::value;
        const auto own = [&](auto with, auto without) { return parts ? go(without) : go(with); };
        switch (c.T) {
            case 16: return own(k_qkv_append<D, 16, true>, k_qkv_append<D, 16, false>);
            case 32: return own(k_qkv_append<D, 32, true>, k_qkv_append<D, 32, false>);
            case 64: return own(k_qkv_append<D, 64, true>, k_qkv_append<D, 64, false>);
            default: return own(k_qkv_append<D, 128, true>, k_qkv_append<D, 128, false>);
        }
    };
    return c.D == 128 ? blocks(std::integral_constant<int, 128>{}) : blocks(std::integral_constant<int, 64>{});
}

}  // namespace awq
