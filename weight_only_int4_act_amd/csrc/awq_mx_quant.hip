// Activations into MX blocks: the quantizer (with an optional gate) and the root-mean-square norm.
#include <algorithm>

#include "awq_mx.h"

namespace awq {
namespace {

__device__ __forceinline__ u32x4 pack_bf16x8(const float (&v)[8]) {
    return u32x4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])};
}

// ---------------------------------------------------------------- quantizer
// p = x, or x g / (1 + e^-g), divided by s per channel.  Bound by HBM: 2 (4 with a gate) bytes read and
// 1.03 or 0.53 written per element; 8192 x 11008 with a gate, 8 bits, takes 83 us (5.4 TB/s), and
// 16 x 28672 2.4 us, of which a launch is 2.  A workgroup takes 64 octets of channels (512) and 4 R rows; a
// wavefront walks its R rows with the reciprocals of s in registers, two rows' loads in flight.
// Four consecutive lanes hold a block.
constexpr int kRowsInFlight = 2;

template <int BITS, bool GATE, bool SCALED>
__global__ __launch_bounds__(256) void k_mx_quantize(const uint16_t* __restrict__ X,
                                                     const uint16_t* __restrict__ gate, int64_t M, int64_t K,
                                                     const float* __restrict__ s, uint8_t* __restrict__ codes,
                                                     uint8_t* __restrict__ scales, int R) {
    const int64_t oct = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63);
    if (oct >= K / 8) return;                    // K / 8 is a multiple of 4: a block's four lanes leave together
    const int64_t m0 = ((int64_t)blockIdx.y * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6)) * R;
    const int64_t m1 = min(m0 + R, M);
    double sr[8];
    if constexpr (SCALED) {
#pragma unroll
        for (int i = 0; i < 8; ++i) sr[i] = mx_recip64(s[oct * 8 + i]);
    }
    for (int64_t m = m0; m < m1; m += kRowsInFlight) {
        u32x4 xv[kRowsInFlight], gv[kRowsInFlight];
#pragma unroll
        for (int u = 0; u < kRowsInFlight; ++u) {
            const int64_t row = min(m + u, m1 - 1);      // past the last row: it again, not stored
            xv[u] = *(const u32x4*)(X + row * K + oct * 8);
            if constexpr (GATE) gv[u] = *(const u32x4*)(gate + row * K + oct * 8);
        }
#pragma unroll
        for (int u = 0; u < kRowsInFlight; ++u) {
            if (m + u >= m1) break;
            float x[8];
            bf16x8_to_f32(xv[u], x);
            if constexpr (GATE) {
                float g[8];
                bf16x8_to_f32(gv[u], g);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    // e^-g as a power of two; where it overflows the factor is zero
                    const float e = __builtin_amdgcn_exp2f(g[i] * -1.44269504f);
                    x[i] *= g[i] * __builtin_amdgcn_rcpf(1.f + e);
                }
            }
            if constexpr (SCALED) {
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = mx_div(x[i], sr[i]);
            }
            mx_store8<BITS>(x, codes + (m + u) * (BITS == 8 ? K : K / 2), scales + (m + u) * (K / kMxBlock), oct);
        }
    }
}

// ---------------------------------------------------------------- root-mean-square norm
// h = x + r, y = h * rsqrt(mean h^2 + eps) * weight; the codes hold y / s, the float32 quotient that the quantizer
// forms of the same y.  It is a true division: y and s share no exponent (weight / s may overflow where
// y / s does not), and a divisor serves one element, so that a reciprocal of its own costs as much (one row of 8192 with s:
// 3.4 us, by 53-bit reciprocals 3.4; 4096 x 8192 50.7 and 54.4).  One pass over the row: T
// threads of a row keep it in registers (U octets of channels each).  The squares are summed in
// float64, so that no finite row overflows and the rounding is that of the result, in one fixed order:
// thread, lanes, wavefronts.  Bound by HBM for many rows (7 bytes per element with the residual and 8-bit codes):
// 4096 x 8192 takes 44 us (5.3 TB/s), 51 with s.  For few by the trip to memory and the sum: one row of 8192
// 2.7 us, where a kernel that read the row twice took 6.3.

// The sum over a wavefront, in every lane: within rows of 16 lanes and then across them.
__device__ __forceinline__ double wave_sum_f64(double v) {
    auto add = [&](auto move) {
        const uint64_t b = __builtin_bit_cast(uint64_t, v);
        const uint64_t o = (uint64_t)(uint32_t)move((int)(uint32_t)b) | ((uint64_t)(uint32_t)move((int)(uint32_t)(b >> 32)) << 32);
        v += __builtin_bit_cast(double, o);
    };
    add([](int x) { return __builtin_amdgcn_mov_dpp(x, 0xB1, 0xf, 0xf, true); });    // lanes 1 0 3 2
    add([](int x) { return __builtin_amdgcn_mov_dpp(x, 0x4E, 0xf, 0xf, true); });    // lanes 2 3 0 1
    add([](int x) { return __builtin_amdgcn_mov_dpp(x, 0x141, 0xf, 0xf, true); });   // mirrored within 8
    add([](int x) { return __builtin_amdgcn_mov_dpp(x, 0x140, 0xf, 0xf, true); });   // mirrored within 16
    add([](int x) { return __shfl_xor(x, 16, kWave); });
    add([](int x) { return __shfl_xor(x, 32, kWave); });
    return v;
}

// 1 / sqrt(x) to float32: the hardware's approximation and one Newton step in float64.
__device__ __forceinline__ float rsqrt_f64(double x) {
    const double y = __builtin_amdgcn_rsq(x);
    return (float)(x < __builtin_inf() ? y * (1.5 - 0.5 * x * y * y) : y);           // infinity: 0; NaN: NaN
}

struct NormArgs {
    const uint16_t *X, *residual, *weight;
    int64_t M, K;
    double eps, inv_k;
    uint16_t *residual_out, *Y;
    const float* s;
    int bits;
    uint8_t *codes, *scales;
};

// the weights and divisors of one octet
template <bool SCALED>
struct NormCols {
    u32x4 w;
    floatx4 s[SCALED ? 2 : 1];
    __device__ __forceinline__ void load(const NormArgs& a, int64_t oct) {
        w = *(const u32x4*)(a.weight + oct * 8);
        if constexpr (SCALED) s[0] = *(const floatx4*)(a.s + oct * 8), s[1] = *(const floatx4*)(a.s + oct * 8 + 4);
    }
    // In registers from here on: behind a store, the wait for these loads would be one for the store, too.
    __device__ __forceinline__ void arrive() {
        asm volatile("" : "+v"(w));
        if constexpr (SCALED) asm volatile("" : "+v"(s[0]), "+v"(s[1]));
    }
};

// the outputs of one octet: h, y, and the codes of y or of the float32 quotient y / s that the quantizer forms
template <bool SCALED>
__device__ __forceinline__ void norm_store(const NormArgs& a, int64_t m, int64_t oct, const float (&h)[8], float rstd,
                                           const NormCols<SCALED>& cols) {
    const int64_t at = m * a.K + oct * 8;
    if (a.residual_out) *(u32x4*)(a.residual_out + at) = pack_bf16x8(h);
    float w[8], y[8];
    bf16x8_to_f32(cols.w, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = h[i] * rstd * w[i];
    if (a.Y) *(u32x4*)(a.Y + at) = pack_bf16x8(y);
    if (!a.codes) return;
    if constexpr (SCALED) {
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] /= cols.s[i / 4][i % 4];
    }
    if (a.bits == 8) mx_store8<8>(y, a.codes + m * a.K, a.scales + m * (a.K / kMxBlock), oct);
    else mx_store8<4>(y, a.codes + m * (a.K / 2), a.scales + m * (a.K / kMxBlock), oct);
}
__device__ __forceinline__ void norm_load(const NormArgs& a, int64_t m, int64_t oct, u32x4& x, u32x4& r) {
    x = *(const u32x4*)(a.X + m * a.K + oct * 8);
    r = a.residual ? *(const u32x4*)(a.residual + m * a.K + oct * 8) : u32x4{0, 0, 0, 0};
}
__device__ __forceinline__ double norm_square(const NormArgs& a, const u32x4& x, const u32x4& r, float (&h)[8]) {
    float t[8];
    bf16x8_to_f32(x, h);
    bf16x8_to_f32(r, t);
    double sum = 0.;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (a.residual) h[i] += t[i];
        sum += (double)h[i] * (double)h[i];
    }
    return sum;
}

// T threads per row (64 or more), U octets per thread, max(1, 256 / T) rows per workgroup.
template <int T, int U, bool SCALED>
__global__ __launch_bounds__(T < 256 ? 256 : T) void k_rms_norm(NormArgs a) {
    constexpr int kRows = T < 256 ? 256 / T : 1, NW = T / 64;
    __shared__ double part[NW];
    lds_poison_start(&part[0], NW);
    const int t = T < 256 ? threadIdx.x % T : threadIdx.x;
    const int64_t m = (int64_t)blockIdx.x * kRows + (T < 256 ? threadIdx.x / T : 0);
    if (T < 256 && m >= a.M) return;             // T = 64: whole wavefronts, no barrier below
    const int64_t octs = a.K / 8;
    u32x4 x[U], r[U];
    float h[U][8];
    NormCols<SCALED> cols[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t oct = min((int64_t)(u * T + t), octs - 1);
        norm_load(a, m, oct, x[u], r[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) cols[u].load(a, min((int64_t)(u * T + t), octs - 1));
    __builtin_amdgcn_sched_barrier(0);           // every load is on its way before the first is waited for
    double sum = 0.;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const double q = norm_square(a, x[u], r[u], h[u]);
        if (u * T + t < octs) sum += q;
    }
    sum = wave_sum_f64(sum);
#pragma unroll
    for (int u = 0; u < U; ++u) cols[u].arrive();
    if constexpr (NW > 1) {
        if ((t & 63) == 0) part[t >> 6] = sum;
        __syncthreads();
        sum = part[0];
#pragma unroll
        for (int i = 1; i < NW; ++i) sum += part[i];
    }
    const float rstd = rsqrt_f64(sum * a.inv_k + a.eps);
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (u * T + t < octs) norm_store(a, m, u * T + t, h[u], rstd, cols[u]);
}

// Rows of more than 32768 channels: a workgroup reads its row twice.
template <bool SCALED>
__global__ __launch_bounds__(1024) void k_rms_norm_long(NormArgs a) {
    __shared__ double part[16];
    lds_poison_start(&part[0], 16);
    const int64_t octs = a.K / 8, m = blockIdx.x;
    double sum = 0.;
    for (int64_t oct = threadIdx.x; oct < octs; oct += 1024) {
        u32x4 x, r;
        float h[8];
        norm_load(a, m, oct, x, r);
        sum += norm_square(a, x, r, h);
    }
    sum = wave_sum_f64(sum);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
    __syncthreads();
    sum = part[0];
    for (int i = 1; i < 16; ++i) sum += part[i];
    const float rstd = rsqrt_f64(sum * a.inv_k + a.eps);
    for (int64_t oct = threadIdx.x; oct < octs; oct += 1024) {
        u32x4 x, r;
        float h[8];
        NormCols<SCALED> cols;
        norm_load(a, m, oct, x, r);
        norm_square(a, x, r, h);
        cols.load(a, oct);
        norm_store(a, m, oct, h, rstd, cols);
    }
}

template <int T, int U>
hipError_t norm(const NormArgs& a, hipStream_t st) {
    constexpr int rows = T < 256 ? 256 / T : 1;
    const dim3 grid((unsigned)((a.M + rows - 1) / rows)), block(T < 256 ? 256 : T);
    if (a.s) k_rms_norm<T, U, true><<<grid, block, 0, st>>>(a);
    else k_rms_norm<T, U, false><<<grid, block, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_quantize(const uint16_t* X, const uint16_t* gate, int64_t M, int64_t K, const float* s, int bits,
                              uint8_t* codes, uint8_t* scales, hipStream_t st) {
    // Rows per wavefront (on inputs that no cache holds).  Two where a wavefront has reciprocals of s to share and one
    // row gives more than two workgroups per CU (4096 x 8192, 8 bits: 23.4 us, with one row 29.1; 8192 x 11008 with a gate: 93 and
    // 109; but 64 x 8192: 2.58 and 2.32), or lanes to spare (100000 x 96: 18.1 and 24.1); else one (4096 x 8192,
    // 8 bits, without s: 20.6 us, with two rows 21.9; 257 x 5120, 4 bits: 2.54 and 2.70; 8192 x 11008 with a gate: 83.1 and 85.6).
    const int64_t cols = (K / 8 + 63) / 64, quads = (M + 3) / 4;
    int R = (s || K < 512) && cols * quads > 2 * kNumXcd * kCusPerXcd ? 2 : 1;
    while ((quads + R - 1) / R > 65535) R *= 2;
    const dim3 grid((unsigned)cols, (unsigned)((quads + R - 1) / R));
    auto go = [&](auto kernel) {
        kernel<<<grid, 256, 0, st>>>(X, gate, M, K, s, codes, scales, R);
        return hipGetLastError();
    };
    if (bits == 8) {
        if (gate) return s ? go(k_mx_quantize<8, true, true>) : go(k_mx_quantize<8, true, false>);
        return s ? go(k_mx_quantize<8, false, true>) : go(k_mx_quantize<8, false, false>);
    }
    if (gate) return s ? go(k_mx_quantize<4, true, true>) : go(k_mx_quantize<4, true, false>);
    return s ? go(k_mx_quantize<4, false, true>) : go(k_mx_quantize<4, false, false>);
}

hipError_t launch_rms_norm(const uint16_t* X, const uint16_t* residual, const uint16_t* weight, int64_t M, int64_t K,
                           float eps, uint16_t* residual_out, uint16_t* Y, const float* s, int bits, uint8_t* codes,
                           uint8_t* scales, hipStream_t st) {
    const NormArgs a{X, residual, weight, M, K, (double)eps, 1. / (double)K, residual_out, Y, s, bits, codes, scales};
    const int64_t octs = K / 8;
    // As many threads as the row has octets, because the sum's chain of float64 additions grows with the
    // octets of a thread (2000 x 4096: 13.7 us with one octet, 13.9 with two); but two octets for 1024 once every CU has a
    // row, so that several rows share a CU (4096 x 8192: 43.5 us, with one octet 47.0, with four 44.4; 256 x 8192:
    // 5.65 us with one, 5.69 with two).  Longer rows take 1024 threads (4096 x 16384: 85.7 us with two octets, 87.1 with 512
    // threads and four).
    const bool few = M <= kNumXcd * kCusPerXcd;
    if (octs <= 64) return norm<64, 1>(a, st);
    if (octs <= 256) return norm<256, 1>(a, st);
    if (octs <= 512) return norm<512, 1>(a, st);
    if (octs <= 1024) return few ? norm<1024, 1>(a, st) : norm<512, 2>(a, st);
    if (octs <= 2048) return norm<1024, 2>(a, st);
    if (octs <= 4096) return norm<1024, 4>(a, st);
    if (a.s) k_rms_norm_long<true><<<(unsigned)M, 1024, 0, st>>>(a);
    else k_rms_norm_long<false><<<(unsigned)M, 1024, 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace awq
