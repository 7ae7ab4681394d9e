// C ABI of the 8-bit cache's operators (declared in include/awq.h): argument validation on the host, then launches on
// the caller's stream.  Nothing is allocated, freed or synchronized here.
#include <algorithm>
#include <cmath>

#include "../../include/awq.h"
#include "awq_cache.h"

namespace {

constexpr int64_t kIntMax = 0x7fffffff;
constexpr int kHeadsMax = 1024;
constexpr int64_t kTokensMax = (int64_t)1 << 30;         // width * T: positions stay far from 2^31
constexpr int64_t kThreadsMax = 0xffffffff;              // of a launch

bool aligned(const void* p, size_t a) { return (uintptr_t)p % a == 0; }
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && x < y + nb && y < x + na;
}
struct Range {
    const void* p;
    size_t n;
};
template <int NO, int NI>
bool disjoint(const Range (&out)[NO], const Range (&in)[NI]) {
    for (int o = 0; o < NO; ++o) {
        for (const Range& r : in)
            if (overlap(out[o].p, out[o].n, r.p, r.n)) return false;
        for (int q = o + 1; q < NO; ++q)
            if (overlap(out[o].p, out[o].n, out[q].p, out[q].n)) return false;
    }
    return true;
}
bool heads_ok(int64_t M, int32_t Hq, int32_t Hk, int32_t D) {
    return M > 0 && Hk > 0 && Hq > 0 && Hq <= kHeadsMax && Hq % Hk == 0 && D > 0 && D <= 1024 &&
           M <= ((int64_t)1 << 31) / ((int64_t)(Hq + 2 * Hk) * D);
}
bool sequences_ok(const int32_t* cu, const int32_t* length, const int32_t* table, int32_t n_seq, int32_t width,
                  int32_t max_q, int64_t T) {
    return cu && length && table && n_seq > 0 && width > 0 && max_q > 0 && width * T <= kTokensMax && aligned(cu, 4) &&
           aligned(length, 4) && aligned(table, 4);
}
bool cache_ok(const uint8_t* k, const uint8_t* v, const uint8_t* scales, int64_t blocks, int32_t Hk, int32_t T,
              int32_t D) {
    return k && v && scales && blocks > 0 && blocks <= kIntMax && blocks * T <= ((int64_t)1 << 42) / ((int64_t)Hk * D) &&
           aligned(k, 16) && aligned(v, 16) && aligned(scales, 2);
}
int log2_of(int32_t T) { return T == 16 ? 4 : T == 32 ? 5 : T == 64 ? 6 : T == 128 ? 7 : -1; }
size_t block_bytes(int64_t blocks, int32_t Hk, int32_t T, int32_t D) { return (size_t)blocks * Hk * T * D; }

}  // namespace

extern "C" {

int awq_qkv_append(const void* qkv_bf16, int64_t M, int32_t Hq, int32_t Hk, int32_t D, const void* q_weight_bf16,
                   const void* k_weight_bf16, float eps, const float* rope, int64_t P, int32_t R, int32_t interleaved,
                   const int32_t* cu, const int32_t* length, const int32_t* table, int32_t n_seq, int32_t width,
                   int32_t max_q, void* q_bf16, uint8_t* k_codes, uint8_t* v_codes, uint8_t* scales, int64_t blocks,
                   int32_t T, void* stream) {
    if (!qkv_bf16 || !q_bf16 || !heads_ok(M, Hq, Hk, D)) return AWQ_ERR_INVALID_ARG;
    if ((D != 64 && D != 128) || log2_of(T) < 0) return AWQ_ERR_UNSUPPORTED;
    if (!sequences_ok(cu, length, table, n_seq, width, max_q, T) || !cache_ok(k_codes, v_codes, scales, blocks, Hk, T, D))
        return AWQ_ERR_INVALID_ARG;
    if ((q_weight_bf16 || k_weight_bf16) && !(eps > 0.f && eps <= 1.f)) return AWQ_ERR_INVALID_ARG;   // NaN fails too
    if (rope && (P <= 0 || P > kIntMax || R <= 0 || R % 16 != 0 || R > D || (interleaved != 0 && interleaved != 1)))
        return AWQ_ERR_INVALID_ARG;
    if (!aligned(qkv_bf16, 16) || !aligned(q_weight_bf16, 16) || !aligned(k_weight_bf16, 16) || !aligned(rope, 16) ||
        !aligned(q_bf16, 16))
        return AWQ_ERR_INVALID_ARG;
    const int32_t most = (int32_t)std::min<int64_t>(max_q, M);
    const int64_t each = (int64_t)Hk * (awq::append_parts(n_seq, most, Hq / Hk, Hk, T, D) + 1);
    if (n_seq * awq::append_per_seq(most, T) > kThreadsMax / 256 / each) return AWQ_ERR_INVALID_ARG;
    const size_t row = (size_t)M * D * 2, kv = block_bytes(blocks, Hk, T, D);
    const Range out[] = {{q_bf16, row * Hq}, {k_codes, kv}, {v_codes, kv}, {scales, (size_t)blocks * Hk * 2}};
    const Range in[] = {{qkv_bf16, row * (Hq + 2 * Hk)}, {q_weight_bf16, (size_t)D * 2}, {k_weight_bf16, (size_t)D * 2},
                        {rope, rope ? (size_t)P * R * 4 : 0}, {cu, ((size_t)n_seq + 1) * 4}, {length, (size_t)n_seq * 4},
                        {table, (size_t)n_seq * width * 4}};
    if (!disjoint(out, in)) return AWQ_ERR_INVALID_ARG;
    const awq::AppendArgs a{(const uint16_t*)qkv_bf16, (const uint16_t*)q_weight_bf16, (const uint16_t*)k_weight_bf16,
                            rope, (uint16_t*)q_bf16, M, Hq, (int)P, R, interleaved, (double)eps};
    const awq::Sequences s{cu, length, table, n_seq, width, most};
    const awq::Cache c{k_codes, v_codes, scales, blocks, Hk, D, T, log2_of(T)};
    return awq::record_hip(awq::launch_qkv_append(a, s, c, (hipStream_t)stream));
}

size_t awq_attention_workspace_size(int64_t M, int32_t n_seq, int32_t max_q, int32_t Hq, int32_t Hk, int32_t D) {
    if (!heads_ok(M, Hq, Hk, D) || n_seq <= 0 || max_q <= 0 || (D != 64 && D != 128)) return 0;
    return awq::plan_attention(M, n_seq, max_q, Hq, Hk, D, 1).ws_bytes;
}

int awq_attention(const void* q_bf16, int64_t M, int32_t Hq, int32_t Hk, int32_t D, const int32_t* cu,
                  const int32_t* length, const int32_t* table, int32_t n_seq, int32_t width, int32_t max_q,
                  const uint8_t* k_codes, const uint8_t* v_codes, const uint8_t* scales, int64_t blocks, int32_t T,
                  float scale, int32_t causal, void* out_bf16, void* workspace, size_t ws_bytes, void* stream) {
    if (!q_bf16 || !out_bf16 || !heads_ok(M, Hq, Hk, D)) return AWQ_ERR_INVALID_ARG;
    if ((D != 64 && D != 128) || log2_of(T) < 0) return AWQ_ERR_UNSUPPORTED;
    if (!sequences_ok(cu, length, table, n_seq, width, max_q, T) || !cache_ok(k_codes, v_codes, scales, blocks, Hk, T, D))
        return AWQ_ERR_INVALID_ARG;
    if (!std::isfinite(scale * awq::kLog2e) || (causal != 0 && causal != 1)) return AWQ_ERR_INVALID_ARG;
    if (!aligned(q_bf16, 16) || !aligned(out_bf16, 16)) return AWQ_ERR_INVALID_ARG;
    const awq::AttentionPlan p = awq::plan_attention(M, n_seq, max_q, Hq, Hk, D, (int64_t)width * T);
    if ((int64_t)n_seq * p.tiles > kThreadsMax / awq::attention_threads(p) / ((int64_t)p.split * Hk)) return AWQ_ERR_INVALID_ARG;
    if (ws_bytes < p.ws_bytes || (p.ws_bytes && !workspace)) return AWQ_ERR_WORKSPACE;
    if (p.ws_bytes && !aligned(workspace, 256)) return AWQ_ERR_INVALID_ARG;
    const size_t row = (size_t)M * Hq * D * 2, kv = block_bytes(blocks, Hk, T, D);
    const Range out[] = {{out_bf16, row}, {p.ws_bytes ? workspace : nullptr, p.ws_bytes}};
    const Range in[] = {{q_bf16, row}, {k_codes, kv}, {v_codes, kv}, {scales, (size_t)blocks * Hk * 2},
                        {cu, ((size_t)n_seq + 1) * 4}, {length, (size_t)n_seq * 4}, {table, (size_t)n_seq * width * 4}};
    if (!disjoint(out, in)) return AWQ_ERR_INVALID_ARG;
    const awq::Sequences s{cu, length, table, n_seq, width, max_q};
    const awq::Cache c{(uint8_t*)k_codes, (uint8_t*)v_codes, (uint8_t*)scales, blocks, Hk, D, T, log2_of(T)};
    return awq::record_hip(awq::launch_attention((const uint16_t*)q_bf16, M, Hq, s, c, scale, causal,
                                                 (uint16_t*)out_bf16, p.ws_bytes ? workspace : nullptr, p,
                                                 (hipStream_t)stream));
}

}  // extern "C"
