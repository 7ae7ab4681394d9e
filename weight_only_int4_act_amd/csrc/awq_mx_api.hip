// C ABI of the microscaled operators (declared in include/awq.h): argument validation on the host,
// then launches on the caller's stream.  Nothing is allocated, freed or synchronized here.
#include "../../include/awq.h"
#include "awq_mx.h"

namespace {

constexpr int64_t kIntMax = 0x7fffffff;
constexpr int64_t kRowsMax = (int64_t)65535 * 16;        // M of the product
constexpr int64_t kNormRowsMax = 4194303;                // M of the norm: threads of one launch below 2^32
constexpr int64_t kColsMax = 4194304;                    // N of the product (32-bit offsets of a row tile of Y)
constexpr int64_t kWeightMax = (int64_t)1 << 36;         // K * N of packed weights

bool aligned(const void* p, size_t a) { return (uintptr_t)p % a == 0; }
bool in_range(int64_t v) { return v > 0 && v <= kIntMax; }
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && x < y + nb && y < x + na;
}

bool weights_ok(int64_t K, int64_t N) {
    return in_range(K) && in_range(N) && K % awq::kMxBlock == 0 && K <= (int64_t)65535 * awq::kMxChunk &&
           K * N <= kWeightMax;
}
bool rows_ok(int64_t M, int64_t K) {
    return in_range(M) && in_range(K) && K % awq::kMxBlock == 0 && M * K <= ((int64_t)1 << 40);
}

}  // namespace

extern "C" {

size_t awq_mx_codes_bytes(int64_t K, int64_t N) { return weights_ok(K, N) ? awq::mx_codes_bytes(K, N) : 0; }
size_t awq_mx_scales_bytes(int64_t K, int64_t N) { return weights_ok(K, N) ? awq::mx_scales_bytes(K, N) : 0; }

int awq_mx_pack(const void* W_bf16, int64_t K, int64_t N, const float* s, uint8_t* codes, uint8_t* scales,
                void* stream) {
    if (!W_bf16 || !codes || !scales || !weights_ok(K, N)) return AWQ_ERR_INVALID_ARG;
    if (!aligned(W_bf16, 2) || !aligned(s, 4) || !aligned(codes, 16) || !aligned(scales, 16))
        return AWQ_ERR_INVALID_ARG;
    const size_t nw = (size_t)K * N * 2, nc = awq::mx_codes_bytes(K, N), ns = awq::mx_scales_bytes(K, N);
    if (overlap(codes, nc, W_bf16, nw) || overlap(scales, ns, W_bf16, nw) || overlap(codes, nc, scales, ns) ||
        overlap(codes, nc, s, (size_t)K * 4) || overlap(scales, ns, s, (size_t)K * 4))
        return AWQ_ERR_INVALID_ARG;
    return awq::record_hip(
        awq::launch_mx_pack((const uint16_t*)W_bf16, K, N, s, codes, scales, (hipStream_t)stream));
}

int awq_mx_unpack(const uint8_t* codes, const uint8_t* scales, int64_t K, int64_t N, const float* s, void* W_bf16,
                  void* stream) {
    if (!W_bf16 || !codes || !scales || !weights_ok(K, N)) return AWQ_ERR_INVALID_ARG;
    if (!aligned(W_bf16, 2) || !aligned(s, 4) || !aligned(codes, 16) || !aligned(scales, 16))
        return AWQ_ERR_INVALID_ARG;
    const size_t nw = (size_t)K * N * 2;
    if (overlap(codes, awq::mx_codes_bytes(K, N), W_bf16, nw) ||
        overlap(scales, awq::mx_scales_bytes(K, N), W_bf16, nw) || overlap(s, (size_t)K * 4, W_bf16, nw))
        return AWQ_ERR_INVALID_ARG;
    return awq::record_hip(
        awq::launch_mx_unpack(codes, scales, K, N, s, (uint16_t*)W_bf16, (hipStream_t)stream));
}

int awq_mx_quantize(const void* X_bf16, const void* gate_bf16, int64_t M, int64_t K, const float* s, int32_t bits,
                    uint8_t* codes, uint8_t* scales, void* stream) {
    if (!X_bf16 || !codes || !scales || !rows_ok(M, K)) return AWQ_ERR_INVALID_ARG;
    if (bits != 8 && bits != 4) return AWQ_ERR_UNSUPPORTED;
    if (!aligned(X_bf16, 16) || !aligned(gate_bf16, 16) || !aligned(s, 16) || !aligned(codes, 16))
        return AWQ_ERR_INVALID_ARG;
    const size_t nx = (size_t)M * K * 2, nc = (size_t)M * K * bits / 8, ns = (size_t)M * K / awq::kMxBlock;
    for (const void* in : {X_bf16, gate_bf16})
        if (overlap(codes, nc, in, nx) || overlap(scales, ns, in, nx)) return AWQ_ERR_INVALID_ARG;
    if (overlap(codes, nc, scales, ns) || overlap(codes, nc, s, (size_t)K * 4) || overlap(scales, ns, s, (size_t)K * 4))
        return AWQ_ERR_INVALID_ARG;
    return awq::record_hip(awq::launch_mx_quantize((const uint16_t*)X_bf16, (const uint16_t*)gate_bf16, M, K, s, bits,
                                                   codes, scales, (hipStream_t)stream));
}

int awq_rms_norm(const void* X_bf16, const void* residual_bf16, const void* weight_bf16, int64_t M, int64_t K,
                 float eps, void* residual_out, void* Y_bf16, const float* s, int32_t bits, uint8_t* codes,
                 uint8_t* scales, void* stream) {
    if (!X_bf16 || !weight_bf16 || (!Y_bf16 && !codes) || !codes != !scales || (residual_out && !residual_bf16) ||
        (s && !codes))
        return AWQ_ERR_INVALID_ARG;
    if (!in_range(M) || M > kNormRowsMax || !in_range(K) || K % (codes ? awq::kMxBlock : 8) != 0 || M * K > ((int64_t)1 << 40))
        return AWQ_ERR_INVALID_ARG;
    if (!(eps > 0.f && eps <= 1.f)) return AWQ_ERR_INVALID_ARG;      // NaN fails too
    if (codes && bits != 8 && bits != 4) return AWQ_ERR_UNSUPPORTED;
    if (!aligned(X_bf16, 16) || !aligned(residual_bf16, 16) || !aligned(weight_bf16, 16) ||
        !aligned(residual_out, 16) || !aligned(Y_bf16, 16) || !aligned(s, 16) || !aligned(codes, 16))
        return AWQ_ERR_INVALID_ARG;
    // a bf16 output may take the place of X or of the residual (the same address); nothing else may overlap
    const size_t nx = (size_t)M * K * 2, nc = codes ? (size_t)M * K * bits / 8 : 0, ns = (size_t)M * K / awq::kMxBlock;
    struct Range { const void* p; size_t n; };
    const Range in[] = {{X_bf16, nx}, {residual_bf16, nx}, {weight_bf16, (size_t)K * 2}, {s, (size_t)K * 4}};
    const Range out[] = {{residual_out, nx}, {Y_bf16, nx}, {codes, nc}, {scales, ns}};
    for (int o = 0; o < 4; ++o) {
        for (int i = 0; i < 4; ++i)
            if (overlap(out[o].p, out[o].n, in[i].p, in[i].n) && !(o < 2 && i < 2 && out[o].p == in[i].p))
                return AWQ_ERR_INVALID_ARG;
        for (int q = o + 1; q < 4; ++q)
            if (overlap(out[o].p, out[o].n, out[q].p, out[q].n)) return AWQ_ERR_INVALID_ARG;
    }
    return awq::record_hip(awq::launch_rms_norm((const uint16_t*)X_bf16, (const uint16_t*)residual_bf16,
                                                (const uint16_t*)weight_bf16, M, K, eps, (uint16_t*)residual_out,
                                                (uint16_t*)Y_bf16, s, bits, codes, scales, (hipStream_t)stream));
}

size_t awq_mx_gemm_workspace_size(int64_t M, int64_t K, int64_t N, int32_t bits) {
    if (!rows_ok(M, K) || M > kRowsMax || !weights_ok(K, N) || N > kColsMax || (bits != 8 && bits != 4))
        return 0;
    return awq::plan_mx_gemm(M, K, N, bits).ws_bytes;
}

int awq_mx_gemm(const uint8_t* xcodes, const uint8_t* xscales, int32_t bits, int64_t M, const uint8_t* codes,
                const uint8_t* scales, int64_t K, int64_t N, void* Y_bf16, void* workspace, size_t ws_bytes,
                void* stream) {
    if (!xcodes || !xscales || !codes || !scales || !Y_bf16) return AWQ_ERR_INVALID_ARG;
    if (!rows_ok(M, K) || M > kRowsMax || !weights_ok(K, N) || N > kColsMax || N % 8 != 0)
        return AWQ_ERR_INVALID_ARG;
    if (bits != 8 && bits != 4) return AWQ_ERR_UNSUPPORTED;
    if (!aligned(xcodes, 16) || !aligned(codes, 16) || !aligned(scales, 16) || !aligned(Y_bf16, 16))
        return AWQ_ERR_INVALID_ARG;
    const awq::MxGemmPlan p = awq::plan_mx_gemm(M, K, N, bits);
    if (ws_bytes < p.ws_bytes || (p.ws_bytes && !workspace)) return AWQ_ERR_WORKSPACE;
    if (p.ws_bytes && !aligned(workspace, 256)) return AWQ_ERR_INVALID_ARG;
    const size_t ny = (size_t)M * N * 2;
    struct Range { const void* p; size_t n; };
    const Range in[] = {{xcodes, (size_t)M * K * bits / 8}, {xscales, (size_t)M * K / awq::kMxBlock},
                        {codes, awq::mx_codes_bytes(K, N)}, {scales, awq::mx_scales_bytes(K, N)}};
    for (const Range& r : in)
        if (overlap(Y_bf16, ny, r.p, r.n) || overlap(p.ws_bytes ? workspace : nullptr, p.ws_bytes, r.p, r.n))
            return AWQ_ERR_INVALID_ARG;
    if (overlap(p.ws_bytes ? workspace : nullptr, p.ws_bytes, Y_bf16, ny)) return AWQ_ERR_INVALID_ARG;
    return awq::record_hip(awq::launch_mx_gemm(xcodes, xscales, bits, M, codes, scales, K, N, (uint16_t*)Y_bf16,
                                               workspace, p, (hipStream_t)stream));
}

}  // extern "C"
