// C ABI of the 8-bit operators with scales for groups of 128 (declared in include/awq.h): argument validation on
// the host, then launches on the caller's stream.  Nothing is allocated, freed or synchronized here.
#include "../../include/awq.h"
#include "awq_fp8.h"

namespace {

constexpr int64_t kIntMax = 0x7fffffff;
constexpr int64_t kRowsMax = (int64_t)65535 * 16;        // M of the product
constexpr int64_t kColsMax = 4194304;                    // N of the product (32-bit offsets of a row tile of Y)
constexpr int64_t kWeightMax = (int64_t)1 << 36;         // K * N of packed weights

bool aligned(const void* p, size_t a) { return (uintptr_t)p % a == 0; }
bool in_range(int64_t v) { return v > 0 && v <= kIntMax; }
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && x < y + nb && y < x + na;
}
bool weights_ok(int64_t K, int64_t N) {
    return in_range(K) && in_range(N) && K % 16 == 0 && K <= (int64_t)65535 * awq::kFp8Group && K * N <= kWeightMax;
}
bool rows_ok(int64_t M, int64_t K) {
    return in_range(M) && in_range(K) && K % 16 == 0 && M * K <= ((int64_t)1 << 40);
}
size_t acts_scales(int64_t M, int64_t K) { return (size_t)M * awq::fp8_kc(K) * 4; }

}  // namespace

extern "C" {

size_t awq_fp8_codes_bytes(int64_t K, int64_t N) { return weights_ok(K, N) ? awq::fp8_codes_bytes(K, N) : 0; }
size_t awq_fp8_scales_count(int64_t K, int64_t N) { return weights_ok(K, N) ? awq::fp8_scales_count(K, N) : 0; }

int awq_fp8_pack(const void* W_bf16, int64_t K, int64_t N, uint8_t* codes, float* scales, void* stream) {
    if (!W_bf16 || !codes || !scales || !weights_ok(K, N)) return AWQ_ERR_INVALID_ARG;
    if (!aligned(W_bf16, 2) || !aligned(codes, 16) || !aligned(scales, 4)) return AWQ_ERR_INVALID_ARG;
    const size_t nw = (size_t)K * N * 2, nc = awq::fp8_codes_bytes(K, N), ns = awq::fp8_scales_count(K, N) * 4;
    if (overlap(codes, nc, W_bf16, nw) || overlap(scales, ns, W_bf16, nw) || overlap(codes, nc, scales, ns))
        return AWQ_ERR_INVALID_ARG;
    return awq::record_hip(awq::launch_fp8_pack((const uint16_t*)W_bf16, K, N, codes, scales, (hipStream_t)stream));
}

int awq_fp8_quantize(const void* X_bf16, const void* gate_bf16, int64_t M, int64_t K, uint8_t* codes, float* scales,
                     void* stream) {
    if (!X_bf16 || !codes || !scales || !rows_ok(M, K)) return AWQ_ERR_INVALID_ARG;
    if (!aligned(X_bf16, 16) || !aligned(gate_bf16, 16) || !aligned(codes, 16) || !aligned(scales, 4))
        return AWQ_ERR_INVALID_ARG;
    const size_t nx = (size_t)M * K * 2, nc = (size_t)M * K, ns = acts_scales(M, K);
    for (const void* in : {X_bf16, gate_bf16})
        if (overlap(codes, nc, in, nx) || overlap(scales, ns, in, nx)) return AWQ_ERR_INVALID_ARG;
    if (overlap(codes, nc, scales, ns)) return AWQ_ERR_INVALID_ARG;
    return awq::record_hip(awq::launch_fp8_quantize((const uint16_t*)X_bf16, (const uint16_t*)gate_bf16, M, K, codes,
                                                    scales, (hipStream_t)stream));
}

size_t awq_fp8_gemm_workspace_size(int64_t M, int64_t K, int64_t N) {
    if (!rows_ok(M, K) || M > kRowsMax || !weights_ok(K, N) || N > kColsMax) return 0;
    return awq::plan_fp8_gemm(M, K, N).ws_bytes;
}

int awq_fp8_gemm(const uint8_t* xcodes, const float* xscales, int64_t M, const uint8_t* codes, const float* scales,
                 int64_t K, int64_t N, void* Y_bf16, void* workspace, size_t ws_bytes, void* stream) {
    if (!xcodes || !xscales || !codes || !scales || !Y_bf16) return AWQ_ERR_INVALID_ARG;
    if (!rows_ok(M, K) || M > kRowsMax || !weights_ok(K, N) || N > kColsMax || N % 8 != 0) return AWQ_ERR_INVALID_ARG;
    if (!aligned(xcodes, 16) || !aligned(xscales, 4) || !aligned(codes, 16) || !aligned(scales, 4) ||
        !aligned(Y_bf16, 16))
        return AWQ_ERR_INVALID_ARG;
    const awq::Fp8GemmPlan p = awq::plan_fp8_gemm(M, K, N);
    if (ws_bytes < p.ws_bytes || (p.ws_bytes && !workspace)) return AWQ_ERR_WORKSPACE;
    if (p.ws_bytes && !aligned(workspace, 256)) return AWQ_ERR_INVALID_ARG;
    const size_t ny = (size_t)M * N * 2;
    void* const ws = p.ws_bytes ? workspace : nullptr;
    struct Range { const void* p; size_t n; };
    const Range in[] = {{xcodes, (size_t)M * K}, {xscales, acts_scales(M, K)}, {codes, awq::fp8_codes_bytes(K, N)},
                        {scales, awq::fp8_scales_count(K, N) * 4}};
    for (const Range& r : in)
        if (overlap(Y_bf16, ny, r.p, r.n) || overlap(ws, p.ws_bytes, r.p, r.n)) return AWQ_ERR_INVALID_ARG;
    if (overlap(ws, p.ws_bytes, Y_bf16, ny)) return AWQ_ERR_INVALID_ARG;
    return awq::record_hip(awq::launch_fp8_gemm(xcodes, xscales, M, codes, scales, K, N, (uint16_t*)Y_bf16, ws, p,
                                                (hipStream_t)stream));
}

}  // extern "C"
