// Host-side argument handling of the microscaled operators under AddressSanitizer and
// UndefinedBehaviorSanitizer (built by tests/test_mx_host_sanitizers.py; needs no GPU).  Every call below
// is rejected on the host before anything is enqueued: the "device" pointers are host canary buffers that
// must come back unchanged.  The size queries and the product's plan are also driven over extreme and many
// ordinary sizes, where an overflow in their arithmetic would be undefined behaviour.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <limits>
#include <vector>

#include "../include/awq.h"

static int failures = 0;
#define EXPECT(cond)                                                        \
    do {                                                                    \
        if (!(cond)) {                                                      \
            std::fprintf(stderr, "FAILED line %d: %s\n", __LINE__, #cond); \
            ++failures;                                                     \
        }                                                                   \
    } while (0)

namespace {
constexpr size_t kCanary = 1 << 16;
struct Canary {
    std::vector<unsigned char> b;
    Canary() : b(kCanary + 256, 0xA5) {}
    uint8_t* p() { return (uint8_t*)(((uintptr_t)b.data() + 255) & ~(uintptr_t)255); }   // 256-byte aligned
    bool intact() const {
        for (unsigned char c : b)
            if (c != 0xA5) return false;
        return true;
    }
};
}  // namespace

int main() {
    Canary a, b, c, d, e, w;
    uint8_t* const odd = a.p() + 2;
    float* const s = (float*)e.p();
    const size_t big = (size_t)1 << 40;
    const int64_t top = std::numeric_limits<int64_t>::max(), low = std::numeric_limits<int64_t>::min();

    // ---- sizes that no dimension may have
    for (int64_t v : {top, low, top / 2, (int64_t)1 << 62, (int64_t)1 << 40, (int64_t)1 << 32, (int64_t)0, (int64_t)-1,
                      (int64_t)-32}) {
        EXPECT(awq_mx_codes_bytes(v, 64) == 0 && awq_mx_codes_bytes(64, v) == 0);
        EXPECT(awq_mx_scales_bytes(v, 64) == 0 && awq_mx_scales_bytes(64, v) == 0);
        EXPECT(awq_mx_gemm_workspace_size(v, 64, 64, 8) == 0 && awq_mx_gemm_workspace_size(8, v, 64, 8) == 0 &&
               awq_mx_gemm_workspace_size(8, 64, v, 4) == 0);
        EXPECT(awq_mx_pack(a.p(), v, 64, nullptr, b.p(), c.p(), nullptr) == AWQ_ERR_INVALID_ARG);
        EXPECT(awq_mx_pack(a.p(), 64, v, nullptr, b.p(), c.p(), nullptr) == AWQ_ERR_INVALID_ARG);
        EXPECT(awq_mx_unpack(b.p(), c.p(), v, 64, nullptr, a.p(), nullptr) == AWQ_ERR_INVALID_ARG);
        EXPECT(awq_mx_unpack(b.p(), c.p(), 64, v, nullptr, a.p(), nullptr) == AWQ_ERR_INVALID_ARG);
        EXPECT(awq_mx_quantize(a.p(), nullptr, v, 64, nullptr, 8, b.p(), c.p(), nullptr) == AWQ_ERR_INVALID_ARG);
        EXPECT(awq_mx_quantize(a.p(), nullptr, 8, v, nullptr, 8, b.p(), c.p(), nullptr) == AWQ_ERR_INVALID_ARG);
        EXPECT(awq_rms_norm(a.p(), nullptr, b.p(), v, 64, 1e-5f, nullptr, c.p(), nullptr, 8, nullptr, nullptr,
                            nullptr) == AWQ_ERR_INVALID_ARG);
        EXPECT(awq_rms_norm(a.p(), nullptr, b.p(), 8, v, 1e-5f, nullptr, c.p(), nullptr, 8, nullptr, nullptr,
                            nullptr) == AWQ_ERR_INVALID_ARG);
        EXPECT(awq_mx_gemm(a.p(), b.p(), 8, v, c.p(), d.p(), 64, 64, e.p(), w.p(), big, nullptr) == AWQ_ERR_INVALID_ARG);
        EXPECT(awq_mx_gemm(a.p(), b.p(), 8, 8, c.p(), d.p(), v, 64, e.p(), w.p(), big, nullptr) == AWQ_ERR_INVALID_ARG);
        EXPECT(awq_mx_gemm(a.p(), b.p(), 8, 8, c.p(), d.p(), 64, v, e.p(), w.p(), big, nullptr) == AWQ_ERR_INVALID_ARG);
    }

    // ---- missing, misaligned and overlapping buffers, parameters out of range
    EXPECT(awq_mx_pack(nullptr, 64, 64, nullptr, b.p(), c.p(), nullptr) == AWQ_ERR_INVALID_ARG);
    EXPECT(awq_mx_pack(a.p(), 48, 64, nullptr, b.p(), c.p(), nullptr) == AWQ_ERR_INVALID_ARG);
    EXPECT(awq_mx_pack(a.p(), 64, 64, nullptr, odd, c.p(), nullptr) == AWQ_ERR_INVALID_ARG);
    EXPECT(awq_mx_pack(a.p(), 64, 64, (float*)odd, b.p(), c.p(), nullptr) == AWQ_ERR_INVALID_ARG);
    EXPECT(awq_mx_pack(a.p(), 64, 64, nullptr, a.p() + 64, c.p(), nullptr) == AWQ_ERR_INVALID_ARG);
    EXPECT(awq_mx_unpack(b.p(), b.p() + 16, 64, 64, nullptr, b.p() + 64, nullptr) == AWQ_ERR_INVALID_ARG);
    EXPECT(awq_mx_quantize(a.p(), nullptr, 4, 64, nullptr, 6, b.p(), c.p(), nullptr) == AWQ_ERR_UNSUPPORTED);
    EXPECT(awq_mx_quantize(odd, nullptr, 4, 64, nullptr, 8, b.p(), c.p(), nullptr) == AWQ_ERR_INVALID_ARG);
    EXPECT(awq_mx_quantize(a.p(), nullptr, 4, 64, nullptr, 8, b.p(), b.p() + 16, nullptr) == AWQ_ERR_INVALID_ARG);
    for (float eps : {0.f, -1.f, 2.f, (float)NAN, (float)INFINITY})
        EXPECT(awq_rms_norm(a.p(), nullptr, b.p(), 2, 64, eps, nullptr, c.p(), nullptr, 8, nullptr, nullptr, nullptr) ==
               AWQ_ERR_INVALID_ARG);
    EXPECT(awq_rms_norm(a.p(), nullptr, b.p(), 2, 64, 1e-5f, c.p(), d.p(), nullptr, 8, nullptr, nullptr, nullptr) ==
           AWQ_ERR_INVALID_ARG);                 // an updated residual without a residual
    EXPECT(awq_rms_norm(a.p(), nullptr, b.p(), 2, 64, 1e-5f, nullptr, a.p() + 16, nullptr, 8, nullptr, nullptr,
                        nullptr) == AWQ_ERR_INVALID_ARG);
    EXPECT(awq_rms_norm(a.p(), nullptr, b.p(), 2, 64, 1e-5f, nullptr, nullptr, s, 5, c.p(), d.p(), nullptr) ==
           AWQ_ERR_UNSUPPORTED);
    EXPECT(awq_rms_norm(a.p(), nullptr, b.p(), 2, 40, 1e-5f, nullptr, nullptr, s, 8, c.p(), d.p(), nullptr) ==
           AWQ_ERR_INVALID_ARG);
    EXPECT(awq_mx_gemm(a.p(), b.p(), 8, 8, c.p(), d.p(), 64, 12, e.p(), w.p(), big, nullptr) == AWQ_ERR_INVALID_ARG);
    EXPECT(awq_mx_gemm(a.p(), b.p(), 7, 8, c.p(), d.p(), 64, 16, e.p(), w.p(), big, nullptr) == AWQ_ERR_UNSUPPORTED);
    EXPECT(awq_mx_gemm(odd, b.p(), 8, 8, c.p(), d.p(), 64, 16, e.p(), w.p(), big, nullptr) == AWQ_ERR_INVALID_ARG);
    EXPECT(awq_mx_gemm(a.p(), b.p(), 8, 8, c.p(), d.p(), 64, 16, a.p(), w.p(), big, nullptr) == AWQ_ERR_INVALID_ARG);
    const size_t need = awq_mx_gemm_workspace_size(8, 32768, 64, 8);
    EXPECT(need > 65536);
    EXPECT(awq_mx_gemm(a.p(), b.p(), 8, 8, c.p(), d.p(), 32768, 64, e.p(), w.p(), need - 1, nullptr) == AWQ_ERR_WORKSPACE);
    EXPECT(awq_mx_gemm(a.p(), b.p(), 8, 8, c.p(), d.p(), 32768, 64, e.p(), nullptr, big, nullptr) == AWQ_ERR_WORKSPACE);
    EXPECT(awq_mx_gemm(a.p(), b.p(), 8, 8, c.p(), d.p(), 32768, 64, e.p(), w.p() + 16, big, nullptr) == AWQ_ERR_INVALID_ARG);

    // ---- the plan over the whole range: a workspace of zero, or the counters and less than 1 GiB of partials
    const int64_t Ms[] = {1, 2, 16, 17, 33, 64, 65, 257, 4096, 65536, 65535 * 16};
    const int64_t Ks[] = {32, 96, 128, 160, 4096, 28672, 1 << 20, (int64_t)65535 * 128};
    const int64_t Ns[] = {8, 16, 72, 256, 264, 4096, 28672, 1 << 20, 4194304};
    for (int64_t M : Ms)
        for (int64_t K : Ks)
            for (int64_t N : Ns)
                for (int bits : {8, 4}) {
                    const size_t ws = awq_mx_gemm_workspace_size(M, K, N, bits);
                    EXPECT(ws == 0 || (ws > 65536 && ws < (size_t)1 << 30));
                }
    for (Canary* q : {&a, &b, &c, &d, &e, &w}) EXPECT(q->intact());
    std::printf("%d failures\n", failures);
    return failures != 0;
}
