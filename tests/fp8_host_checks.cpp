// Host-side argument handling of the 8-bit operators under AddressSanitizer and UndefinedBehaviorSanitizer (built by
// tests/test_fp8_host_sanitizers.py; needs no GPU).  Every call below is rejected on the host before anything is
// enqueued: the "device" pointers are host canary buffers that must come back unchanged.  The size queries and the plans are
// also driven over extreme and many ordinary sizes, where an overflow in their arithmetic would be undefined behaviour.
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
Canary x, y, kc, vc, sc, cu, len, tab, rope, qw, w;

struct Append {
    int64_t M = 3;
    int32_t Hq = 8, Hk = 2, D = 64;
    float eps = 1e-5f;
    int64_t P = 16;
    int32_t R = 64, inter = 0, n = 2, width = 4, max_q = 3;
    int64_t blocks = 8;
    int32_t T = 16;
    const void *qkv = x.p(), *weight = qw.p();
    const float* turn = (const float*)rope.p();
    void* q = y.p();
    int run() const {
        return awq_qkv_append(qkv, M, Hq, Hk, D, weight, weight, eps, turn, P, R, inter, (int32_t*)cu.p(), (int32_t*)len.p(),
                              (int32_t*)tab.p(), n, width, max_q, q, kc.p(), vc.p(), sc.p(), blocks, T, nullptr);
    }
};
struct Attend {
    int64_t M = 3;
    int32_t Hq = 8, Hk = 2, D = 64, n = 2, width = 4, max_q = 3;
    int64_t blocks = 8;
    int32_t T = 16;
    float scale = .125f;
    int32_t causal = 1;
    const void* q = x.p();
    void *out = y.p(), *ws = w.p();
    size_t bytes = (size_t)1 << 40;
    int run() const {
        return awq_attention(q, M, Hq, Hk, D, (int32_t*)cu.p(), (int32_t*)len.p(), (int32_t*)tab.p(), n, width, max_q,
                             kc.p(), vc.p(), sc.p(), blocks, T, scale, causal, out, ws, bytes, nullptr);
    }
};
}  // namespace

#define REFUSED(type, member, value, status) \
    do {                                     \
        type t;                              \
        t.member = value;                    \
        EXPECT(t.run() == status);           \
    } while (0)

int main() {
    const int64_t top = std::numeric_limits<int64_t>::max(), low = std::numeric_limits<int64_t>::min();
    const int32_t itop = std::numeric_limits<int32_t>::max(), ilow = std::numeric_limits<int32_t>::min();
    const size_t big = (size_t)1 << 40;
    uint8_t* const odd = x.p() + 2;
    float* const s = (float*)sc.p();

    // ---- sizes that no dimension may have
    for (int64_t v : {top, low, top / 2, (int64_t)1 << 62, (int64_t)1 << 41, (int64_t)0, (int64_t)-1, (int64_t)-16}) {
        EXPECT(awq_fp8_codes_bytes(v, 64) == 0 && awq_fp8_codes_bytes(64, v) == 0);
        EXPECT(awq_fp8_scales_count(v, 64) == 0 && awq_fp8_scales_count(64, v) == 0);
        EXPECT(awq_fp8_gemm_workspace_size(v, 64, 64) == 0 && awq_fp8_gemm_workspace_size(8, v, 64) == 0 &&
               awq_fp8_gemm_workspace_size(8, 64, v) == 0);
        EXPECT(awq_attention_workspace_size(v, 2, 3, 8, 2, 64) == 0);
        EXPECT(awq_fp8_pack(x.p(), v, 64, y.p(), s, nullptr) == AWQ_ERR_INVALID_ARG);
        EXPECT(awq_fp8_pack(x.p(), 64, v, y.p(), s, nullptr) == AWQ_ERR_INVALID_ARG);
        EXPECT(awq_fp8_quantize(x.p(), nullptr, v, 64, y.p(), s, nullptr) == AWQ_ERR_INVALID_ARG);
        EXPECT(awq_fp8_quantize(x.p(), nullptr, 8, v, y.p(), s, nullptr) == AWQ_ERR_INVALID_ARG);
        EXPECT(awq_fp8_gemm(x.p(), s, v, kc.p(), s, 64, 64, y.p(), w.p(), big, nullptr) == AWQ_ERR_INVALID_ARG);
        EXPECT(awq_fp8_gemm(x.p(), s, 8, kc.p(), s, v, 64, y.p(), w.p(), big, nullptr) == AWQ_ERR_INVALID_ARG);
        EXPECT(awq_fp8_gemm(x.p(), s, 8, kc.p(), s, 64, v, y.p(), w.p(), big, nullptr) == AWQ_ERR_INVALID_ARG);
        REFUSED(Append, M, v, AWQ_ERR_INVALID_ARG);
        REFUSED(Append, P, v, AWQ_ERR_INVALID_ARG);
        REFUSED(Append, blocks, v, AWQ_ERR_INVALID_ARG);
        REFUSED(Attend, M, v, AWQ_ERR_INVALID_ARG);
        REFUSED(Attend, blocks, v, AWQ_ERR_INVALID_ARG);
    }
    for (int32_t v : {itop, ilow, 0, -1}) {
        REFUSED(Append, Hq, v, AWQ_ERR_INVALID_ARG);
        REFUSED(Append, Hk, v, AWQ_ERR_INVALID_ARG);
        REFUSED(Append, D, v, AWQ_ERR_INVALID_ARG);
        REFUSED(Append, R, v, AWQ_ERR_INVALID_ARG);
        REFUSED(Append, T, v, AWQ_ERR_UNSUPPORTED);
        REFUSED(Attend, Hq, v, AWQ_ERR_INVALID_ARG);
        REFUSED(Attend, Hk, v, AWQ_ERR_INVALID_ARG);
        REFUSED(Attend, D, v, AWQ_ERR_INVALID_ARG);
        REFUSED(Attend, T, v, AWQ_ERR_UNSUPPORTED);
        REFUSED(Append, width, v, AWQ_ERR_INVALID_ARG);
        REFUSED(Attend, width, v, AWQ_ERR_INVALID_ARG);
        REFUSED(Append, n, v, AWQ_ERR_INVALID_ARG);          // the largest: more threads than a launch has
        REFUSED(Attend, n, v, AWQ_ERR_INVALID_ARG);
        if (v <= 0) {
            REFUSED(Append, max_q, v, AWQ_ERR_INVALID_ARG);
            REFUSED(Attend, max_q, v, AWQ_ERR_INVALID_ARG);
        }
        EXPECT(awq_attention_workspace_size(3, v, 3, 8, 2, 64) == 0 && (v == itop || awq_attention_workspace_size(3, 2, v, 8, 2, 64) == 0));
        EXPECT(awq_attention_workspace_size(3, 2, 3, v, 2, 64) == 0 && awq_attention_workspace_size(3, 2, 3, 8, v, 64) == 0 &&
               awq_attention_workspace_size(3, 2, 3, 8, 2, v) == 0);
    }

    // ---- missing, misaligned and overlapping buffers, parameters out of range
    for (float eps : {0.f, -1.f, 2.f, (float)NAN, (float)INFINITY}) REFUSED(Append, eps, eps, AWQ_ERR_INVALID_ARG);
    for (float f : {(float)NAN, (float)INFINITY, -(float)INFINITY}) REFUSED(Attend, scale, f, AWQ_ERR_INVALID_ARG);
    REFUSED(Append, qkv, nullptr, AWQ_ERR_INVALID_ARG);
    REFUSED(Append, qkv, odd, AWQ_ERR_INVALID_ARG);
    REFUSED(Append, weight, odd, AWQ_ERR_INVALID_ARG);
    REFUSED(Append, turn, (const float*)odd, AWQ_ERR_INVALID_ARG);
    REFUSED(Append, q, nullptr, AWQ_ERR_INVALID_ARG);
    REFUSED(Append, q, x.p() + 16, AWQ_ERR_INVALID_ARG);
    REFUSED(Append, q, kc.p(), AWQ_ERR_INVALID_ARG);
    REFUSED(Append, q, rope.p(), AWQ_ERR_INVALID_ARG);
    REFUSED(Append, inter, 2, AWQ_ERR_INVALID_ARG);
    REFUSED(Append, R, 72, AWQ_ERR_INVALID_ARG);
    REFUSED(Append, D, 80, AWQ_ERR_UNSUPPORTED);
    REFUSED(Append, Hk, 3, AWQ_ERR_INVALID_ARG);
    REFUSED(Attend, causal, 2, AWQ_ERR_INVALID_ARG);
    REFUSED(Attend, q, odd, AWQ_ERR_INVALID_ARG);
    REFUSED(Attend, out, x.p(), AWQ_ERR_INVALID_ARG);
    REFUSED(Attend, out, tab.p(), AWQ_ERR_INVALID_ARG);
    REFUSED(Attend, ws, nullptr, AWQ_ERR_WORKSPACE);
    REFUSED(Attend, ws, w.p() + 16, AWQ_ERR_INVALID_ARG);
    const size_t part = awq_attention_workspace_size(3, 2, 3, 8, 2, 64);
    EXPECT(part > 65536);
    REFUSED(Attend, bytes, part - 1, AWQ_ERR_WORKSPACE);
    EXPECT(awq_fp8_pack(odd + 1, 64, 64, y.p(), s, nullptr) == AWQ_ERR_INVALID_ARG);
    EXPECT(awq_fp8_pack(x.p(), 64, 64, x.p() + 64, s, nullptr) == AWQ_ERR_INVALID_ARG);
    EXPECT(awq_fp8_quantize(x.p(), odd, 4, 64, y.p(), s, nullptr) == AWQ_ERR_INVALID_ARG);
    EXPECT(awq_fp8_quantize(x.p(), y.p(), 4, 64, y.p(), s, nullptr) == AWQ_ERR_INVALID_ARG);
    EXPECT(awq_fp8_gemm(x.p(), s, 8, kc.p(), s, 64, 12, y.p(), w.p(), big, nullptr) == AWQ_ERR_INVALID_ARG);
    EXPECT(awq_fp8_gemm(odd, s, 8, kc.p(), s, 64, 16, y.p(), w.p(), big, nullptr) == AWQ_ERR_INVALID_ARG);
    EXPECT(awq_fp8_gemm(x.p(), s, 8, kc.p(), s, 64, 16, sc.p(), w.p(), big, nullptr) == AWQ_ERR_INVALID_ARG);
    const size_t need = awq_fp8_gemm_workspace_size(8, 32768, 64);
    EXPECT(need > 65536);
    EXPECT(awq_fp8_gemm(x.p(), s, 8, kc.p(), s, 32768, 64, y.p(), w.p(), need - 1, nullptr) == AWQ_ERR_WORKSPACE);
    EXPECT(awq_fp8_gemm(x.p(), s, 8, kc.p(), s, 32768, 64, y.p(), nullptr, big, nullptr) == AWQ_ERR_WORKSPACE);
    EXPECT(awq_fp8_gemm(x.p(), s, 8, kc.p(), s, 32768, 64, y.p(), w.p() + 16, big, nullptr) == AWQ_ERR_INVALID_ARG);

    // ---- the plans over the whole range: a workspace of zero, or the first 64 KiB and less than 1 GiB of partials
    const int64_t Ms[] = {1, 2, 16, 17, 33, 64, 65, 257, 4096, 65536, 65535 * 16};
    const int64_t Ks[] = {16, 80, 128, 144, 4096, 28672, 1 << 20, (int64_t)65535 * 128};
    const int64_t Ns[] = {8, 16, 72, 256, 264, 4096, 28672, 1 << 20, 4194304};
    for (int64_t M : Ms)
        for (int64_t K : Ks)
            for (int64_t N : Ns) {
                const size_t bytes = awq_fp8_gemm_workspace_size(M, K, N);
                EXPECT(bytes == 0 || (bytes > 65536 && bytes < (size_t)1 << 30));
            }
    for (int64_t M : {(int64_t)1, (int64_t)300, (int64_t)1 << 20})
        for (int32_t n : {1, 2, 63, 1000, itop})
            for (int32_t q : {1, 2, 33, 2048, itop})
                for (int32_t Hk : {1, 8, 128, 1024})
                    for (int32_t G : {1, 8, 1024})
                        for (int32_t D : {64, 128}) {
                            if ((int64_t)Hk * G > 1024) continue;
                            const size_t bytes = awq_attention_workspace_size(M, n, q, Hk * G, Hk, D);
                            EXPECT(bytes == 0 || (bytes > 65536 && bytes < (size_t)1 << 30));
                        }
    for (Canary* c : {&x, &y, &kc, &vc, &sc, &cu, &len, &tab, &rope, &qw, &w}) EXPECT(c->intact());
    std::printf("%d failures\n", failures);
    return failures != 0;
}
