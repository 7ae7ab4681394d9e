// Prints the plan of the attention over the cache for each "n_seq max_q tokens Hq Hk D" line of its input: rows per
// workgroup, most slices, row tiles, and whether its workspace is within the size that callers are told (built by
// tests/test_attention_plan_paths.py; host code only).
#include <cinttypes>
#include <cstdio>

#include "../include/awq.h"
#include "../weight_only_int4_act_amd/csrc/awq_cache.h"

int main() {
    int n, q, Hq, Hk, D;
    int64_t tokens;
    while (std::scanf("%d %d %" SCNd64 " %d %d %d", &n, &q, &tokens, &Hq, &Hk, &D) == 6) {
        const int64_t M = (int64_t)n * q;
        const awq::AttentionPlan p = awq::plan_attention(M, n, q, Hq, Hk, D, tokens);
        const size_t part = (size_t)n * p.tiles * Hk * p.split * p.rows * (8 + 4 * (size_t)D) + 65536;
        const size_t told = awq_attention_workspace_size(M, n, q, Hq, Hk, D);
        std::printf("%d %d %d %d\n", p.rows, p.split, p.tiles, p.ws_bytes == told && (p.split == 1 || part <= told));
    }
    return 0;
}
