// Prints the product's plan for each "M K N bits" line of its input: the register kernel ("rows", 16-row
// fragments) or tiles ("tile", rows / 64), and the slices of K (built by tests/test_mx_plan_paths.py; host code only).
#include <cinttypes>
#include <cstdio>

#include "../weight_only_int4_act_amd/csrc/awq_mx.h"

int main() {
    int64_t M, K, N;
    int bits;
    while (std::scanf("%" SCNd64 " %" SCNd64 " %" SCNd64 " %d", &M, &K, &N, &bits) == 4) {
        const awq::MxGemmPlan p = awq::plan_mx_gemm(M, K, N, bits);
        std::printf("%s %d %d\n", p.wm ? "tile" : "rows", p.wm ? p.wm : (int)p.row_tiles, p.nz);
    }
    return 0;
}
