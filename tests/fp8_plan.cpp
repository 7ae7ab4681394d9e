// Prints the plan of the product with scales per 128 for each "M K N" line of its input: the register kernel ("rows", 16-row
// fragments) or tiles ("tile", rows / 64), and the slices of K (built by tests/test_fp8_plan_paths.py; host code only).
#include <cinttypes>
#include <cstdio>

#include "../weight_only_int4_act_amd/csrc/awq_fp8.h"

int main() {
    int64_t M, K, N;
    while (std::scanf("%" SCNd64 " %" SCNd64 " %" SCNd64, &M, &K, &N) == 3) {
        const awq::Fp8GemmPlan p = awq::plan_fp8_gemm(M, K, N);
        std::printf("%s %d %d\n", p.wm ? "tile" : "rows", p.wm ? p.wm : M <= 16 ? 1 : M <= 32 ? 2 : 4, p.nz);
    }
    return 0;
}
