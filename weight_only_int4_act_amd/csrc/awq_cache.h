// The 8-bit cache of keys and values: its layout and sequences as the kernels see them, and the host-side launchers
// (internal; the public ABI is include/awq.h).
//
// Elements are e4m3; a block of T tokens of one head has one scale byte E each for K and V, for 2^(E - 127): the least
// E >= 0 with max|p| <= 448 * 2^(E - 127); 255 once an infinity or a NaN has been appended.
#pragma once
#include "awq_device.h"

namespace awq {

struct Cache {
    uint8_t *k, *v, *scales;     // [blocks, Hk, T, D], [blocks, Hk, T/16, D, 16], [blocks, Hk, 2]
    int64_t blocks;
    int Hk, D, T, logT;
};
struct Sequences {
    const int32_t *cu, *length, *table;   // [n + 1], [n], [n, width]
    int n, width, max_q;
};

// The new tokens of a sequence: rows row0 .. row0 + count - 1, at positions start, start + 1, ...  In bounds whatever the
// arrays hold.  Counts that decrease may give a row to two sequences: looking through the counts before one's own would tell,
// but cost every call (one token behind 4096: 10.3 -> 10.7 us; 4096 sequences of 200: 167 -> 209).
struct NewTokens {
    int row0, count, start, length;
};
__device__ __forceinline__ NewTokens new_tokens(const Sequences& s, int b, int M) {
    NewTokens t;
    t.row0 = min(max(s.cu[b], 0), M);
    t.count = min(max(s.cu[b + 1], t.row0), M) - t.row0;
    t.length = max(s.length[b], 0);
    t.start = t.length - t.count;
    return t;
}

// ---- host side
int record_hip(hipError_t e);    // records a HIP error for awq_last_hip_error, returns the call's status (awq_api.hip)

struct AppendArgs {
    const uint16_t *qkv, *q_weight, *k_weight;
    const float* rope;
    uint16_t* q;
    int64_t M;
    int Hq, P, R, interleaved;
    double eps;
};
// The blocks that max_q tokens touch at most, wherever the first lies, and the workgroups that share the heads of q of one of
// them and one head of K and V: up to four rounds of heads each, or eight where there are thousands of workgroups and K's
// and V's have as much to do (4096 tokens of 64 heads on 8, T = 64: 49.0 and 46.4 us, 12000, T = 128: 116 and 109; but 3
// sequences of 40 7.2 and 9.7, and 18000 of 32 heads on 8, T = 32: 66 and 74).  None, where these are no more heads than a block has of K and there are workgroups enough for several per
// CU: K's and V's take them along (6100 tokens of 40 heads, each with its own K, T = 16: 97 us, with a workgroup of their own
// 120; one token of 64 such sequences 14.5 and 17.8; but one token of one sequence of 64 and 8 heads 6.2 and 5.0).
inline int64_t append_per_seq(int max_q, int T) { return ((int64_t)max_q + T - 2) / T + 1; }
inline int append_parts(int n_seq, int max_q, int G, int Hk, int T, int D) {
    const int64_t heads = (int64_t)(max_q < T ? max_q : T) * G, round = 256 / (D / 8), blocks = n_seq * append_per_seq(max_q, T);
    if (heads <= T && blocks >= 1024 / Hk) return 0;
    const int64_t parts = (heads + 4 * round - 1) / (4 * round);
    return (int)(T >= 64 && blocks * Hk * parts > 4096 ? (parts + 1) / 2 : parts);
}
hipError_t launch_qkv_append(const AppendArgs& a, const Sequences& s, const Cache& c, hipStream_t st);

constexpr float kLog2e = 1.44269504088896340736f;
struct AttentionPlan {
    int split;                   // most slices of a sequence's tokens
    int rows;                    // rows per workgroup, which says which kernel: 16, 128 or 256
    int tiles;                   // row tiles per sequence and head
    size_t ws_bytes;             // of any `tokens`
};
inline int attention_threads(const AttentionPlan& p) { return p.rows == 256 ? 512 : 256; }   // of a workgroup
AttentionPlan plan_attention(int64_t M, int n_seq, int max_q, int Hq, int Hk, int D, int64_t tokens);
hipError_t launch_attention(const uint16_t* q, int64_t M, int Hq, const Sequences& s, const Cache& c, float scale,
                            int causal, uint16_t* out, void* ws, const AttentionPlan& p, hipStream_t st);

}  // namespace awq
