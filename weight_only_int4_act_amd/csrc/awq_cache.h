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

// The new tokens of a sequence: rows row0 .. row0 + count - 1, at positions start, start + 1, ...
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
hipError_t launch_qkv_append(const AppendArgs& a, const Sequences& s, const Cache& c, hipStream_t st);

struct AttentionPlan {
    int split;                   // most slices of a sequence's tokens
    int rows;                    // rows per workgroup, which says which kernel: 16, 128 or 256
    int tiles;                   // row tiles per sequence and head
    size_t ws_bytes;
};
AttentionPlan plan_attention(int64_t M, int n_seq, int max_q, int Hq, int Hk, int D);
hipError_t launch_attention(const uint16_t* q, int64_t M, int Hq, const Sequences& s, const Cache& c, float scale,
                            int causal, uint16_t* out, void* ws, const AttentionPlan& p, hipStream_t st);

}  // namespace awq
