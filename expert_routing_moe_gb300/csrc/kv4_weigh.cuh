// kv4_weigh.cuh -- what the two kernels of moe_kv4_weigh share: the arguments,
// the rows that count and the score's update.
#pragma once

#include <cuda_bf16.h>

#include "attn_kv4.cuh"
#include "common.cuh"
#include "kv4.cuh"
#include "ranges.h"

namespace moe {

struct WeighArgs {
    const __nv_bfloat16* q;
    long long ld_q;
    int T, n_q, group;
    moe_kv4_cache c;
    const int32_t* q_start;
    const float* lse;
    float scale;
    int window, last, max_new;
    float* score;
    long long ld_score;
    bool fresh;
    int many;                   // sequences with that many counted rows or more go to the kernel for prompts (1: all that have any)
    moe_dev_status* st;
};

// A sequence's rows that count, and the places that they may see.
struct WeighSeq {
    int q0, n, len;             // n: rows, of which the first i0 do not count
    int i0;
    bool fit;
    __device__ int base() const { return len - n; }                 // place of row 0
    __device__ int first_new() const { return max(0, len - n); }
};
__device__ __forceinline__ WeighSeq weigh_seq(const WeighArgs& a, int s) {
    WeighSeq q;
    q.q0 = a.q_start[s];
    const int q1 = a.q_start[s + 1];
    q.len = a.c.seq_len[s];
    q.fit = rows_fit(q.q0, q1, q.len, a.T, a.c.max_pages) && q1 - q.q0 <= a.max_new;
    q.n = q.fit ? q1 - q.q0 : 0;
    if (!q.fit) q.len = 0;
    q.i0 = a.last > 0 && a.last < q.n ? q.n - a.last : 0;
    return q;
}
// The first place that the call touches: the first row's window, and the rows' own tokens where they are set.
__device__ __forceinline__ int weigh_first(const WeighArgs& a, const WeighSeq& q) {
    const int p0 = q.base() + q.i0;
    const int lo = a.window > 0 ? max(0, p0 - a.window + 1) : 0;
    return a.fresh ? min(lo, q.first_new()) : lo;
}
// The counted rows [ia, ib) that see something of the places key0 .. key0 + keys - 1.
__device__ __forceinline__ void weigh_rows(const WeighArgs& a, const WeighSeq& q, int key0, int keys, int& ia, int& ib) {
    ia = max(q.i0, key0 - q.base());
    ib = q.n;
    if (a.window > 0) ib = static_cast<int>(min(static_cast<long long>(ib), static_cast<long long>(key0) + keys - 1 + a.window - q.base()));
    if (ib < ia) ib = ia;
}
__device__ __forceinline__ void weigh_add(const WeighArgs& a, const WeighSeq& q, int s, int key, float v) {
    float* out = a.score + s * a.ld_score + key;
    *out = a.fresh && key >= q.first_new() ? v : *out + v;
}

// The kernel for prompts takes sequences of that many counted rows (times query heads of a key head).  9001 tokens, 32 + 4 heads:
// 64 rows 14.6 us without it and 20.5 with it (it is three launches), 128 rows 23.6 and 18.0, 256 rows 42 and 19, 1024 rows
// 154 and 27; six such sequences 14.4 / 21.4, 23.8 / 22.1, 42 / 24, 154 / 34; 128 rows of 500 tokens 23.2 / 17.0.
constexpr int kWeighMany = 128;
bool weigh_tc_fits(int group);
size_t kv4_weigh_tc_workspace(int S, int max_pages);
cudaError_t launch_kv4_weigh_tc(const WeighArgs& a, void* ws, cudaStream_t s);

}  // namespace moe
