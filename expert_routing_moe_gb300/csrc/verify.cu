// verify.cu -- verification of drafted tokens against the target's
// distribution (moe_verify_drafts).
//
// First the rows' maxima and the sums of their tokens' weights: a cluster a row
// where there are few, and otherwise a kernel for the maxima and one for the
// sums, a warp a chunk of a row.  Then a cluster for every sequence accepts its
// drafts or not and draws the token that follows.  Weights are whole multiples of 2^-42
// made from fp32 numbers whose every operation is rounded in a known way, so
// that sums of them do not depend on their order and a draw not on the grid.
//
// 32 sequences of up to five rows of 128001 bf16 logits and as many of a drafting
// model's: 54 MB, 8 us at the rate of a copy; 41 us, about 10 for the maxima, 16 for the sums (24 instructions for two
// weights, half of the issue slots) and 15 for the draw, a chain of loads and
// meetings.  One sequence of five rows of 32000: 9.8 us, all of it such a chain.
// Tried: a row's cluster that finds the maximum and the sum at once for all sizes
// (53 us), one kernel with a cluster a sequence for everything (56 us, one
// sequence 14.9), the draw by a warp a chunk and the last one (44 us, 12.8).
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "kv4.cuh"
#include "launch.h"
#include "ranges.h"
#include "tmap.h"

namespace moe {

namespace cg = cooperative_groups;

namespace {

constexpr int kThreads = 512;        // of the clusters
constexpr int kWarps = kThreads / 32;
constexpr int kHeld = 4;             // 16-byte runs of a row that a thread of a cluster loads at once
constexpr int kMaxCluster = 8;
constexpr int kRowCtas = 304;        // a wave of clusters, two CTAs an SM
constexpr int kMaxThreads = 256;     // of the kernel for the maxima; a CTA's chunk has kChunkHeld runs a thread
constexpr int kSumThreads = 128;     // of the sums; a warp's chunk has kChunkHeld runs a lane
constexpr int kChunkHeld = 8;        // 16-byte runs of a chunk that a thread has
constexpr float kLog2eF = 0x1.715476p+0f;
constexpr float kGreedyBelow = 0x1p-60f;

// What a row's tokens weigh, of a chunk of it.
struct ChunkSum {
    long long z;                     // sum of the weights
    int32_t best;                    // greedy: place of the row's largest logit
    int32_t pad;
};

struct VerifyArgs {
    const void *logits, *draft;
    long long ld, ld_draft;
    int T, V, S;
    const int32_t *tokens, *q_start;
    const float *uniform, *temperature;
    int32_t *accepted, *next, *n_new;
    int items;                       // rows of the target, then of the drafting model
    int max_chunks, max_per;         // chunks of a row and their 16-byte runs, for the maxima
    int chunks, per;                 // for the sums
    float* scale;                    // [items]: what the row was weighed with: 1 / temperature, 0: greedy, below: it was not
    float* maxima;                   // [items][max_chunks]
    ChunkSum* sums;                  // [items][chunks]
    moe_dev_status* st;
};

template <typename L>
struct Run {                         // 16 bytes of logits
    static constexpr int E = 16 / sizeof(L);
};
template <typename L>
__device__ __forceinline__ float as_float(uint4 v, int i) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (sizeof(L) == 4) return __uint_as_float(w[i]);
    else return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
}
template <typename L>
__device__ __forceinline__ float load_one(const void* p, long long i) {
    if constexpr (sizeof(L) == 4) return static_cast<const float*>(p)[i];
    else return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// A row in 16-byte runs from the boundary at or before its first number: run v holds numbers v*E - off .. + E - 1, of
// which some lie outside the row at its ends (they share its first or last 16 bytes).
template <typename L>
struct Row {
    const uint4* runs;
    int off, V, n;                   // n: runs
    __device__ Row(const void* base, long long ld, int row, int v) {
        const uintptr_t p = reinterpret_cast<uintptr_t>(static_cast<const L*>(base) + row * ld);
        runs = reinterpret_cast<const uint4*>(p & ~static_cast<uintptr_t>(15));
        off = static_cast<int>(p & 15) / static_cast<int>(sizeof(L));
        V = v;
        n = (off + V + Run<L>::E - 1) / Run<L>::E;
    }
    __device__ int first(int v) const { return v * Run<L>::E - off; }      // number of the run's first place
    __device__ bool whole(int v) const { return first(v) >= 0 && first(v) + Run<L>::E <= V; }
};

// The run with -inf in the places outside the row, which then weigh nothing.
template <typename L>
__device__ __noinline__ uint4 mask_ends(uint4 x, int e, int V) {
    uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(L) == 4) {
            if (e + i < 0 || e + i >= V) w[i] = 0xff800000u;
        } else {
            if (e + 2 * i < 0 || e + 2 * i >= V) w[i] = (w[i] & 0xffff0000u) | 0xff80u;
            if (e + 2 * i + 1 < 0 || e + 2 * i + 1 >= V) w[i] = (w[i] & 0xffffu) | 0xff800000u;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename L>
__device__ __forceinline__ uint4 mask_run(const Row<L>& r, uint4 x, int v) {
    return r.whole(v) ? x : mask_ends<L>(x, r.first(v), r.V);
}
// The largest of the run's numbers, or a NaN.
template <typename L>
__device__ __forceinline__ float max_run(uint4 x);

__device__ __forceinline__ float max_nan(float x, float y) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
    return r;
}

template <>
__device__ __forceinline__ float max_run<float>(uint4 x) {
    return max_nan(max_nan(__uint_as_float(x.x), __uint_as_float(x.y)), max_nan(__uint_as_float(x.z), __uint_as_float(x.w)));
}
__device__ __forceinline__ uint32_t max_nan_bf2(uint32_t x, uint32_t y) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    return r;
}
template <>
__device__ __forceinline__ float max_run<__nv_bfloat16>(uint4 x) {
    const uint32_t m = max_nan_bf2(max_nan_bf2(x.x, x.y), max_nan_bf2(x.z, x.w));
    return max_nan(__uint_as_float(m << 16), __uint_as_float(m & 0xffff0000u));
}

// What two tokens weigh relative to the row's strongest: 2^t, t = n + f, the series of 2^f by Horner.  Every operation is
// rounded as the definition has it (a product by -1 is exact, so t - n may be a fused product).  For logits up to m.
struct Scale {
    float2 minus_m, it;
    __device__ Scale(float m, float it_) : minus_m(make_float2(-m, -m)), it(make_float2(it_, it_)) {}
};
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 weight2(float2 l, const Scale& s) {
    float2 t = mul2(add2(l, s.minus_m), s.it);
    t = make_float2(fmaxf(t.x, -60.f), fmaxf(t.y, -60.f));
    const float2 y = add2(t, both(0x1.8p23f));            // rounds t to a whole number, ties to even
    const float2 f = fma2(add2(y, both(-0x1.8p23f)), both(-1.f), t);
    float2 p = both(0x1.430912p-13f);                     // ln(2)^i / i!, i = 6 .. 0, nearest fp32
    p = fma2(p, f, both(0x1.5d87fep-10f));
    p = fma2(p, f, both(0x1.3b2ab6p-7f));
    p = fma2(p, f, both(0x1.c6b08ep-5f));
    p = fma2(p, f, both(0x1.ebfbe0p-3f));
    p = fma2(p, f, both(0x1.62e430p-1f));
    p = fma2(p, f, both(1.f));
    // y's low bits are n
    return make_float2(__uint_as_float(__float_as_uint(p.x) + (__float_as_uint(y.x) << 23)),
                       __uint_as_float(__float_as_uint(p.y) + (__float_as_uint(y.y) << 23)));
}
__device__ __forceinline__ float weight(float l, const Scale& s) { return weight2(both(l), s).x; }

// rint(w * 2^42) for 0 <= w < 4 as hi * 2^22 + lo (a conversion to 64 bits runs at 1/64 of an addition's rate): hi counts
// units of 2^-20, what is left of w is exact and counts units of 2^-42.  The bits of two fp32 numbers count them, from those
// of 12 (whose neighbours are 2^-20 apart) and of 1.5 * 2^23.
constexpr uint32_t kHi0 = 0x41400000u, kLo0 = 0x4b400000u;
__device__ __forceinline__ void split2(float2 w, float2& hi, float2& lo) {
    hi = add2(w, both(12.f));
    const float2 r = fma2(add2(hi, both(-12.f)), both(-1.f), w);
    lo = fma2(r, both(0x1p42f), both(0x1.8p23f));
}
__device__ __forceinline__ long long units(uint32_t hi, uint32_t lo) {     // of the bits less kHi0 and kLo0
    return static_cast<long long>(static_cast<int>(hi)) * (1 << 22) + static_cast<int>(lo);
}
__device__ __forceinline__ long long units_of(float w) {
    float2 hi, lo;
    split2(both(w), hi, lo);
    return units(__float_as_uint(hi.x) - kHi0, __float_as_uint(lo.x) - kLo0);
}
// Sums of them, for up to 2^10 numbers.
struct Units {
    uint32_t hi = 0u, lo = 0u, n = 0u;
    __device__ __forceinline__ void add(float2 w) {
        float2 h, l;
        split2(w, h, l);
        hi += __float_as_uint(h.x) + __float_as_uint(h.y);
        lo += __float_as_uint(l.x) + __float_as_uint(l.y);
        n += 2;
    }
    __device__ __forceinline__ long long sum() const { return units(hi - n * kHi0, lo - n * kLo0); }
    // Of a warp, up to 2^6 numbers a lane.
    __device__ __forceinline__ long long warp_sum() const {
        const int l = static_cast<int>(lo - n * kLo0);
        const long long h = __reduce_add_sync(kFull, hi - n * kHi0);
        return (h << 22) + (static_cast<long long>(__reduce_add_sync(kFull, l >> 16)) << 16) + __reduce_add_sync(kFull, l & 0xffff);
    }
};

// The sequence's temperature: 1 / it, greedy or bad.
struct Temp {
    float it;
    bool greedy, bad;
};
__device__ __forceinline__ Temp temp_of(const VerifyArgs& a, int s) {
    const float t = a.temperature == nullptr ? 1.f : a.temperature[s];
    Temp r;
    r.bad = !(t >= 0.f) || t - t != 0.f;
    r.greedy = !r.bad && t < kGreedyBelow;
    r.it = r.bad || r.greedy ? 1.f : __fdiv_rn(kLog2eF, t);
    return r;
}
// What a sequence's rows are weighed with, as it stands beside their sums.
__device__ __forceinline__ float scale_of(const Temp& t) { return t.bad ? -1.f : t.greedy ? 0.f : t.it; }
// Rows of sequence s; none if they are not rows of the step.
__device__ __forceinline__ bool seq_rows(const VerifyArgs& a, int s, int& r0, int& r1) {
    r0 = a.q_start[s];
    r1 = a.q_start[s + 1];
    if (0 <= r0 && r0 <= r1 && r1 <= a.T) return true;
    r1 = r0;
    return false;
}

__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
    return v;
}

// Sequence of an item's row, -1 without one.  Bad starts can give a row to several: it is the first one's, so that all
// CTAs of the row find the same.
template <int THREADS>
__device__ __forceinline__ int find_seq(const VerifyArgs& a, int row, bool draft, int* s_seq) {
    if (threadIdx.x == 0) *s_seq = 0x7fffffff;
    __syncthreads();
    for (int s = threadIdx.x; s < a.S; s += THREADS) {
        const int r0 = __ldg(a.q_start + s), r1 = __ldg(a.q_start + s + 1);
        // a drafting model's row is read for the draft behind it
        if (r0 >= 0 && r0 <= row && row + (draft ? 1 : 0) < r1 && r1 <= a.T) atomicMin(s_seq, s);
    }
    __syncthreads();
    return *s_seq == 0x7fffffff ? -1 : *s_seq;
}

// What acceptance needs of a row: the sum of its weights, its largest logit, the weight of the draft behind it and 2^42 / z.
struct Weighed {
    long long z, u;
    float m, inv;
};

__device__ __noinline__ double ratio(double x, long long z) { return x / __ll2double_rn(z); }
// 2^42 / z in fp64, rounded to fp32, for 2^42 <= z <= 2^62.  An SM has two fp64 lanes and a division takes a microsecond there:
// with z = zh + zl and r = 1 / zh in fp32, r + r (1 - (zh + zl) r) is within 2^-45 of the quotient, and the division
// is only needed where numbers that close to it round differently.
__device__ __forceinline__ float inverse(long long z) {
    const float top = __ll2float_rn(z), zh = top * 0x1p-42f, zl = __ll2float_rn(z - __float2ll_rn(top)) * 0x1p-42f;
    const float r = __frcp_rn(zh), c = r * fmaf(-zl, r, fmaf(-zh, r, 1.f)), d = r * 0x1p-43f;
    const float lo = r + (c - d), hi = r + (c + d);
    return lo == hi ? lo : __double2float_rn(ratio(0x1p42, z));
}
// uniform * q < p, each p of a token u / z in fp64: again fp32 decides unless both sides are close.
__device__ __forceinline__ bool accepts(float uniform, const Weighed& p, const Weighed& q, bool model) {
    const float pr = __ll2float_rn(p.u) * 0x1p-42f * p.inv, other = uniform * (model ? __ll2float_rn(q.u) * 0x1p-42f * q.inv : 1.f);
    if (fabsf(pr - other) > 0x1p-20f * pr) return other < pr;
    const double exact = model ? ratio(__ll2double_rn(q.u), q.z) : 1.0;
    return __dmul_rn(static_cast<double>(uniform), exact) < ratio(__ll2double_rn(p.u), p.z);
}

// A row by a cluster.
template <typename L>
__global__ void __launch_bounds__(kThreads, 2) verify_rows_kernel(const VerifyArgs a) {
    constexpr int E = Run<L>::E;
    cg::cluster_group cluster = cg::this_cluster();
    const int parts = static_cast<int>(cluster.num_blocks()), part = static_cast<int>(cluster.block_rank());
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    __shared__ int s_seq, s_best[kWarps];
    __shared__ float s_max[kWarps], s_part_max[kMaxCluster];
    __shared__ long long s_sum[kWarps], s_part_sum[kMaxCluster];
    __shared__ int s_part_best[kMaxCluster];
    const int item = blockIdx.x / parts;
    const bool draft = item >= a.T;
    const int row = draft ? item - a.T : item;
    cluster.barrier_arrive();        // waited for before the cluster's shared memory is written
    const Row<L> rw(draft ? a.draft : a.logits, draft ? a.ld_draft : a.ld, row, a.V);
    const int v0 = static_cast<int>(static_cast<long long>(rw.n) * part / parts), v1 = static_cast<int>(static_cast<long long>(rw.n) * (part + 1) / parts);
    uint4 held[kHeld];
    pdl_wait();
    pdl_trigger();
    // the row is on its way while its sequence is looked for
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
        if (v0 + tid + i * kThreads < v1) held[i] = __ldg(rw.runs + v0 + tid + i * kThreads);
    const int s = find_seq<kThreads>(a, row, draft, &s_seq);
    cluster.barrier_wait();
    const Temp temp = s < 0 ? Temp{1.f, false, true} : temp_of(a, s);
    const bool needed = !temp.bad && !(draft && temp.greedy);
    if (part == 0 && tid == 0) a.scale[item] = needed ? scale_of(temp) : -1.f;
    if (!needed) {                                         // the whole cluster
        if (part == 0 && tid == 0) a.maxima[item] = NAN;   // (a sequence that reads the row all the same finds it bad)
        return;
    }
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
        if (v0 + tid + i * kThreads < v1) {
            held[i] = mask_run(rw, held[i], v0 + tid + i * kThreads);
            m = max_nan(m, max_run<L>(held[i]));
        }
    for (int v = v0 + tid + kHeld * kThreads; v < v1; v += kThreads) m = max_nan(m, max_run<L>(mask_run(rw, __ldg(rw.runs + v), v)));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = max_nan(m, __shfl_xor_sync(kFull, m, off));
    if (lane == 0) s_max[warp] = m;
    __syncthreads();
    if (tid < parts) {
        m = s_max[0];
        for (int i = 1; i < kWarps; ++i) m = max_nan(m, s_max[i]);
        cluster.map_shared_rank(s_part_max, tid)[part] = m;
    }
    cluster.sync();
    m = s_part_max[0];
    for (int i = 1; i < parts; ++i) m = max_nan(m, s_part_max[i]);
    const bool bad = !(m - m == 0.f);
    if (bad && part == 0 && tid == 0) report(a.st, MOE_DEV_NONFINITE, item);

    int best = 0x7fffffff;
    Units u;
    if (!bad) {
        const Scale scale(m, temp.it);
        auto add = [&](uint4 x, int v) {
            if (temp.greedy) {
                const int e = rw.first(v);
#pragma unroll
                for (int i = 0; i < E; ++i)
                    if (as_float<L>(x, i) == m) best = min(best, e + i);       // (the places outside the row are -inf)
            } else {
#pragma unroll
                for (int i = 0; i < E; i += 2) u.add(weight2(make_float2(as_float<L>(x, i), as_float<L>(x, i + 1)), scale));
            }
        };
#pragma unroll
        for (int i = 0; i < kHeld; ++i)
            if (v0 + tid + i * kThreads < v1) add(held[i], v0 + tid + i * kThreads);
        for (int v = v0 + tid + kHeld * kThreads; v < v1; v += kThreads) add(mask_run(rw, __ldg(rw.runs + v), v), v);
    }
    const long long sum = warp_sum(u.sum());
    best = __reduce_min_sync(kFull, best);
    if (lane == 0) { s_sum[warp] = sum; s_best[warp] = best; }
    __syncthreads();
    if (tid == 0) {
        long long z = 0;
        for (int i = 0; i < kWarps; ++i) { z += s_sum[i]; best = min(best, s_best[i]); }
        cluster.map_shared_rank(s_part_sum, 0)[part] = z;
        cluster.map_shared_rank(s_part_best, 0)[part] = best;
    }
    cluster.sync();
    if (part == 0 && tid == 0) {
        ChunkSum c = {0, best, 0};
        for (int i = 0; i < parts; ++i) { c.z += s_part_sum[i]; c.best = min(c.best, s_part_best[i]); }
        a.maxima[item] = m;
        a.sums[item] = c;
    }
}

template <typename L>
__global__ void __launch_bounds__(kMaxThreads) verify_max_kernel(const VerifyArgs a) {
    __shared__ int s_seq;
    __shared__ float s_max[kMaxThreads / 32];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int item = blockIdx.x / a.max_chunks, chunk = blockIdx.x % a.max_chunks;
    const bool draft = item >= a.T;
    const int row = draft ? item - a.T : item;
    pdl_wait();
    pdl_trigger();
    const int s = find_seq<kMaxThreads>(a, row, draft, &s_seq);
    const Temp temp = s < 0 ? Temp{1.f, false, true} : temp_of(a, s);
    const bool needed = !temp.bad && !(draft && temp.greedy);
    if (chunk == 0 && tid == 0) a.scale[item] = needed ? scale_of(temp) : -1.f;
    if (!needed) {
        if (tid == 0) a.maxima[blockIdx.x] = NAN;          // (see above)
        return;
    }
    const Row<L> rw(draft ? a.draft : a.logits, draft ? a.ld_draft : a.ld, row, a.V);
    const int v0 = chunk * a.max_per + tid, v1 = min(rw.n, (chunk + 1) * a.max_per);
    uint4 held[kChunkHeld];
#pragma unroll
    for (int i = 0; i < kChunkHeld; ++i)
        if (v0 + i * kMaxThreads < v1) held[i] = __ldg(rw.runs + v0 + i * kMaxThreads);
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kChunkHeld; ++i)
        if (v0 + i * kMaxThreads < v1) m = max_nan(m, max_run<L>(mask_run(rw, held[i], v0 + i * kMaxThreads)));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = max_nan(m, __shfl_xor_sync(kFull, m, off));
    if (lane == 0) s_max[warp] = m;
    __syncthreads();
    if (tid == 0) {
        for (int i = 1; i < kMaxThreads / 32; ++i) m = max_nan(m, s_max[i]);
        a.maxima[blockIdx.x] = m;
    }
}

// The row's largest logit, or what is not finite.
__device__ __forceinline__ float row_max(const VerifyArgs& a, int item, int lane) {
    float m = -INFINITY;
    for (int i = lane; i < a.max_chunks; i += 32) m = max_nan(m, __ldcg(a.maxima + static_cast<size_t>(item) * a.max_chunks + i));
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) m = max_nan(m, __shfl_xor_sync(kFull, m, off));
    return m;
}

template <typename L>
__global__ void __launch_bounds__(kSumThreads, 8) verify_sum_kernel(const VerifyArgs a) {
    constexpr int E = Run<L>::E;
    const int lane = threadIdx.x & 31;
    const int unit = blockIdx.x * (kSumThreads / 32) + (threadIdx.x >> 5);
    const int item = unit / a.chunks, chunk = unit - item * a.chunks;
    if (item >= a.items) return;
    const bool draft = item >= a.T;
    const int row = draft ? item - a.T : item;
    const Row<L> rw(draft ? a.draft : a.logits, draft ? a.ld_draft : a.ld, row, a.V);
    const int v0 = chunk * a.per + lane, v1 = min(rw.n, (chunk + 1) * a.per);
    pdl_wait();
    pdl_trigger();
    const float it = __ldcg(a.scale + item);
    const float m = row_max(a, item, lane);
    if (it < 0.f) return;
    uint4 held[kChunkHeld];
#pragma unroll
    for (int i = 0; i < kChunkHeld; ++i)
        if (v0 + i * 32 < v1) held[i] = __ldg(rw.runs + v0 + i * 32);
    if (!(m - m == 0.f)) {
        if (chunk == 0 && lane == 0) report(a.st, MOE_DEV_NONFINITE, item);
        return;
    }
    if (it == 0.f) {
        int best = 0x7fffffff;
#pragma unroll
        for (int i = 0; i < kChunkHeld; ++i) {
            const int v = v0 + i * 32;
            if (v >= v1) continue;
            const uint4 x = mask_run(rw, held[i], v);
            const int e = rw.first(v);
#pragma unroll
            for (int j = 0; j < E; ++j)
                if (as_float<L>(x, j) == m) best = min(best, e + j);   // (the places outside the row are -inf)
        }
        best = __reduce_min_sync(kFull, best);
        if (lane == 0) a.sums[unit] = {0, best, 0};
        return;
    }
    Units u;
    const Scale scale(m, it);
#pragma unroll
    for (int i = 0; i < kChunkHeld; ++i) {
        const int v = v0 + i * 32;
        if (v >= v1) continue;
        const uint4 x = mask_run(rw, held[i], v);
#pragma unroll
        for (int j = 0; j < E; j += 2) u.add(weight2(make_float2(as_float<L>(x, j), as_float<L>(x, j + 1)), scale));
    }
    const long long sum = u.warp_sum();
    if (lane == 0) a.sums[unit] = {sum, 0x7fffffff, 0};
}

// A row's maximum and sum, by a warp, for a sequence that takes them with `scale`.  Bad too where the row was weighed for another
// sequence with another temperature.
struct RowInfo {
    float m;
    bool bad;
    long long z;
    int best;
};
__device__ __forceinline__ RowInfo row_info(const VerifyArgs& a, int item, float scale, int lane) {
    const float with = __ldcg(a.scale + item);
    RowInfo r = {row_max(a, item, lane), false, 0, 0x7fffffff};
    r.bad = !(r.m - r.m == 0.f) || with != scale;
    if (r.bad) return r;
    for (int i = lane; i < a.chunks; i += 32) {
        const int4 c = __ldcg(reinterpret_cast<const int4*>(a.sums + static_cast<size_t>(item) * a.chunks + i));
        r.z += static_cast<long long>(static_cast<unsigned long long>(static_cast<uint32_t>(c.y)) << 32 | static_cast<uint32_t>(c.x));
        r.best = min(r.best, c.z);
    }
    r.z = warp_sum(r.z);
    r.best = __reduce_min_sync(kFull, r.best);
    return r;
}

// What the tokens of the row behind the last accepted draft weigh for the draw.
template <typename L>
struct Draw {
    Row<L> p, q;
    Scale sp, sq;
    float ip, iq;
    int mode, without;               // mode 0: the target's weights, 1: those but for one token, 2: max(p - q, 0)
    static constexpr int E = Run<L>::E;
    // the drafting model's logits beside the target's run
    __device__ __forceinline__ uint4 beside(int v) const {
        return q.off == p.off ? __ldg(q.runs + v) : gather(q.runs, q.off + p.first(v), p.first(v), p.V);
    }
    __device__ static __noinline__ uint4 gather(const uint4* runs, int at, int e, int V) {
        uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < E; ++i) {
            if (e + i < 0 || e + i >= V) continue;
            if constexpr (sizeof(L) == 4) w[i] = __float_as_uint(load_one<L>(runs, at + i));
            else w[i / 2] |= (__float_as_uint(load_one<L>(runs, at + i)) >> 16) << (16 * (i & 1));
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    // the weights of a run's numbers two by two; less than half a unit in the places outside the row, where both are -inf
    template <typename F>
    __device__ __forceinline__ void run(int v, uint4 x, uint4 y, F use) const {
        const int e = p.first(v);
        x = mask_run(p, x, v);
        // (a logit above its row's maximum, as what lies beside the row may be, has no weight: its exponent can reach the sign)
        if (mode == 2) y = mask_run(p, y, v);
#pragma unroll
        for (int i = 0; i < E; i += 2) {
            float2 w = weight2(make_float2(as_float<L>(x, i), as_float<L>(x, i + 1)), sp);
            if (mode == 2) {
                const float2 o = mul2(weight2(make_float2(as_float<L>(y, i), as_float<L>(y, i + 1)), sq), both(iq));
                w = fma2(o, both(-1.f), mul2(w, both(ip)));
                w = make_float2(fmaxf(w.x, 0.f), fmaxf(w.y, 0.f));
            }
            if (mode == 1) {
                if (e + i == without) w.x = 0.f;
                if (e + i + 1 == without) w.y = 0.f;
            }
            use(i, w);
        }
    }
};

// Rows of a sequence that are looked at in a turn, and what was found at the row that ends the accepted drafts.
struct Looked {
    long long z[kWarps][2], u[kWarps][2];          // of the target and of the drafting model: sum, the draft's weight
    float m[kWarps][2];
    int best[kWarps];
    int stop, bad, stop_best;
    float stop_m[2], stop_inv[2];
    long long target;
};

template <typename L>
__global__ void __launch_bounds__(kThreads, 2) verify_draw_kernel(const VerifyArgs a) {
    constexpr int E = Run<L>::E;
    cg::cluster_group cluster = cg::this_cluster();
    const int parts = static_cast<int>(cluster.num_blocks()), part = static_cast<int>(cluster.block_rank());
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    __shared__ Looked s_l;
    __shared__ long long s_sums[2][kMaxCluster * kWarps];
    const int s = blockIdx.x / parts;
    if (tid == 0) { s_l.stop = -1; s_l.bad = 0; }
    cluster.sync();
    pdl_wait();
    pdl_trigger();
    int r0, r1;
    const bool lead = part == 0 && tid == 0;
    const bool fit = seq_rows(a, s, r0, r1);
    if (!fit && lead) report(a.st, MOE_DEV_BAD_INDEX, s);
    const int n = r1 - r0;
    const Temp temp = temp_of(a, s);
    if (temp.bad && n > 0 && lead) report(a.st, MOE_DEV_NONFINITE, -1 - s);
    auto answer = [&](int accepted, int next) {
        a.accepted[s] = accepted;
        a.next[s] = next;
        if (a.n_new != nullptr) a.n_new[s] = n > 0 ? accepted - (n - 1) : 0;
    };
    if (n == 0 || temp.bad) {
        if (lead) answer(0, -1);
        return;                      // the whole cluster
    }
    // every CTA looks at all drafts for itself: a warp gathers what is known of a row, then the first warp looks at them
    for (int base = 0; base < n; base += kWarps) {
        const int j = base + warp;
        if (j < n) {
            const bool last = j == n - 1, with = a.draft != nullptr && !temp.greedy && !last;
            const int x = last ? 0 : a.tokens[r0 + j + 1];
            const bool in = x >= 0 && x < a.V;
            int best = 0;
            bool bad = !in;
#pragma unroll 1
            for (int q = 0; q <= with; ++q) {
                const float l = in ? load_one<L>(q ? a.draft : a.logits, (r0 + j) * (q ? a.ld_draft : a.ld) + x) : 0.f;
                const RowInfo r = row_info(a, r0 + j + q * a.T, scale_of(temp), lane);
                bad = bad || r.bad;
                if (q == 0) best = r.best;
                if (lane == 0) {
                    s_l.z[warp][q] = r.z;
                    s_l.m[warp][q] = r.m;
                    s_l.u[warp][q] = units_of(weight(l, Scale(r.m, temp.it)));
                }
            }
            if (lane == 0) {
                s_l.best[warp] = temp.greedy && !last && x != best ? -1 - best : best;
                if (bad) s_l.bad = 1;
                if (!in && part == 0) report(a.st, MOE_DEV_BAD_INDEX, r0 + j + 1);
            }
        }
        __syncthreads();
        if (warp == 0 && s_l.stop < 0) {
            const int row = base + lane;
            const bool in = lane < kWarps && row < n;
            bool ends = in && row == n - 1;
            Weighed p = {}, q = {};
            if (in && temp.greedy) {
                ends = ends || s_l.best[lane] < 0;
            } else if (in) {
                const bool with = a.draft != nullptr && !ends;
#pragma unroll 1
                for (int i = 0; i <= with; ++i) {
                    q = p;
                    p = {s_l.z[lane][with - i], s_l.u[lane][with - i], s_l.m[lane][with - i], inverse(s_l.z[lane][with - i])};
                }
                ends = ends || !accepts(a.uniform[r0 + row + 1], p, q, with);
            }
            const unsigned mask = __ballot_sync(kFull, ends);
            if (mask != 0 && lane == __ffs(mask) - 1) {
                s_l.stop = row;
                s_l.stop_m[0] = p.m;
                s_l.stop_m[1] = q.m;
                s_l.stop_inv[0] = p.inv;
                s_l.stop_inv[1] = q.inv;
                s_l.stop_best = s_l.best[lane] < 0 ? -1 - s_l.best[lane] : s_l.best[lane];
            }
        }
        __syncthreads();
    }
    if (s_l.bad) {
        if (lead) answer(0, -1);
        return;
    }
    const int stop = s_l.stop;
    const int row = r0 + stop;
    if (temp.greedy) {
        if (lead) answer(stop, s_l.stop_best);
        return;
    }
    Draw<L> d = {Row<L>(a.logits, a.ld, row, a.V), Row<L>(a.logits, a.ld, row, a.V), Scale(s_l.stop_m[0], temp.it), Scale(s_l.stop_m[1], temp.it), s_l.stop_inv[0], s_l.stop_inv[1], 0, -1};
    if (stop < n - 1) {
        d.mode = 1;
        d.without = a.tokens[row + 1];
        if (a.draft != nullptr) {
            d.mode = 2;
            d.q = Row<L>(a.draft, a.ld_draft, row, a.V);
        }
    }
    // a warp's runs are neighbours, so that the warps' sums are the cumulated weight in order
    const int warps = parts * kWarps, w = part * kWarps + warp;
    const int v0 = static_cast<int>(static_cast<long long>(d.p.n) * w / warps), v1 = static_cast<int>(static_cast<long long>(d.p.n) * (w + 1) / warps);
    long long before = 0, target = 0;
    bool search = false;
    // once or twice for the sums, then by the warp whose runs hold the token (one loop: the code is fetched once)
#pragma unroll 1
    for (int turn = 0;;) {
        long long own = 0;
        uint4 x = {}, y = {};
        auto load = [&](int v) {
            if (v >= v1) return;
            x = __ldg(d.p.runs + v);
            if (d.mode == 2) y = d.beside(v);
        };
        load(v0 + lane);
#pragma unroll 1
        for (int v = v0 + lane; v - lane < v1; v += 32) {
            const uint4 xv = x, yv = y;
            load(v + 32);
            long long u[E], mine = 0;
#pragma unroll
            for (int i = 0; i < E; ++i) u[i] = 0;
            if (v < v1)
                d.run(v, xv, yv, [&](int i, float2 f) {
                    u[i] = units_of(f.x);
                    u[i + 1] = units_of(f.y);
                });
#pragma unroll
            for (int i = 0; i < E; ++i) mine += u[i];
            own += mine;
            if (!search) continue;
            long long inc = mine;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const long long o = __shfl_up_sync(kFull, inc, off);
                if (lane >= off) inc += o;
            }
            long long c = before + inc - mine;
            if (target >= c && target < c + mine) {
                int at = 0;
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    c += u[i];
                    at += target >= c;
                }
                answer(stop, d.p.first(v) + at);
            }
            before += __shfl_sync(kFull, inc, 31);
            if (target < before) break;
        }
        if (search) return;
        own = warp_sum(own);
        if (lane < parts) cluster.map_shared_rank(s_sums[turn], lane)[w] = own;
        cluster.sync();
        // all of them, and those of the warps before
        long long total = 0;
        before = 0;
        for (int i = lane; i < warps; i += 32) {
            const long long o = s_sums[turn][i];
            total += o;
            if (i < w) before += o;
        }
        total = warp_sum(total);
        before = warp_sum(before);
        if (total == 0) {            // nothing of the target is beyond the draft; the same in every CTA
            d.mode = 0;
            ++turn;
            continue;
        }
        if (tid == 0) {
            const long long t = __double2ll_rd(__dmul_rn(static_cast<double>(a.uniform[r0]), __ll2double_rn(total)));
            s_l.target = max(0ll, min(t, total - 1));
        }
        __syncthreads();
        target = s_l.target;
        if (target < before || target >= before + own) return;
        search = true;
    }
}

template <typename K>
cudaError_t launch_clusters(K kernel, int items, int parts, cudaStream_t s, const VerifyArgs& a) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(items * parts);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = parts;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

int cdiv(int n, int d) { return (n + d - 1) / d; }
template <typename L>
cudaError_t launch(VerifyArgs a, void* ws, cudaStream_t s) {
    const int runs = a.V / Run<L>::E + 2;
    int parts = 1;
    while (parts < kMaxCluster && runs > parts * kThreads) parts *= 2;
    if (a.T > 0) {
        a.items = a.draft != nullptr ? 2 * a.T : a.T;
        // (clusters / chunks, five rows of 32000 fp32 logits a sequence: 1 sequence 10.0 / 10.9 us, 8 12.5 / 12.3, 16 17.4 /
        // 15.3, 64 48.9 / 27.2; of 2000, with a drafting model's: 1 11.1 / 11.9, 32 11.8 / 12.7, 64 15.3 / 13.9)
        const bool few = static_cast<long long>(a.items) * parts <= kRowCtas;
        a.max_per = few ? runs : kMaxThreads * kChunkHeld;
        a.max_chunks = cdiv(runs, a.max_per);
        a.per = few ? runs : 32 * kChunkHeld;
        a.chunks = cdiv(runs, a.per);
        const size_t units = static_cast<size_t>(a.items) * a.chunks;
        a.sums = static_cast<ChunkSum*>(ws);
        a.maxima = reinterpret_cast<float*>(a.sums + units);
        a.scale = a.maxima + static_cast<size_t>(a.items) * a.max_chunks;
        cudaError_t e;
        if (few) {
            e = launch_clusters(verify_rows_kernel<L>, a.items, parts, s, a);
        } else {
            e = launch_pdl(verify_max_kernel<L>, dim3(a.items * a.max_chunks), dim3(kMaxThreads), 0, s, a);
            if (e == cudaSuccess) e = launch_pdl(verify_sum_kernel<L>, dim3((units + kSumThreads / 32 - 1) / (kSumThreads / 32)), dim3(kSumThreads), 0, s, a);
        }
        if (e != cudaSuccess) return e;
    }
    return launch_clusters(verify_draw_kernel<L>, a.S, parts, s, a);
}

}  // namespace

size_t verify_workspace(int T, int V) {
    if (T == 0) return 0;
    const int runs = V / Run<float>::E + 2;
    const long long items = 2ll * T;
    return static_cast<size_t>(items * cdiv(runs, 32 * kChunkHeld)) * sizeof(ChunkSum) +
           static_cast<size_t>(items * (cdiv(runs, kMaxThreads * kChunkHeld) + 1)) * sizeof(float);
}

cudaError_t launch_verify(const void* logits, int dtype, long long ld, int T, int V, const int32_t* tokens, const float* uniform,
                          const int32_t* q_start, int S, const void* draft, long long ld_draft, const float* temperature, int32_t* accepted,
                          int32_t* next, int32_t* n_new, void* ws, moe_dev_status* st, cudaStream_t s) {
    VerifyArgs a = {logits, draft, ld, ld_draft, T, V, S, tokens, q_start, uniform, temperature, accepted, next, n_new};
    a.st = st;
    return dtype == MOE_DTYPE_BF16 ? launch<__nv_bfloat16>(a, ws, s) : launch<float>(a, ws, s);
}

}  // namespace moe
