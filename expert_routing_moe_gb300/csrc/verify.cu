// verify.cu -- verification of drafted tokens against the target's
// distribution (moe_verify_drafts).
//
// First a cluster for every row finds its maximum and the sum of its tokens'
// weights; then a cluster for every sequence judges its drafts and draws the
// token that follows.  Weights are whole multiples of 2^-42 made from fp32
// numbers whose every operation is rounded in a known way, so that sums of
// them do not depend on their order and a draw not on the grid.
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "common.cuh"
#include "kv4.cuh"
#include "launch.h"
#include "ranges.h"
#include "tmap.h"

namespace moe {

namespace cg = cooperative_groups;

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kHeld = 4;             // 16-byte runs of a row that a thread keeps in registers
constexpr int kMaxCluster = 8;
constexpr float kLog2eF = 0x1.715476p+0f;
constexpr float kGreedyBelow = 0x1p-60f;

struct RowInfo {
    unsigned long long z;            // sum of the weights
    float m;                         // largest logit
    int32_t best;                    // greedy: its place
    int32_t bad;
    int32_t pad[3];
};

struct VerifyArgs {
    const void *logits, *draft;
    long long ld, ld_draft;
    int T, V, S;
    const int32_t *tokens, *q_start;
    const float *uniform, *temperature;
    int32_t *accepted, *next, *n_new;
    RowInfo* rows;                   // [T] of the target, then [T] of the drafting model
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
__device__ __forceinline__ uint4 mask_run(const Row<L>& r, uint4 x, int v) {
    if (r.whole(v)) return x;
    const int e = r.first(v);
    uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(L) == 4) {
            if (e + i < 0 || e + i >= r.V) w[i] = 0xff800000u;
        } else {
            if (e + 2 * i < 0 || e + 2 * i >= r.V) w[i] = (w[i] & 0xffff0000u) | 0xff80u;
            if (e + 2 * i + 1 < 0 || e + 2 * i + 1 >= r.V) w[i] = (w[i] & 0xffffu) | 0xff800000u;
        }
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
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
// rounded as the definition has it (a product by -1 is exact, so t - n may be a fused product).
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

template <typename L>
__global__ void __launch_bounds__(kThreads) verify_rows_kernel(const VerifyArgs a) {
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
    if (tid == 0) s_seq = -1;
    cluster.sync();                  // every CTA of the cluster runs: its shared memory can be written
    pdl_wait();
    pdl_trigger();
    for (int s = tid; s < a.S; s += kThreads) {
        const int r0 = a.q_start[s], r1 = a.q_start[s + 1];
        // a drafting model's row is read for the draft behind it
        if (r0 >= 0 && r0 <= row && row + (draft ? 1 : 0) < r1 && r1 <= a.T) s_seq = s;
    }
    __syncthreads();
    const int s = s_seq;
    if (s < 0) return;               // the whole cluster
    const Temp temp = temp_of(a, s);
    if (temp.bad || (draft && temp.greedy)) return;

    const Row<L> rw(draft ? a.draft : a.logits, draft ? a.ld_draft : a.ld, row, a.V);
    const int v0 = static_cast<int>(static_cast<long long>(rw.n) * part / parts), v1 = static_cast<int>(static_cast<long long>(rw.n) * (part + 1) / parts);
    uint4 held[kHeld];
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
        if (v0 + tid + i * kThreads < v1) held[i] = __ldg(rw.runs + v0 + tid + i * kThreads);
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
        RowInfo r;
        long long z = 0;
        for (int i = 0; i < parts; ++i) { z += s_part_sum[i]; best = min(best, s_part_best[i]); }
        r.z = static_cast<unsigned long long>(z);
        r.m = m;
        r.best = best;
        r.bad = bad;
        r.pad[0] = r.pad[1] = r.pad[2] = 0;
        a.rows[item] = r;
    }
}

// What the tokens of the row behind the last accepted draft weigh for the draw.
template <typename L>
struct Draw {
    Row<L> p, q;
    Scale sp, sq;
    float ip, iq;
    int mode, without;               // mode 0: the target's weights, 1: those but for one token, 2: max(p - q, 0)
    static constexpr int E = Run<L>::E;
    // the weights of a run's numbers two by two; 0 (or less than half a unit) outside the row
    template <typename F>
    __device__ __forceinline__ void run(int v, F use) const {
        const int e = p.first(v);
        const uint4 x = mask_run(p, __ldg(p.runs + v), v);
        uint4 y = make_uint4(0u, 0u, 0u, 0u);
        if (mode == 2) {
            if (q.off == p.off) {
                y = mask_run(q, __ldg(q.runs + v), v);
            } else {
                uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    if (e + i < 0 || e + i >= p.V) continue;
                    if constexpr (sizeof(L) == 4) w[i] = __float_as_uint(load_one<L>(q.runs, q.off + e + i));
                    else w[i / 2] |= (__float_as_uint(load_one<L>(q.runs, q.off + e + i)) >> 16) << (16 * (i & 1));
                }
                y = make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
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

template <typename L>
__global__ void __launch_bounds__(kThreads) verify_draw_kernel(const VerifyArgs a) {
    constexpr int E = Run<L>::E;
    cg::cluster_group cluster = cg::this_cluster();
    const int parts = static_cast<int>(cluster.num_blocks()), part = static_cast<int>(cluster.block_rank());
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    __shared__ int s_stop, s_bad;
    __shared__ long long s_sums[2][kMaxCluster * kWarps];
    const int s = blockIdx.x / parts;
    if (tid == 0) { s_stop = 0x7fffffff; s_bad = 0; }
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
    // every CTA judges the drafts for itself
    for (int j = tid; j < n; j += kThreads) {
        const RowInfo ri = a.rows[r0 + j];
        if (ri.bad) s_bad = 1;
        if (j == n - 1) continue;
        const int x = a.tokens[r0 + j + 1];
        if (x < 0 || x >= a.V) {
            s_bad = 1;
            if (part == 0) report(a.st, MOE_DEV_BAD_INDEX, r0 + j + 1);
            continue;
        }
        bool ok;
        if (temp.greedy) {
            ok = x == ri.best;
        } else {
            double q = 1.0;
            if (a.draft != nullptr) {
                const RowInfo rq = a.rows[a.T + r0 + j];
                if (rq.bad) { s_bad = 1; continue; }
                const float l = load_one<L>(a.draft, (r0 + j) * a.ld_draft + x);
                q = __ll2double_rn(units_of(weight(l, Scale(rq.m, temp.it)))) / __ll2double_rn(static_cast<long long>(rq.z));
            }
            if (ri.bad) continue;
            const float l = load_one<L>(a.logits, (r0 + j) * a.ld + x);
            const double p = __ll2double_rn(units_of(weight(l, Scale(ri.m, temp.it)))) / __ll2double_rn(static_cast<long long>(ri.z));
            ok = __dmul_rn(static_cast<double>(a.uniform[r0 + j + 1]), q) < p;
        }
        if (!ok) atomicMin(&s_stop, j);
    }
    __syncthreads();
    if (s_bad) {
        if (lead) answer(0, -1);
        return;
    }
    const int stop = min(s_stop, n - 1);
    const int row = r0 + stop;
    const RowInfo ri = a.rows[row];
    if (temp.greedy) {
        if (lead) answer(stop, ri.best);
        return;
    }
    Draw<L> d = {Row<L>(a.logits, a.ld, row, a.V), Row<L>(a.logits, a.ld, row, a.V), Scale(ri.m, temp.it), Scale(0.f, temp.it), 0.f, 0.f, 0, -1};
    if (stop < n - 1) {
        d.mode = 1;
        d.without = a.tokens[row + 1];
        if (a.draft != nullptr) {
            const RowInfo rq = a.rows[a.T + row];
            d.mode = 2;
            d.q = Row<L>(a.draft, a.ld_draft, row, a.V);
            d.sq = Scale(rq.m, temp.it);
            d.ip = __double2float_rn(0x1p42 / __ll2double_rn(static_cast<long long>(ri.z)));
            d.iq = __double2float_rn(0x1p42 / __ll2double_rn(static_cast<long long>(rq.z)));
        }
    }
    // a warp's runs are neighbours, so that the warps' sums are the cumulated weight in order
    const int warps = parts * kWarps, w = part * kWarps + warp;
    const int v0 = static_cast<int>(static_cast<long long>(d.p.n) * w / warps), v1 = static_cast<int>(static_cast<long long>(d.p.n) * (w + 1) / warps);
    long long total = 0, before = 0, own = 0;
    for (int turn = 0; turn < 2; ++turn) {
        Units u;
        for (int v = v0 + lane; v < v1; v += 32) d.run(v, [&](int, float2 x) { u.add(x); });
        own = warp_sum(u.sum());
        if (lane < parts) cluster.map_shared_rank(s_sums[turn], lane)[w] = own;
        cluster.sync();
        // all of them, and those of the warps before
        total = before = 0;
        for (int i = lane; i < warps; i += 32) {
            const long long v = s_sums[turn][i];
            total += v;
            if (i < w) before += v;
        }
        total = warp_sum(total);
        before = warp_sum(before);
        if (total > 0) break;        // the same in every CTA
        d.mode = 0;                  // nothing of the target is beyond the draft
    }
    long long target = __double2ll_rd(__dmul_rn(static_cast<double>(a.uniform[r0]), __ll2double_rn(total)));
    target = max(0ll, min(target, total - 1));
    if (lead) {
        a.accepted[s] = stop;
        if (a.n_new != nullptr) a.n_new[s] = stop - (n - 1);
    }
    if (target < before || target >= before + own) return;
    // this warp's runs hold the token
    for (int v = v0; v < v1; v += 32) {
        long long u[E], mine = 0;
#pragma unroll
        for (int i = 0; i < E; ++i) u[i] = 0;
        if (v + lane < v1) {
            d.run(v + lane, [&](int i, float2 x) {
                u[i] = units_of(x.x);
                u[i + 1] = units_of(x.y);
            });
#pragma unroll
            for (int i = 0; i < E; ++i) mine += u[i];
        }
        long long inc = mine;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long o = __shfl_up_sync(kFull, inc, off);
            if (lane >= off) inc += o;
        }
        const long long all = __shfl_sync(kFull, inc, 31);
        if (target < before + all) {
            long long c = before + inc - mine;
            if (target >= c && target < c + mine)
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    if (target >= c && target < c + u[i]) a.next[s] = d.p.first(v + lane) + i;
                    c += u[i];
                }
            return;
        }
        before += all;
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

template <typename L>
cudaError_t launch(const VerifyArgs& a, cudaStream_t s) {
    const int runs = a.V / Run<L>::E + 2;
    int parts = 1;
    while (parts < kMaxCluster && runs > parts * kThreads * kHeld / 2) parts *= 2;
    if (a.T > 0) {
        const cudaError_t e = launch_clusters(verify_rows_kernel<L>, a.draft != nullptr ? 2 * a.T : a.T, parts, s, a);
        if (e != cudaSuccess) return e;
    }
    return launch_clusters(verify_draw_kernel<L>, a.S, parts, s, a);
}

}  // namespace

size_t verify_workspace(int T) { return 2 * static_cast<size_t>(T) * sizeof(RowInfo); }

cudaError_t launch_verify(const void* logits, int dtype, long long ld, int T, int V, const int32_t* tokens, const float* uniform,
                          const int32_t* q_start, int S, const void* draft, long long ld_draft, const float* temperature, int32_t* accepted,
                          int32_t* next, int32_t* n_new, void* ws, moe_dev_status* st, cudaStream_t s) {
    const VerifyArgs a = {logits, draft, ld, ld_draft, T, V, S, tokens, q_start, uniform, temperature, accepted, next, n_new, static_cast<RowInfo*>(ws), st};
    return dtype == MOE_DTYPE_BF16 ? launch<__nv_bfloat16>(a, s) : launch<float>(a, s);
}

}  // namespace moe
