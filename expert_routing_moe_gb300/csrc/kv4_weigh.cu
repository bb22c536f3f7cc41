// kv4_weigh.cu -- the attention weight that cached tokens draw (moe_kv4_weigh):
//     score[j] += sum over rows i and heads h of exp(scale * q_i . k_j - lse[i][h])
//
// Few rows (prompts: kv4_weigh_tc.cu).  A warp takes a page and a key head, its
// CTA as many pages at a time as it has warps for their heads.  Scores come
// from m16n8k16 products with the cached keys as the 16-row operand, as in the
// attention over few rows; a lane adds up the probabilities of its eight tokens
// over all rows that it sees, so that only one sum a token is left to add
// across lanes and warps, in a fixed order.  The pages of all sequences are cut
// into equal runs for a grid of two CTAs an SM, and up to 16 rows stay
// in registers over a run (KEEP): a step of 32 sequences of up to 8192 tokens,
// 32 + 4 heads of 128, took 14.7 us with a CTA a page, which loads the rows again
// for every page, and takes 7.5; one of 131071 tokens 21.8 and 13.5 (38 MB of
// keys: 2.8 TB/s).  What bounds it is the turning of codes into fp16 and the
// latency of a page's chain from table to sum, not the bytes.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kv4_weigh.cuh"
#include "launch.h"
#include "tmap.h"

namespace moe {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// NT times eight query rows as fragments: row 8 i + g of them, numbers (D/4) t + 4 ks + 0..3, scaled by a power of two
// that puts the row's largest magnitude into [2^10, 2^11) (see the streaming attention); and for the lane's
// rows 8 i + 2 t + c the scores' factor, -lse in powers of two, and the place (-1: it adds nothing).
template <int D, int NT>
struct Queries {
    uint32_t f[NT][D / 16][2];
    float up[NT][2], z[NT][2];
    int place[NT][2];
};
template <int D, int NT>
__device__ __forceinline__ void load_rows(Queries<D, NT>& w, const WeighArgs& a, const WeighSeq& s, int h, int r_first, int r_end, int lane, float k_scale) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int r = r_first + 8 * i + g;
        const bool live = r < r_end;
        uint32_t raw[D / 8];
#pragma unroll
        for (int x = 0; x < D / 8; ++x) raw[x] = 0u;
        float lse = -INFINITY;
        if (live) {
            const long long row = s.q0 + r / a.group;
            const int head = h * a.group + r % a.group;
            const __nv_bfloat16* p = a.q + row * a.ld_q + static_cast<long long>(head) * D + (D / 4) * t;
            lse = a.lse[row * a.n_q + head];
#pragma unroll
            for (int x = 0; x < D / 32; ++x) {
                const uint4 v = reinterpret_cast<const uint4*>(p)[x];
                raw[4 * x] = v.x; raw[4 * x + 1] = v.y; raw[4 * x + 2] = v.z; raw[4 * x + 3] = v.w;
            }
        }
        const bool none = lse == -INFINITY;
        float top = 0.f;
#pragma unroll
        for (int x = 0; x < D / 8; ++x)
            top = fmaxf(top, fmaxf(fabsf(__uint_as_float(raw[x] << 16)), fabsf(__uint_as_float(raw[x] & 0xffff0000u))));
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
        int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
        e = (top > 0.f && e < 128) ? max(-100, min(100, 10 - e)) : 0;
        const float up = __int_as_float((e + 127) << 23);
        const float factor = none ? 0.f : a.scale * kLog2e * k_scale * __int_as_float((127 - e) << 23);
        const float z = none ? -INFINITY : lse * -kLog2e;
        const int place = none ? -1 : s.base() + r / a.group;
#pragma unroll
        for (int x = 0; x < D / 8; ++x)
            w.f[i][x / 2][x & 1] = none ? 0u : pack_f16(__uint_as_float(raw[x] << 16) * up, __uint_as_float(raw[x] & 0xffff0000u) * up);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            w.up[i][c] = __shfl_sync(kFull, factor, (2 * t + c) * 4);
            w.z[i][c] = __shfl_sync(kFull, z, (2 * t + c) * 4);
            w.place[i][c] = __shfl_sync(kFull, place, (2 * t + c) * 4);
        }
    }
}

// A lane's part of a head's keys of a page: tokens 8 i + g (i < 8), numbers (D/4) t .. + D/4 - 1.
template <int D>
struct Keys {
    uint32_t c[8][D / 32];
    uint32_t s[D == 128 ? 4 : 2];
};
template <int D>
__device__ __forceinline__ void load_keys(Keys<D>& k, const uint8_t* base, int lane) {
    using L = Kv4Layout<D>;
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint8_t* p = base + (8 * i + g) * (D / 2) + t * (D / 8);
        if constexpr (D == 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(p);
            k.c[i][0] = v.x; k.c[i][1] = v.y; k.c[i][2] = v.z; k.c[i][3] = v.w;
        } else {
            const uint2 v = *reinterpret_cast<const uint2*>(p);
            k.c[i][0] = v.x; k.c[i][1] = v.y;
        }
    }
    const uint8_t* p = base + L::kScales + (t * 8 + g) * 8 * L::R;
    if constexpr (D == 128) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        k.s[0] = v.x; k.s[1] = v.y; k.s[2] = v.z; k.s[3] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2*>(p);
        k.s[0] = v.x; k.s[1] = v.y;
    }
}
// Adds the probabilities of the lane's tokens over its rows.
template <int D, int NT>
__device__ __forceinline__ void add_page(float (&sum)[8], const Keys<D>& k, const Queries<D, NT>& w, int key0, unsigned span, int lane) {
    using L = Kv4Layout<D>;
    const int g = lane >> 2;
    constexpr int W = D / 32;
    bool edge = false;                          // a row does not see all of the page
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) edge |= w.place[n][c] < key0 + kPage - 1 || static_cast<unsigned>(w.place[n][c] - key0) >= span;
    edge = __any_sync(kFull, edge);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
        float acc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[n][c] = 0.f;
        uint32_t s0[L::R], s1[L::R];            // scales of tokens 16 m + g and 16 m + 8 + g
        if constexpr (L::R == 2) {
            const uint32_t x = e4m3x2_to_f16(k.s[m] & 0xffffu), y = e4m3x2_to_f16(k.s[m] >> 16);
            s0[0] = __byte_perm(x, 0, 0x1010); s0[1] = __byte_perm(x, 0, 0x3232);
            s1[0] = __byte_perm(y, 0, 0x1010); s1[1] = __byte_perm(y, 0, 0x3232);
        } else {
            const uint32_t x = e4m3x2_to_f16((k.s[m / 2] >> (16 * (m & 1))) & 0xffffu);
            s0[0] = __byte_perm(x, 0, 0x1010);
            s1[0] = __byte_perm(x, 0, 0x3232);
        }
#pragma unroll
        for (int k2 = 0; k2 < W; ++k2) {
            uint32_t x[4], y[4];
            e2m1x8_to_f16(k.c[2 * m][k2], x[0], x[1], x[2], x[3]);
            e2m1x8_to_f16(k.c[2 * m + 1][k2], y[0], y[1], y[2], y[3]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int ks = 2 * k2 + e, r = ks / 4;
                const uint32_t af[4] = {hmul2_u(x[2 * e], s0[r]), hmul2_u(y[2 * e], s1[r]), hmul2_u(x[2 * e + 1], s0[r]), hmul2_u(y[2 * e + 1], s1[r])};
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_f16(acc[n], af, w.f[n][ks][0], w.f[n][ks][1]);
            }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int key = key0 + 16 * m + 8 * i + g;
                    float x = ex2(fmaf(acc[n][2 * i + c], w.up[n][c], w.z[n][c]));
                    if (edge) x = static_cast<unsigned>(w.place[n][c] - key) < span ? x : 0.f;
                    sum[2 * m + i] += x;
                }
    }
}

// A CTA takes pages of one sequence, as many at a time as eight warps have when each takes a key head (a warp takes several
// where there are more than eight).  KEEP: no sequence has more than 8 NT rows a key head, and there are no more than eight key heads:
// the rows stay in registers over all pages.
//
// A step is as many pages as fit at once; the steps of all sequences are one row, cut into equal runs for the CTAs.
template <int D, int NT, bool KEEP>
__global__ void __launch_bounds__(kThreads, KEEP ? 2 : 1) kv4_weigh_kernel(const WeighArgs a) {
    using L = Kv4Layout<D>;
    __shared__ float s_sum[2][kWarps][kPage];
    __shared__ int s_scan[kWarps], s_seq, s_at, s_steps;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int per = min(a.c.n_kv, kWarps), at_once = kWarps / per;     // warps of a page, pages at a time
    const int which = warp / per, h0 = warp % per;
    const bool busy = which < at_once;
    const unsigned span = a.window > 0 ? a.window : 0x7fffffff;        // places from a key's own on that see it
    pdl_wait();
    pdl_trigger();
    auto steps_of = [&](const WeighSeq& q) {
        if (q.n == 0 || q.len == 0 || (q.n - q.i0) * a.group >= a.many) return 0;
        return (pages_of(q.len) - weigh_first(a, q) / kPage + at_once - 1) / at_once;
    };
    // Every CTA adds up the steps for itself (a 32-bit number: the pages fit the device's memory), and with few sequences every warp:
    // a lane is one.
    const bool few = a.c.S <= 32;
    const int each = few ? 1 : (a.c.S + kThreads - 1) / kThreads, me = few ? lane : tid;
    const int sa = min(a.c.S, me * each), sb = min(a.c.S, sa + each);
    int mine = 0;
    WeighSeq q = {0, 0, 0, 0, true};
    for (int s = sa; s < sb; ++s) {
        q = weigh_seq(a, s);
        if (!q.fit && blockIdx.x == 0 && (!few || warp == 0)) report(a.st, MOE_DEV_BAD_INDEX, s);
        mine += steps_of(q);
    }
    int inc = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int v = __shfl_up_sync(kFull, inc, off);
        if (lane >= off) inc += v;
    }
    int before = inc - mine, total = __shfl_sync(kFull, inc, 31);
    if (!few) {
        if (lane == 31) s_scan[warp] = inc;
        __syncthreads();
        total = 0;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            if (i < warp) before += s_scan[i];
            total += s_scan[i];
        }
    }
    // (one sequence: every gridDim.x-th step; 131071 tokens took 13.4 us so, and 15.0 in runs)
    const bool one = a.c.S == 1;
    const int hop = one ? static_cast<int>(gridDim.x) * at_once : at_once;
    int u = one ? static_cast<int>(blockIdx.x) : static_cast<int>(static_cast<long long>(total) * blockIdx.x / gridDim.x);
    const int u1 = one ? total : static_cast<int>(static_cast<long long>(total) * (blockIdx.x + 1) / gridDim.x);
    const WeighSeq own = q;
    int buf = 0;
    while (u < u1) {
        int s, at, steps;
        if (few) {
            s = __ffs(__ballot_sync(kFull, u >= before && u < before + mine)) - 1;
            q.q0 = __shfl_sync(kFull, own.q0, s);
            q.n = __shfl_sync(kFull, own.n, s);
            q.len = __shfl_sync(kFull, own.len, s);
            q.i0 = __shfl_sync(kFull, own.i0, s);
            at = u - __shfl_sync(kFull, before, s);
            steps = __shfl_sync(kFull, mine, s);
        } else {
            // the sequence of step u is found by the thread that added it up
            if (u >= before && u < before + mine) {
                int b = before;
                for (int x = sa; x < sb; ++x) {
                    const int n = each == 1 ? mine : steps_of(weigh_seq(a, x));
                    if (u < b + n) {
                        s_seq = x;
                        s_at = u - b;
                        s_steps = n;
                        break;
                    }
                    b += n;
                }
            }
            __syncthreads();             // (s_seq is written again only after the barriers of this sequence's steps)
            s = s_seq;
            at = s_at;
            steps = s_steps;
            q = weigh_seq(a, s);
        }
        steps = one ? (total - u + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x) : min(steps - at, u1 - u);
        const int pages = pages_of(q.len), first = weigh_first(a, q) / kPage + at * at_once;
        const int32_t* table = a.c.page_table + static_cast<long long>(s) * a.c.max_pages;
        Queries<D, NT> w;
        int next = busy && first + which < pages ? table[first + which] : -1;
        if (KEEP && busy) load_rows<D, NT>(w, a, q, h0, q.i0 * a.group, q.n * a.group, lane, a.c.k_scale != nullptr ? a.c.k_scale[h0] : 1.f);
        for (int i = 0; i < steps; ++i, buf ^= 1) {
            const int page = first + i * hop + which, id = next;
            const bool there = busy && page < pages, ok = there && id >= 0 && id < a.c.n_pages;
            next = busy && i + 1 < steps && page + hop < pages ? table[page + hop] : -1;
            if (there && !ok && h0 == 0 && lane == 0) report(a.st, MOE_DEV_BAD_INDEX, id);
            const int key0 = page * kPage;
            float sum[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) sum[k] = 0.f;
            if (ok) {
                const uint8_t* base = static_cast<const uint8_t*>(a.c.pages) + static_cast<long long>(id) * a.c.n_kv * L::bytes;
                if constexpr (KEEP) {
                    Keys<D> k;
                    load_keys<D>(k, base + h0 * L::bytes, lane);
                    add_page<D, NT>(sum, k, w, key0, span, lane);
                } else {
                    int ia, ib;
                    weigh_rows(a, q, key0, kPage, ia, ib);
                    for (int h = h0; h < a.c.n_kv; h += per) {
                        Keys<D> k;
                        load_keys<D>(k, base + h * L::bytes, lane);
                        for (int r = ia * a.group; r < ib * a.group; r += 8 * NT) {
                            load_rows<D, NT>(w, a, q, h, r, ib * a.group, lane, a.c.k_scale != nullptr ? a.c.k_scale[h] : 1.f);
                            add_page<D, NT>(sum, k, w, key0, span, lane);
                        }
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                sum[k] += __shfl_xor_sync(kFull, sum[k], 1);
                sum[k] += __shfl_xor_sync(kFull, sum[k], 2);
                if (t == 0) s_sum[buf][warp][8 * k + g] = sum[k];
            }
            __syncthreads();             // (the other buffer is read no more when its next sums come)
            // the warps' sums in the order of the heads: two tokens a lane of each page's first warp
            if (h0 == 0 && ok) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int tok = lane + 32 * k;
                    if (key0 + tok < q.len) {
                        float v = 0.f;
                        for (int j = 0; j < per; ++j) v += s_sum[buf][warp + j][tok];
                        weigh_add(a, q, s, key0 + tok, v);
                    }
                }
            }
        }
        if (one) break;
        u += steps;
    }
}

template <int D, int NT, bool KEEP>
cudaError_t launch(const WeighArgs& a, cudaStream_t s) {
    return launch_pdl(kv4_weigh_kernel<D, NT, KEEP>, dim3((KEEP ? 2 : 1) * sm_count()), dim3(kThreads), 0, s, a);
}
template <int D>
cudaError_t launch(const WeighArgs& a, long long rows, cudaStream_t s) {
    if (rows > 16 || a.c.n_kv > kWarps) return launch<D, 2, false>(a, s);
    return rows <= 8 ? launch<D, 1, true>(a, s) : launch<D, 2, true>(a, s);
}

}  // namespace

size_t kv4_weigh_workspace(int S, int T, int n_q, int n_kv, int D, int max_pages) {
    (void)D;
    const int group = n_q / n_kv;
    return static_cast<long long>(T) * group >= kWeighMany && weigh_tc_fits(group) ? kv4_weigh_tc_workspace(S, max_pages) : 0;
}

cudaError_t launch_kv4_weigh(const void* q, long long ld_q, int T, int n_q, const moe_kv4_cache& c, const int32_t* q_start, int max_new,
                             const float* lse, float scale, int window, int last, float* score, long long ld_score, bool fresh, void* ws,
                             moe_dev_status* st, cudaStream_t s) {
    if (c.max_pages < 1) return cudaSuccess;
    const int group = n_q / c.n_kv;
    long long most = max_new < T ? max_new : T;        // rows of a sequence that count
    if (last > 0 && last < most) most = last;
    const bool prompts = most * group >= kWeighMany && weigh_tc_fits(group);
    // where sequences have many rows on average all go there (the last 64 rows of 6 chunks of 500: a launch less, 22.7 -> 20.6 us with the
    // host's part); one prompt among many single tokens does not take them along
    const bool all = prompts && static_cast<long long>(T) * group >= static_cast<long long>(kWeighMany) * c.S;
    const WeighArgs a = {static_cast<const __nv_bfloat16*>(q), ld_q, T, n_q, group, c, q_start, lse, scale, window, last, max_new, score, ld_score, fresh,
                         all ? 1 : prompts ? kWeighMany : 0x7fffffff, st};
    if (prompts) {
        const cudaError_t e = launch_kv4_weigh_tc(a, ws, s);
        if (e != cudaSuccess || all) return e;
    }
    return c.head_dim == 64 ? launch<64>(a, most * group, s) : launch<128>(a, most * group, s);
}

}  // namespace moe
