// kv4_evict.cu -- eviction from the 4-bit cache by the tokens' scores
// (moe_kv4_evict): three launches.
//
//  select  a CTA for each sequence finds the score that a token needs (a radix
//          select over the scores' bits, eight at a time) and lists the kept
//          tokens in order
//  plan    one CTA gives every sequence its free pages, all or nothing
//  move    tables, references, lengths and scores, a CTA for each sequence; and
//          the kept tokens' codes and scales, a CTA for each (layer, head,
//          sequence)
//
// Moving in place: the k-th kept token comes from a place >= k, so a page is read
// only for itself and for pages before it.  A CTA reads the sources of
// eight pages, then writes them: whatever it writes has been read by then.
#include "common.cuh"
#include "kv4.cuh"
#include "launch.h"
#include "ranges.h"
#include "tmap.h"

namespace moe {

namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMoveThreads = 256;
constexpr int kMoveWarps = kMoveThreads / 32;

// What is known of a sequence.
struct SeqPlan {
    int32_t len, now;        // tokens before and after; now = len: it stays
    int32_t first;           // page of the first token that goes
    int32_t fresh;           // free pages that it takes
    int32_t base;            // the first of them, among those handed out
    int32_t bad;             // it cannot be done
    int32_t pad[2];
};
struct EvictWs {
    int* header;             // [0] the plan stands
    SeqPlan* seqs;           // [S]
    int* free_pages;         // [n_pages] those handed out, ascending
    int* old_page;           // [S][max_pages] the tables as they were
    int* rank;               // [S][max_pages] which of its free pages a page is written to, -1: itself
    int* kept;               // [S][max_pages * 64] places of the kept tokens
};
__host__ __device__ inline EvictWs evict_ws(void* ws, int S, int max_pages, int n_pages) {
    EvictWs w;
    w.header = static_cast<int*>(ws);
    w.seqs = reinterpret_cast<SeqPlan*>(w.header + 64);
    w.free_pages = reinterpret_cast<int*>(w.seqs + S);
    w.old_page = w.free_pages + n_pages;
    w.rank = w.old_page + static_cast<long long>(S) * max_pages;
    w.kept = w.rank + static_cast<long long>(S) * max_pages;
    return w;
}

struct EvictArgs {
    moe_kv4_pool p;
    int n_kv;
    float* score;
    long long ld_score;
    const int32_t* budget;
    int sinks, recent;
    int32_t* kept;
    long long ld_kept;
    void* ws;
    moe_dev_status* st;
};

// Scores as whole numbers in the same order; a NaN is the lowest, and -0 is 0.
__device__ __forceinline__ uint32_t order_of(float x) {
    if (x != x) return 0u;
    const uint32_t b = __float_as_uint(x + 0.f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Exclusive prefix sum over the CTA, and the total.
__device__ __forceinline__ int scan(int v, int& total, int* s_warp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int x = __shfl_up_sync(kFull, inc, off);
        if (lane >= off) inc += x;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    int w = s_warp[lane];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int x = __shfl_up_sync(kFull, w, off);
        if (lane >= off) w += x;
    }
    total = __shfl_sync(kFull, w, 31);
    const int before = __shfl_sync(kFull, w, max(warp - 1, 0));
    return (warp > 0 ? before : 0) + inc - v;
}

__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(const EvictArgs a) {
    __shared__ int s_hist[256], s_warp[kSelWarps], s_pick[2], s_first, s_bad;
    const int s = blockIdx.x, tid = threadIdx.x;
    const EvictWs w = evict_ws(a.ws, a.p.S, a.p.max_pages, a.p.n_pages);
    if (tid == 0) { s_first = 0x7fffffff; s_bad = 0; }
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    const int len = a.p.seq_len[s], budget = a.budget[s];
    const long long most = min(static_cast<long long>(a.p.max_pages) * kPage, 0x7fffffffll);
    SeqPlan r = {len, len, 0, 0, 0, 0, {0, 0}};
    const bool bad_len = len < 0 || len > most;
    const int pages = bad_len ? 0 : pages_of(len);
    const bool cut = !bad_len && budget >= 0 && budget < len;
    bool bad = bad_len || (cut && static_cast<long long>(a.sinks) + a.recent > budget);
    const int32_t* row = a.p.page_table + static_cast<long long>(s) * a.p.max_pages;
    int* old_page = w.old_page + static_cast<long long>(s) * a.p.max_pages;
    if (cut)
        for (int c = tid; c < pages; c += kSelThreads) {
            const int id = row[c];
            if (id < 0 || id >= a.p.n_pages) s_bad = 1;
            old_page[c] = id;
        }
    __syncthreads();
    bad = bad || s_bad;
    if (bad || !cut) {
        r.bad = bad;
        if (tid == 0) w.seqs[s] = r;
        return;
    }
    // the best k of the places between the first and the last ones
    const int lo = a.sinks, hi = len - a.recent, k = budget - a.sinks - a.recent;
    const float* score = a.score + s * a.ld_score;
    uint32_t prefix = 0u;
    int want = k;                       // of those whose higher bits are the prefix's
    for (int shift = 24; shift >= 0 && k > 0; shift -= 8) {
        for (int i = tid; i < 256; i += kSelThreads) s_hist[i] = 0;
        __syncthreads();
        for (int j = lo + tid; j < hi; j += kSelThreads) {
            const uint32_t o = order_of(score[j]);
            if (shift == 24 || (o >> (shift + 8)) == (prefix >> (shift + 8))) atomicAdd(&s_hist[(o >> shift) & 255u], 1);
        }
        __syncthreads();
        int total;
        const int mine = tid < 256 ? s_hist[255 - tid] : 0;      // from the highest down
        const int before = scan(mine, total, s_warp);
        if (tid < 256 && before < want && before + mine >= want) {
            s_pick[0] = 255 - tid;
            s_pick[1] = before;
        }
        __syncthreads();
        prefix |= static_cast<uint32_t>(s_pick[0]) << shift;
        want -= s_pick[1];
        __syncthreads();
    }
    // prefix: the score of the last one that is kept; `want` of those that have it are, the first ones
    int* kept = w.kept + static_cast<long long>(s) * a.p.max_pages * kPage;
    int n_kept = 0, n_equal = 0;
    for (int j0 = 0; j0 < len; j0 += kSelThreads) {
        const int j = j0 + tid;
        bool keep = j < len && (j < lo || j >= hi), equal = false;
        if (j >= lo && j < hi && k > 0) {
            const uint32_t o = order_of(score[j]);
            keep = o > prefix;
            equal = o == prefix;
        }
        int total;
        const int e = scan(equal, total, s_warp);
        if (equal && n_equal + e < want) keep = true;
        n_equal += total;
        const int at = n_kept + scan(keep, total, s_warp);
        n_kept += total;
        if (keep) kept[at] = j;
        else if (j < len && j < s_first) atomicMin(&s_first, j);
    }
    __syncthreads();
    r.now = n_kept;
    r.first = s_first / kPage;
    // pages that others hold too are written elsewhere
    int* rank = w.rank + static_cast<long long>(s) * a.p.max_pages;
    for (int c0 = r.first; c0 < pages_of(r.now); c0 += kSelThreads) {
        const int c = c0 + tid;
        const bool in = c < pages_of(r.now);
        const bool shared = in && a.p.ref[row[c]] > 1;
        int total;
        const int at = r.fresh + scan(shared, total, s_warp);
        if (in) rank[c] = shared ? at : -1;
        r.fresh += total;
    }
    if (tid == 0) w.seqs[s] = r;
}

__global__ void __launch_bounds__(kSelThreads, 1) evict_plan_kernel(const EvictArgs a) {
    __shared__ int s_warp[kSelWarps];
    const EvictWs w = evict_ws(a.ws, a.p.S, a.p.max_pages, a.p.n_pages);
    __shared__ int s_bad;
    const int tid = threadIdx.x;
    if (tid == 0) s_bad = 0x7fffffff;
    pdl_wait();
    pdl_trigger();
    __syncthreads();
    int want = 0;
    for (int s0 = 0; s0 < a.p.S; s0 += kSelThreads) {
        const int s = s0 + tid;
        int total;
        const int mine = s < a.p.S ? w.seqs[s].fresh : 0;
        if (s < a.p.S && w.seqs[s].bad) atomicMin(&s_bad, s);
        const int at = scan(mine, total, s_warp);
        if (s < a.p.S) w.seqs[s].base = want + at;
        want += total;
    }
    int have = 0;
    for (int g0 = 0; g0 < a.p.n_pages && have < want; g0 += kSelThreads) {
        const int g = g0 + tid;
        const bool is_free = g < a.p.n_pages && a.p.ref[g] == 0;
        int total;
        const int at = have + scan(is_free, total, s_warp);
        if (is_free && at < want) w.free_pages[at] = g;
        have += total;
    }
    __syncthreads();
    if (tid == 0) {
        const bool bad = s_bad != 0x7fffffff;
        w.header[0] = !bad && have >= want;
        if (bad) report(a.st, MOE_DEV_BAD_INDEX, s_bad);
        else if (have < want) report(a.st, MOE_DEV_NO_PAGES, want - have);
    }
}

// Tables, references, lengths and scores of sequence s.
__device__ __forceinline__ void move_book(const EvictArgs& a, const EvictWs& w, int s) {
    const SeqPlan r = w.seqs[s];
    const int tid = threadIdx.x;
    const int* kept = w.kept + static_cast<long long>(s) * a.p.max_pages * kPage;
    const bool cut = r.now < r.len;
    if (a.kept != nullptr)
        for (long long i = tid; i < a.ld_kept; i += kMoveThreads) a.kept[s * a.ld_kept + i] = i >= r.now ? -1 : cut ? kept[i] : static_cast<int>(i);
    if (!cut) return;
    float* score = a.score + s * a.ld_score;
    // a score moves to a place at or before its own: what is written has been read
    for (int i0 = 0; i0 < r.len; i0 += kMoveThreads * 4) {
        float v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + u * kMoveThreads + tid;
            v[u] = i < r.now ? score[kept[i]] : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int i = i0 + u * kMoveThreads + tid;
            if (i < r.len) score[i] = v[u];
        }
    }
    int32_t* row = a.p.page_table + static_cast<long long>(s) * a.p.max_pages;
    const int* old_page = w.old_page + static_cast<long long>(s) * a.p.max_pages;
    const int* rank = w.rank + static_cast<long long>(s) * a.p.max_pages;
    const int after = pages_of(r.now);
    for (int c = r.first + tid; c < pages_of(r.len); c += kMoveThreads) {
        if (c >= after) {
            atomicSub(&a.p.ref[old_page[c]], 1);
            row[c] = -1;
        } else if (rank[c] >= 0) {
            const int g = w.free_pages[r.base + rank[c]];
            atomicSub(&a.p.ref[old_page[c]], 1);
            a.p.ref[g] = 1;
            row[c] = g;
        }
    }
    if (tid == 0) a.p.seq_len[s] = r.now;
}

// The kept tokens of page c of (layer, head, sequence), read by one warp into registers and written from them.
// A lane reads and writes 16-byte runs of the page that it makes, but for the scales' sources.
template <int D>
struct Page {
    using L = Kv4Layout<D>;
    static constexpr int KC = kPage * D / 2 / 512;       // 16-byte runs of key codes of a lane
    static constexpr int VC = KC;                        // and of value codes
    uint4 k[KC], va[VC];
    uint32_t ks[L::R == 2 ? 4 : 2], vs[4];
};

template <int D>
__device__ __forceinline__ void read_page(Page<D>& g, const uint8_t* head, long long page_bytes, const int* kept, const int* old_page, int c, int now, int lane) {
    using L = Kv4Layout<D>;
    // lane's two tokens of the page and the pages that hold them
    int src[2];
    const uint8_t* from[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const int i = c * kPage + 2 * lane + u;
        src[u] = i < now ? kept[i] : -1;
        from[u] = src[u] < 0 ? nullptr : head + old_page[src[u] / kPage] * page_bytes;
    }
    auto token = [&](int tok, const uint8_t*& base, int& t) {       // of another lane
        const int l = tok >> 1;
        const int s0 = __shfl_sync(kFull, src[0], l), s1 = __shfl_sync(kFull, src[1], l);
        const unsigned long long b0 = __shfl_sync(kFull, reinterpret_cast<unsigned long long>(from[0]), l);
        const unsigned long long b1 = __shfl_sync(kFull, reinterpret_cast<unsigned long long>(from[1]), l);
        const int v = tok & 1 ? s1 : s0;
        base = reinterpret_cast<const uint8_t*>(tok & 1 ? b1 : b0);
        t = v & (kPage - 1);
    };
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    // key codes: D/32 runs a token
    constexpr int per = D / 32;
#pragma unroll
    for (int x = 0; x < Page<D>::KC; ++x) {
        const int run = x * 32 + lane;
        const uint8_t* b;
        int t;
        token(run / per, b, t);
        g.k[x] = b == nullptr ? zero : *reinterpret_cast<const uint4*>(b + t * (D / 2) + run % per * 16);
    }
    // key scales: R bytes of tokens g + 8 i (i < 8), block t: place (t*8 + g)*8 + i
    {
#pragma unroll
        for (int x = 0; x < (L::R == 2 ? 4 : 2); ++x) g.ks[x] = 0u;
        const int gg = lane & 7, tt = lane >> 3;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint8_t* b;
            int t;
            token(gg + 8 * i, b, t);
            if (L::R == 2) {
                const uint32_t v = b == nullptr ? 0u : *reinterpret_cast<const uint16_t*>(b + L::kScales + ((tt * 8 + t % 8) * 8 + t / 8) * 2);
                g.ks[i / 2] |= v << (16 * (i & 1));
            } else {
                const uint32_t v = b == nullptr ? 0u : b[L::kScales + (tt * 8 + t % 8) * 8 + t / 8];
                g.ks[i / 4] |= v << (8 * (i & 3));
            }
        }
    }
    // value codes: two tokens share a byte; run z of the page: tokens 2j, 2j+1, numbers 16-byte runs
    constexpr int U = L::U;                              // bytes of a pair's run: 16 or 8
#pragma unroll
    for (int x = 0; x < Page<D>::VC; ++x) {
        const int at = (x * 32 + lane) * 16;             // byte of the value codes
        uint32_t out[4];
#pragma unroll
        for (int half = 0; half < 16 / U; ++half) {
            const int run = (at + half * U) / U;         // ((j/4)*8 + g')*4 + j%4
            const int j = run / 32 * 4 + run % 4, gp = run / 4 % 8;
            uint32_t v[2][U / 4];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint8_t* b;
                int t;
                token(2 * j + u, b, t);
                const int js = t >> 1;
#pragma unroll
                for (int y = 0; y < U / 4; ++y) v[u][y] = 0u;
                if (b != nullptr) {
                    const uint8_t* p = b + L::vCodes + ((js / 4 * 8 + gp) * 4 + js % 4) * U;
                    if constexpr (U == 16) {
                        const uint4 q = *reinterpret_cast<const uint4*>(p);
                        v[u][0] = q.x; v[u][1] = q.y; v[u][2] = q.z; v[u][3] = q.w;
                    } else {
                        const uint2 q = *reinterpret_cast<const uint2*>(p);
                        v[u][0] = q.x; v[u][1] = q.y;
                    }
                    const int sh = 4 * (t & 1);
#pragma unroll
                    for (int y = 0; y < U / 4; ++y) v[u][y] = v[u][y] >> sh & 0x0f0f0f0fu;
                }
            }
#pragma unroll
            for (int y = 0; y < U / 4; ++y) out[half * (U / 4) + y] = v[0][y] | v[1][y] << 4;
        }
        g.va[x] = make_uint4(out[0], out[1], out[2], out[3]);
    }
    // value scales: block b, pair j, token parity: byte ((b*4 + j%4)*8 + j/4)*2 + parity
    {
#pragma unroll
        for (int x = 0; x < 4; ++x) g.vs[x] = 0u;
        const int blk = lane >> 2, j4 = lane & 3;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint8_t* b;
            int t;
            token(2 * (j4 + 4 * (i >> 1)) + (i & 1), b, t);
            const int js = t >> 1;
            const uint32_t v = b == nullptr || blk >= D / 16 ? 0u : b[L::vScales + ((blk * 4 + js % 4) * 8 + js / 4) * 2 + (t & 1)];
            g.vs[i / 4] |= v << (8 * (i & 3));
        }
    }
}

template <int D>
__device__ __forceinline__ void write_page(const Page<D>& g, uint8_t* to, int lane) {
    using L = Kv4Layout<D>;
#pragma unroll
    for (int x = 0; x < Page<D>::KC; ++x) *reinterpret_cast<uint4*>(to + (x * 32 + lane) * 16) = g.k[x];
    if constexpr (L::R == 2) *reinterpret_cast<uint4*>(to + L::kScales + ((lane >> 3) * 8 + (lane & 7)) * 16) = make_uint4(g.ks[0], g.ks[1], g.ks[2], g.ks[3]);
    else *reinterpret_cast<uint2*>(to + L::kScales + ((lane >> 3) * 8 + (lane & 7)) * 8) = make_uint2(g.ks[0], g.ks[1]);
#pragma unroll
    for (int x = 0; x < Page<D>::VC; ++x) *reinterpret_cast<uint4*>(to + L::vCodes + (x * 32 + lane) * 16) = g.va[x];
    if ((lane >> 2) < D / 16) *reinterpret_cast<uint4*>(to + L::vScales + lane * 16) = make_uint4(g.vs[0], g.vs[1], g.vs[2], g.vs[3]);
}

template <int D>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const EvictArgs a) {
    using L = Kv4Layout<D>;
    const EvictWs w = evict_ws(a.ws, a.p.S, a.p.max_pages, a.p.n_pages);
    pdl_wait();
    pdl_trigger();
    if (w.header[0] == 0) return;
    if (static_cast<int>(blockIdx.x) < a.p.S) {
        move_book(a, w, blockIdx.x);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long items = static_cast<long long>(a.p.n_layers) * a.n_kv * a.p.S;
    for (long long item = blockIdx.x - a.p.S; item < items; item += gridDim.x - a.p.S) {
        const int s = static_cast<int>(item % a.p.S);
        const long long rest = item / a.p.S;
        const int h = static_cast<int>(rest % a.n_kv);
        const long long layer = rest / a.n_kv;
        const SeqPlan r = w.seqs[s];
        if (r.now >= r.len) continue;
        uint8_t* head = static_cast<uint8_t*>(a.p.pages) + layer * a.p.layer_stride + static_cast<long long>(h) * L::bytes;
        const int* kept = w.kept + static_cast<long long>(s) * a.p.max_pages * kPage;
        const int* old_page = w.old_page + static_cast<long long>(s) * a.p.max_pages;
        const int* rank = w.rank + static_cast<long long>(s) * a.p.max_pages;
        const int end = pages_of(r.now);
        for (int c0 = r.first; c0 < end; c0 += kMoveWarps) {
            const int c = c0 + warp;
            Page<D> g;
            if (c < end) read_page<D>(g, head, a.p.page_bytes, kept, old_page, c, r.now, lane);
            __syncthreads();
            if (c < end) {
                const int to = rank[c] >= 0 ? w.free_pages[r.base + rank[c]] : old_page[c];
                write_page<D>(g, head + to * a.p.page_bytes, lane);
            }
        }
        __syncthreads();
    }
}

}  // namespace

size_t kv4_evict_workspace(int S, int max_pages, int n_pages) {
    const size_t table = static_cast<size_t>(S) * max_pages;
    return (64 + static_cast<size_t>(n_pages) + table * (2 + kPage)) * sizeof(int) + static_cast<size_t>(S) * sizeof(SeqPlan);
}

cudaError_t launch_kv4_evict(const moe_kv4_pool& p, int head_dim, int n_kv, float* score, long long ld_score, const int32_t* budget, int sinks,
                             int recent, int32_t* kept, long long ld_kept, void* ws, moe_dev_status* st, cudaStream_t s) {
    const EvictArgs a = {p, n_kv, score, ld_score, budget, sinks, recent, kept, ld_kept, ws, st};
    cudaError_t e = launch_pdl(evict_select_kernel, dim3(p.S), dim3(kSelThreads), 0, s, a);
    if (e != cudaSuccess) return e;
    e = launch_pdl(evict_plan_kernel, dim3(1), dim3(kSelThreads), 0, s, a);
    if (e != cudaSuccess) return e;
    const long long items = static_cast<long long>(p.n_layers) * n_kv * p.S;
    const int grid = p.S + static_cast<int>(items < 16 * sm_count() ? items : 16 * sm_count());
    return head_dim == 64 ? launch_pdl(evict_move_kernel<64>, dim3(grid), dim3(kMoveThreads), 0, s, a)
                          : launch_pdl(evict_move_kernel<128>, dim3(grid), dim3(kMoveThreads), 0, s, a);
}

}  // namespace moe
