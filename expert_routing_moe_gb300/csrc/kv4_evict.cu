// kv4_evict.cu -- eviction from the 4-bit cache by the tokens' scores
// (moe_kv4_evict): three launches.
//
//  select  a cluster for each sequence finds the score that a token needs (a
//          radix select over the scores' 32 bits, 11, 11 and 10 at a time) and
//          lists the kept tokens in order
//  plan    one CTA gives every sequence its free pages, all or nothing
//  move    tables, references, lengths and scores, a CTA for each sequence; and
//          the kept tokens' codes and scales, a cluster for each (layer, head,
//          sequence)
//
// Moving in place: the k-th kept token comes from a place >= k, so a page is read
// only for itself and for pages before it.  A cluster reads the sources of
// up to 16 pages into registers, meets, then writes them: whatever it writes has
// been read by then.  A sequence whose pages all go to free ones needs no meeting.
//
// 32001 tokens of 48 layers (4 heads of 128) cut to 8192: 168 us onto free pages,
// 181 in place, of which the selection takes 23; 32 sequences of 8 layers 141 and 154.
// 453 MB are to be moved, which is 67 us at the rate of a copy; kept tokens lie
// scattered, 64 bytes of keys and as many of values that they share with a
// neighbour, so that whole sectors of others come with them.  (A CTA a page, whose
// threads look for their sources in the list: 353 us; sources of a page's tokens in
// shared memory, three warps a page: 238; the next pages' sources looked for ahead: 207
// against 200; four pages a CTA in three warps each 200, two pages 185, in six warps each 182, and 168
// with a loop of its own for pages that need no meeting;
// sources made out of line, so that nothing spills: 197.)
#include <cooperative_groups.h>

#include "common.cuh"
#include "kv4.cuh"
#include "launch.h"
#include "ranges.h"
#include "tmap.h"

namespace moe {

namespace cg = cooperative_groups;

namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kMovePages = 2;             // pages of a CTA at a time, six warps each: two halves of the keys, four quarters of the values
constexpr int kMoveThreads = kMovePages * 192;

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
__device__ __forceinline__ long long scan_pair(long long v, long long& total, long long* s_warp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    long long inc = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long x = __shfl_up_sync(kFull, inc, off);
        if (lane >= off) inc += x;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    long long before = 0;
    total = 0;
    for (int i = 0; i < kSelWarps; ++i) {
        if (i < warp) before += s_warp[i];
        total += s_warp[i];
    }
    return before + inc - v;
}
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

// A sequence's places are shared by the CTAs of a cluster, and a CTA's by its threads, in neighbouring runs: so one prefix sum
// gives every kept token its place.
__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(const EvictArgs a) {
    cg::cluster_group cluster = cg::this_cluster();
    const int parts = static_cast<int>(cluster.num_blocks()), part = static_cast<int>(cluster.block_rank());
    __shared__ __align__(16) int s_hist[kBins];
    __shared__ int s_warp[kSelWarps], s_pick[2], s_bad, s_first;
    __shared__ long long s_warp2[kSelWarps], s_count;
    const int s = blockIdx.x / parts, tid = threadIdx.x;
    const EvictWs w = evict_ws(a.ws, a.p.S, a.p.max_pages, a.p.n_pages);
    if (tid == 0) { s_first = 0x7fffffff; s_bad = 0; }
    for (int i = tid; i < kBins; i += kSelThreads) s_hist[i] = 0;
    cluster.sync();
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
        for (int c = tid; c < pages; c += kSelThreads) {       // every CTA looks at all of them: all know whether one is bad
            const int id = row[c];
            if (id < 0 || id >= a.p.n_pages) s_bad = 1;
            if (part == 0) old_page[c] = id;
        }
    __syncthreads();
    bad = bad || s_bad;
    if (bad || !cut) {
        r.bad = bad;
        if (part == 0 && tid == 0) w.seqs[s] = r;
        return;                                                // the whole cluster
    }
    // the best k of the places between the first and the last ones
    const int lo = a.sinks, hi = len - a.recent, k = budget - a.sinks - a.recent;
    const float* score = a.score + s * a.ld_score;
    const int c0 = static_cast<int>(static_cast<long long>(len) * part / parts), c1 = static_cast<int>(static_cast<long long>(len) * (part + 1) / parts);
    const int m0 = max(c0, lo), m1 = min(c1, hi);
    uint32_t prefix = 0u;
    int want = k;                       // of those whose higher bits are the prefix's
    for (int pass = 0; pass < 3 && k > 0; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
        // (unsigned: a step beyond the last place of the longest tables is not below it)
        for (unsigned j = static_cast<unsigned>(m0) + tid; j < static_cast<unsigned>(m1); j += kSelThreads) {
            const uint32_t o = order_of(score[j]);
            if (pass == 0 || (o >> (shift + bits)) == (prefix >> (shift + bits))) atomicAdd(&s_hist[o >> shift & ((1u << bits) - 1)], 1);
        }
        cluster.sync();
        // two bins a thread, from the highest down
        const int b1 = (1 << bits) - 1 - 2 * tid;
        int n[2] = {0, 0};
        if (b1 > 0)
            for (int i = 0; i < parts; ++i) {
                const int2 v = *reinterpret_cast<const int2*>(cluster.map_shared_rank(s_hist, i) + b1 - 1);
                n[0] += v.y;
                n[1] += v.x;
            }
        int total;
        int before = scan(n[0] + n[1], total, s_warp);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (before < want && before + n[i] >= want) {
                s_pick[0] = b1 - i;
                s_pick[1] = before;
            }
            before += n[i];
        }
        cluster.sync();                 // every CTA has read the counts
        prefix |= static_cast<uint32_t>(s_pick[0]) << shift;
        want -= s_pick[1];
        for (int i = tid; i < kBins; i += kSelThreads) s_hist[i] = 0;
        __syncthreads();
    }
    // prefix: the score of the last one that is kept; `want` of those that have it are, the first ones
    const int each = (c1 - c0 + kSelThreads - 1) / kSelThreads, j0 = min(c1, c0 + tid * each), j1 = j0 + min(c1 - j0, each);
    // 1: kept, 2: kept if it is among the first `want`, 0: not
    auto kind = [&](int j) {
        if (j < lo || j >= hi) return 1;
        if (k == 0) return 0;
        const uint32_t o = order_of(score[j]);
        return o > prefix ? 1 : o == prefix ? 2 : 0;
    };
    long long mine = 0;                 // kept ones, and in the upper half those that may be
    for (int j = j0; j < j1; ++j) {
        const int v = kind(j);
        mine += v == 1 ? 1ll : v == 2 ? 1ll << 32 : 0ll;
    }
    long long total2;
    long long at2 = scan_pair(mine, total2, s_warp2);
    if (tid == 0) s_count = total2;
    cluster.sync();
    long long all = 0;
    for (int i = 0; i < parts; ++i) {
        const long long c = *cluster.map_shared_rank(&s_count, i);
        if (i < part) at2 += c;
        all += c;
    }
    int* kept = w.kept + static_cast<long long>(s) * a.p.max_pages * kPage;
    int sure = static_cast<int>(at2), equal = static_cast<int>(at2 >> 32);
    int first = 0x7fffffff;
    for (int j = j0; j < j1; ++j) {
        const int v = kind(j);
        if (v == 1 || (v == 2 && equal < want)) kept[sure + min(equal, want)] = j;
        else first = min(first, j);
        sure += v == 1;
        equal += v == 2;
    }
    first = __reduce_min_sync(kFull, first);
    if ((tid & 31) == 0 && first != 0x7fffffff) atomicMin(&s_first, first);
    cluster.sync();
    if (part == 0) {
        first = 0x7fffffff;
        for (int i = 0; i < parts; ++i) first = min(first, *cluster.map_shared_rank(&s_first, i));
    }
    cluster.sync();                     // no CTA leaves while its shared memory is read
    if (part != 0) return;
    r.now = static_cast<int>(all) + min(static_cast<int>(all >> 32), want);
    r.first = first / kPage;
    // pages that others hold too are written elsewhere
    int* rank = w.rank + static_cast<long long>(s) * a.p.max_pages;
    for (int x0 = r.first; x0 < pages_of(r.now); x0 += kSelThreads) {
        const int c = x0 + tid;
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
    constexpr int kEach = 12;
    const unsigned now = r.now;           // (unsigned: a step beyond the last place of the longest tables is not below it)
    for (unsigned i0 = 0; i0 < now; i0 += kMoveThreads * kEach) {
        int from[kEach];
        float v[kEach];
#pragma unroll
        for (int u = 0; u < kEach; ++u) {
            const unsigned i = i0 + u * kMoveThreads + tid;
            from[u] = i < now ? kept[i] : -1;
        }
#pragma unroll
        for (int u = 0; u < kEach; ++u) v[u] = from[u] >= 0 ? score[from[u]] : 0.f;
        __syncthreads();
#pragma unroll
        for (int u = 0; u < kEach; ++u) {
            const unsigned i = i0 + u * kMoveThreads + tid;
            if (i < now) score[i] = v[u];
        }
    }
    __syncthreads();
    for (unsigned i = now + tid; i < static_cast<unsigned>(r.len); i += kMoveThreads) score[i] = 0.f;
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

// The CTAs of a cluster, or the threads of one.
__device__ __forceinline__ void meet(cg::cluster_group& cluster, int parts) {
    if (parts > 1) cluster.sync();
    else __syncthreads();
}

// Where a token of a page that is made comes from, in shared memory: its keys' codes and its values' codes (NULL: no token,
// zeros), and what leads from there to the scales.  A lane's place is added by whoever reads.
struct __align__(16) Source {
    const uint8_t* codes;
    int scales;
    int shift;                       // values: 4 where the token's codes are in the high halves
};
template <int D>
struct Sources {
    Source k[kPage], v[kPage];
    __device__ __forceinline__ void set(int tok, const uint8_t* head, int t) {     // head: the head's part of the page, t: the token in it
        using L = Kv4Layout<D>;
        Source x = {nullptr, 0, 0}, y = {nullptr, 0, 0};
        if (head != nullptr) {
            const int j = t >> 1;
            x.codes = head + t * (D / 2);
            x.scales = L::kScales + ((t % 8) * 8 + t / 8) * L::R - t * (D / 2);
            const int vc = L::vCodes + ((j / 4 * 8) * 4 + j % 4) * L::U;
            y.codes = head + vc;
            y.scales = L::vScales + ((j % 4) * 8 + j / 4) * 2 + (t & 1) - vc;
            y.shift = 4 * (t & 1);
        }
        k[tok] = x;
        v[tok] = y;
    }
};

// The keys of 32 tokens of a page: lane (part, g) = (lane / 8, lane % 8) has 16-byte runs of tokens g + 8 x -- for D = 64, where a
// token has two, parts 0 and 1 of tokens 16 x + g and parts 2 and 3 of 8 further -- and the scales of blocks part*R .. of
// tokens g + 8 i.
template <int D>
struct KeyPart {
    using L = Kv4Layout<D>;
    static constexpr int runs = kPage * D / 4 / 512, per = D / 32;
    uint4 c[runs];
    uint32_t s[L::R];
    __device__ __forceinline__ int token(int x, int lane) const { return per == 4 ? 8 * x + (lane & 7) : 16 * x + (lane & 7) + 8 * (lane >> 4); }
    __device__ __forceinline__ int run(int lane) const { return per == 4 ? lane >> 3 : lane >> 3 & 1; }
    __device__ __forceinline__ void read(const Sources<D>& src, int half, int lane) {
#pragma unroll
        for (int x = 0; x < L::R; ++x) s[x] = 0u;
#pragma unroll
        for (int x = 0; x < runs; ++x) {
            const Source a = src.k[32 * half + token(x, lane)];
            c[x] = make_uint4(0u, 0u, 0u, 0u);
            if (a.codes != nullptr) c[x] = *reinterpret_cast<const uint4*>(a.codes + run(lane) * 16);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const Source a = src.k[32 * half + 8 * i + (lane & 7)];
            if (a.codes == nullptr) continue;
            const uint8_t* p = a.codes + a.scales + (lane >> 3) * 64 * L::R;
            if constexpr (L::R == 2) s[i / 2] |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(p)) << (16 * (i & 1));
            else s[0] |= static_cast<uint32_t>(*p) << (8 * i);
        }
    }
    __device__ __forceinline__ void write(uint8_t* to, int half, int lane) const {
#pragma unroll
        for (int x = 0; x < runs; ++x) *reinterpret_cast<uint4*>(to + (32 * half + token(x, lane)) * (D / 2) + run(lane) * 16) = c[x];
        uint8_t* p = to + L::kScales + (lane * 8 + 4 * half) * L::R;
        if constexpr (L::R == 2) *reinterpret_cast<uint2*>(p) = make_uint2(s[0], s[1]);
        else *reinterpret_cast<uint32_t*>(p) = s[0];
    }
};
// The values of 16 tokens of a page: lane (g', j) = (lane / 4, lane % 4) has the runs of tokens 8 x + 2 j and + 1, which share
// bytes, and numbers g' (D/8) .., and the scales of the same tokens, block g'.
template <int D>
struct ValuePart {
    using L = Kv4Layout<D>;
    static constexpr int U = L::U, W = U / 4;            // U: bytes of two tokens' run, 16 or 8
    uint32_t c[2][W];
    uint32_t s;
    __device__ __forceinline__ void read(const Sources<D>& src, int quarter, int lane) {
        const int gp = lane >> 2, j = lane & 3;
        s = 0u;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const Source a = src.v[16 * quarter + 8 * x + 2 * j + u];
                uint32_t v[W];
                uint32_t sc = 0u;
#pragma unroll
                for (int y = 0; y < W; ++y) v[y] = 0u;
                if (a.codes != nullptr) {
                    const uint8_t* p = a.codes + gp * 4 * U;
                    if constexpr (U == 16) {
                        const uint4 q = *reinterpret_cast<const uint4*>(p);
                        v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
                    } else {
                        const uint2 q = *reinterpret_cast<const uint2*>(p);
                        v[0] = q.x; v[1] = q.y;
                    }
                    if (gp < D / 16) sc = a.codes[a.scales + gp * 64];
                }
#pragma unroll
                for (int y = 0; y < W; ++y) {
                    v[y] = v[y] >> a.shift & 0x0f0f0f0fu;
                    c[x][y] = u == 0 ? v[y] : c[x][y] | v[y] << 4;
                }
                s |= sc << (8 * (2 * x + u));
            }
    }
    __device__ __forceinline__ void write(uint8_t* to, int quarter, int lane) const {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            uint8_t* p = to + L::vCodes + (quarter * 2 + x) * 32 * U + lane * U;
            if constexpr (U == 16) *reinterpret_cast<uint4*>(p) = make_uint4(c[x][0], c[x][1], c[x][2], c[x][3]);
            else *reinterpret_cast<uint2*>(p) = make_uint2(c[x][0], c[x][1]);
        }
        if ((lane >> 2) < D / 16) *reinterpret_cast<uint32_t*>(to + L::vScales + lane * 16 + quarter * 4) = s;
    }
};

// The first S CTAs keep the books; then a cluster for each (layer, head, sequence) moves its pages.
template <int D>
__global__ void __launch_bounds__(kMoveThreads, 3) evict_move_kernel(const EvictArgs a) {
    using L = Kv4Layout<D>;
    __shared__ Sources<D> s_src[kMovePages];
    cg::cluster_group cluster = cg::this_cluster();
    const int parts = static_cast<int>(cluster.num_blocks()), part = static_cast<int>(cluster.block_rank());
    const EvictWs w = evict_ws(a.ws, a.p.S, a.p.max_pages, a.p.n_pages);
    pdl_wait();
    pdl_trigger();
    if (w.header[0] == 0) return;
    const int books = (a.p.S + parts - 1) / parts;         // clusters that keep them
    if (static_cast<int>(blockIdx.x) / parts < books) {
        if (static_cast<int>(blockIdx.x) < a.p.S) move_book(a, w, blockIdx.x);
        return;
    }
    const int tid = threadIdx.x, lane = tid & 31, mine = tid / 192, role = tid % 192 / 32;
    const long long items = static_cast<long long>(a.p.n_layers) * a.n_kv * a.p.S;
    const int clusters = static_cast<int>(gridDim.x) / parts - books;
    for (long long item = static_cast<int>(blockIdx.x) / parts - books; item < items; item += clusters) {
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
        const bool apart = r.fresh == end - r.first;       // every page is written to a free one: nothing is read that is written
        for (int c0 = r.first + part * kMovePages; c0 - part * kMovePages < end; c0 += parts * kMovePages) {
            __syncthreads();                               // the sources before have been read
            if (tid < kMovePages * kPage) {
                const long long i = static_cast<long long>(c0) * kPage + tid;
                const int src = i < r.now ? kept[i] : -1;
                s_src[tid / kPage].set(tid % kPage, src < 0 ? nullptr : head + old_page[src / kPage] * a.p.page_bytes, src & (kPage - 1));
            }
            const int c = c0 + mine;
            const bool live = c < end;
            uint8_t* to = nullptr;
            if (live) to = head + (rank[c] >= 0 ? w.free_pages[r.base + rank[c]] : old_page[c]) * a.p.page_bytes;
            __syncthreads();
            if (apart) {
                if (live && role < 2) {
                    KeyPart<D> g;
                    g.read(s_src[mine], role, lane);
                    g.write(to, role, lane);
                } else if (live) {
                    ValuePart<D> g;
                    g.read(s_src[mine], role - 2, lane);
                    g.write(to, role - 2, lane);
                }
                continue;
            }
            // what is written has been read by then (pages that come later read neither)
            union {                                        // (a warp has keys or values, in the same registers)
                KeyPart<D> keys;
                ValuePart<D> values;
            } g;
            if (live) {
                if (role < 2) g.keys.read(s_src[mine], role, lane);
                else g.values.read(s_src[mine], role - 2, lane);
            }
            meet(cluster, parts);
            if (live) {
                if (role < 2) g.keys.write(to, role, lane);
                else g.values.write(to, role - 2, lane);
            }
        }
    }
}

cudaError_t launch_clusters(void (*kernel)(EvictArgs), int ctas, int parts, int threads, cudaStream_t s, const EvictArgs& a) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
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

template <int D>
cudaError_t launch_move(const EvictArgs& a, cudaStream_t s) {
    // enough CTAs for every SM eight times over (four times: 221 us for 185), by clusters of up to eight, but none wider than a quarter of a table
    const long long items = static_cast<long long>(a.p.n_layers) * a.n_kv * a.p.S;
    int parts = 1;
    while (parts < 8 && items * parts < 8ll * sm_count() && parts * kMovePages * 4 < a.p.max_pages) parts *= 2;
    const long long most = 16ll * sm_count() / parts > 0 ? 16ll * sm_count() / parts : 1;
    const long long n = ((a.p.S + parts - 1) / parts + (items < most ? items : most)) * parts;
    return launch_clusters(evict_move_kernel<D>, static_cast<int>(n), parts, kMoveThreads, s, a);
}

}  // namespace

size_t kv4_evict_workspace(int S, int max_pages, int n_pages) {
    const size_t table = static_cast<size_t>(S) * max_pages;
    return (64 + static_cast<size_t>(n_pages) + table * (2 + kPage)) * sizeof(int) + static_cast<size_t>(S) * sizeof(SeqPlan);
}

cudaError_t launch_kv4_evict(const moe_kv4_pool& p, int head_dim, int n_kv, float* score, long long ld_score, const int32_t* budget, int sinks,
                             int recent, int32_t* kept, long long ld_kept, void* ws, moe_dev_status* st, cudaStream_t s) {
    const EvictArgs a = {p, n_kv, score, ld_score, budget, sinks, recent, kept, ld_kept, ws, st};
    // a CTA for about 4096 places of the longest sequence that there can be, up to eight
    int parts = 1;
    while (parts < 8 && parts * 64 < p.max_pages) parts *= 2;
    cudaError_t e = launch_clusters(evict_select_kernel, p.S * parts, parts, kSelThreads, s, a);
    if (e != cudaSuccess) return e;
    e = launch_pdl(evict_plan_kernel, dim3(1), dim3(kSelThreads), 0, s, a);
    if (e != cudaSuccess) return e;
    return head_dim == 64 ? launch_move<64>(a, s) : launch_move<128>(a, s);
}

}  // namespace moe
