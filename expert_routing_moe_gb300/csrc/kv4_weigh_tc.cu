// kv4_weigh_tc.cu -- the attention weight that cached tokens draw from many rows
// (prompts): tcgen05.
//
// An item is 256 places of a sequence, in two halves of 128 TMEM lanes.  For one
// key head the places' keys stay in TMEM as the products' A operand (bf16,
// exact); query rows come by TMA, up to 96 at a time (whole tokens of the key
// head's query heads), as the B operand:
//     D[place][row] = K[place] . Q[row]              (fp32 in TMEM, two buffers)
// and two threads for each place add up 2^(f D - lse) over half of the rows
// each.  Sums stay in registers over all rows and heads.
//
// A prompt of 8192 tokens with 32 + 4 heads of 128 is 275 GFLOP (144 us at 1910
// TFLOP/s) and 1.07e9 exponentials (about 120 us at 30 a clock and SM): 232 us.  The
// products alone take 146; without the exponentials it takes 201, without
// the loads of lse 205: no unit is full (exponentials 54%), the chain from a product
// to the buffer's release is what is left.  Eight warps with a whole tile's
// columns each, the next half loaded ahead, took 283 us; sixteen with a
// place of both halves and a quarter of the columns 251; sixteen that load
// a quarter ahead 242.
//
// Warps: 0-15 turn keys to bf16 and add up (eight for each half: two for each of its four groups of
// 32 lanes), 16 and 17 issue a half's products each, 18 brings the rows.
//
// The tiles (rows of a head of an item) of all items are one sequence, cut
// into equal runs for the CTAs; what a run has of an item that others share goes to
// the workspace and is added up in order by a second kernel.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kv4_weigh.cuh"
#include "launch.h"
#include "tc_ts.cuh"
#include "tmap.h"

namespace moe {

namespace {

constexpr int kHalves = 2;
constexpr int kKeys = 256;                // places of an item
constexpr int kMaxRows = 96;              // of a tile
constexpr int kPart = kMaxRows / 2;       // columns that a thread takes at a time
constexpr int kEpi = 16;                  // warps that convert keys and add up
constexpr int kWarpMma = kEpi, kWarpQ = kEpi + kHalves;
constexpr int kThreads = (kWarpQ + 1) * 32;
constexpr int kPlanThreads = 1024;
constexpr int kMaxCtas = 160;
constexpr int kMinRun = 6;                // tiles of a CTA at least

struct Item {
    int32_t s, key0, tiles, ia, ib, q0, len, base;     // tiles: of a head; base: place of row 0
};
// What a head of an item costs beside its tiles, in tiles: its keys' conversion with the start and end of the pipeline, and what the
// tiles at the diagonal take more than others.  (A prompt of 8192 tokens with 2 + a hundredth, a third and half of those: 303, 282,
// 278 us: the last runs are all diagonal.)
__device__ __forceinline__ int head_cost(int tiles, int ntok) { return tiles > 0 ? 3 + min(tiles, kKeys / ntok + 1) / 2 : 0; }
// Workspace: header, the runs' first items, their pieces, then the items and the tiles before each.
struct WeighWs {
    long long* total;
    int* start;                           // [kMaxCtas]
    float* part;                          // [kMaxCtas][2][kKeys]: of the item that the run starts in and of the one that it ends in
    Item* items;
    long long* before;                    // [items + 1]
};
__host__ __device__ inline WeighWs weigh_ws(void* ws, size_t items) {
    WeighWs w;
    w.total = static_cast<long long*>(ws);
    w.start = reinterpret_cast<int*>(w.total) + 64;
    w.part = reinterpret_cast<float*>(w.start + kMaxCtas);
    w.items = reinterpret_cast<Item*>(w.part + kMaxCtas * 2 * kKeys);
    w.before = reinterpret_cast<long long*>(w.items + items);
    return w;
}
__host__ __device__ inline size_t max_items(int S, int max_pages) {
    return static_cast<size_t>(S) * ((static_cast<size_t>(max_pages) * kPage + kKeys - 1) / kKeys);
}
__device__ __forceinline__ long long run_share(long long total, int grid) {
    const long long share = (total + grid - 1) / grid;
    return share < kMinRun ? kMinRun : share;
}

// ---------------------------------------------------------------------------
// The items, the tiles before each, and the one that every CTA starts in: one CTA.
// ---------------------------------------------------------------------------
__device__ __forceinline__ long long scan_long(long long v, long long& total, long long* s_warp) {
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
    for (int i = 0; i < kPlanThreads / 32; ++i) {
        if (i < warp) before += s_warp[i];
        total += s_warp[i];
    }
    return before + inc - v;
}

__global__ void __launch_bounds__(kPlanThreads, 1) weigh_plan_kernel(const WeighArgs a, void* ws, int ntok, int grid) {
    constexpr int kSeqs = kPlanThreads / 32;
    __shared__ long long s_warp[kSeqs];
    __shared__ WeighSeq s_seq[kSeqs];
    __shared__ int s_b0[kSeqs], s_n[kSeqs], s_first[kSeqs + 1];
    const WeighWs w = weigh_ws(ws, max_items(a.c.S, a.c.max_pages));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    pdl_wait();
    pdl_trigger();
    long long items = 0, tiles = 0, own = -1, own_u0 = 0, own_u1 = 0;
    for (int s0 = 0; s0 < a.c.S; s0 += kSeqs) {
        // a warp for each sequence, then a thread for each item
        const int s = s0 + warp;
        WeighSeq q = {0, 0, 0, 0, true};
        if (s < a.c.S) q = weigh_seq(a, s);
        const bool mine = s < a.c.S && q.fit && (q.n - q.i0) * a.group >= a.many && q.len > 0;
        if (lane == 0) {
            if (!q.fit && a.many == 1) report(a.st, MOE_DEV_BAD_INDEX, s);     // (the other kernel does it otherwise)
            s_seq[warp] = q;
            s_b0[warp] = mine ? weigh_first(a, q) / kKeys : 0;
            s_n[warp] = mine ? (q.len + kKeys - 1) / kKeys - s_b0[warp] : 0;
        }
        __syncthreads();
        if (warp == 0) {
            int inc = s_n[lane];
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const int x = __shfl_up_sync(kFull, inc, off);
                if (lane >= off) inc += x;
            }
            s_first[lane + 1] = inc;
            if (lane == 0) s_first[0] = 0;
        }
        __syncthreads();
        const int n = s_first[kSeqs];
        for (int i0 = 0; i0 < n; i0 += kPlanThreads) {
            const int i = i0 + tid;
            long long cost = 0, all;
            if (i < n) {
                int j = 0;
#pragma unroll
                for (int step = kSeqs / 2; step > 0; step >>= 1)
                    if (s_first[j + step] <= i) j += step;
                const WeighSeq x = s_seq[j];
                Item it;
                it.s = s0 + j;
                it.key0 = (s_b0[j] + i - s_first[j]) * kKeys;
                weigh_rows(a, x, it.key0, kKeys, it.ia, it.ib);
                it.tiles = (it.ib - it.ia + ntok - 1) / ntok;
                it.q0 = x.q0;
                it.len = x.len;
                it.base = x.base();
                w.items[items + i] = it;
                // an item without rows has one unit all the same: its new tokens' scores may have to be set
                cost = max(1ll, static_cast<long long>(it.tiles + head_cost(it.tiles, ntok)) * a.c.n_kv);
            }
            const long long at = tiles + scan_long(cost, all, s_warp);
            if (i < n) {
                w.before[items + i] = at;
                own = items + i;
                own_u0 = at;
                own_u1 = at + cost;
            }
            tiles += all;
        }
        items += n;
        __syncthreads();
    }
    const long long share = run_share(tiles, grid);
    auto starts = [&](long long i, long long u0, long long u1) {
        for (long long b = (u0 + share - 1) / share; b * share < u1 && b < grid; ++b) w.start[b] = static_cast<int>(i);
    };
    if (a.c.S <= kSeqs && items <= kPlanThreads) {
        if (own >= 0) starts(own, own_u0, own_u1);
    } else {
        __threadfence_block();
        __syncthreads();
        for (long long i = tid; i < items; i += kPlanThreads) starts(i, w.before[i], i + 1 < items ? w.before[i + 1] : tiles);
    }
    if (tid == 0) {
        w.before[items] = tiles;
        *w.total = tiles;
    }
}

// ---------------------------------------------------------------------------
template <int D>
struct Tc {
    static constexpr int box = kMaxRows * 128;            // 64 numbers of the tile's rows
    static constexpr int stage = box * (D / 64);
    static constexpr int stages = D == 128 ? 7 : 8;
    static constexpr int smem = stages * stage + 1024;    // slack for 1024-byte alignment
    static constexpr int c_a = 2 * kHalves * kMaxRows;    // TMEM columns: D [half][buffer][96], then A [half][D/2]
};
enum Site : int { kSiteQFull = 51, kSiteQEmpty, kSiteA, kSiteDFull, kSiteDEmpty, kSiteSeg };

__device__ __forceinline__ void st_cols(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
__device__ __forceinline__ void ld_cols(uint32_t taddr, uint32_t (&v)[48]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr)
        : "memory");
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(v[32]), "=r"(v[33]), "=r"(v[34]), "=r"(v[35]), "=r"(v[36]), "=r"(v[37]), "=r"(v[38]), "=r"(v[39]),
          "=r"(v[40]), "=r"(v[41]), "=r"(v[42]), "=r"(v[43]), "=r"(v[44]), "=r"(v[45]), "=r"(v[46]), "=r"(v[47])
        : "r"(taddr + 32)
        : "memory");
}
// Barrier of a half's warps; the AND of what they bring.
__device__ __forceinline__ bool half_sync_and(int m, bool v) {
    uint32_t r;
    if (m == 0)
        asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, 2, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(r) : "r"(v ? 1u : 0u) : "memory");
    else
        asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %1, 0;\n\tbar.red.and.pred q, 3, 256, p;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(r) : "r"(v ? 1u : 0u) : "memory");
    return r != 0;
}
// 4-d box of query numbers: numbers, query heads of a key head, key head, tokens.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, int x, int y, int z, int w, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
        : "memory");
}

// A run's walk over its items, their heads and tiles: the same in every role.  A head's units are its cost, then one for each
// tile; a run has the tiles whose units it holds.
struct Walk {
    const WeighWs& w;
    long long u1;                          // end of the run
    long long begin;                       // first unit of the item
    int idx, head, cost, units;            // units: the item's
    int at, end;                           // the run's units of the head at hand
    int left;                              // the run's units of the item, from the head at hand on
    Item it;
    int n_kv, ntok;
    __device__ Walk(const WeighWs& w_, int n_kv_, int ntok_, int start, long long u0, long long u1_) : w(w_), u1(u1_), n_kv(n_kv_), ntok(ntok_) {
        idx = start;
        load(u0);
    }
    __device__ void load(long long u0) {
        it = w.items[idx];
        begin = w.before[idx];
        const long long next = w.before[idx + 1];
        units = static_cast<int>(next - begin);
        cost = head_cost(it.tiles, ntok);
        const int per = it.tiles + cost, from = static_cast<int>(u0 - begin);
        left = static_cast<int>(min(next, u1) - u0);
        head = per > 0 ? from / per : 0;
        at = per > 0 ? from % per : 0;
        end = per > 0 ? min(per, at + left) : 0;
    }
    __device__ bool starts() const { return head == 0 && at == 0; }
    __device__ bool whole() const { return begin + units <= u1; }    // (with a start at the item's first unit)
    // tiles of the head at hand that are this run's: the first, and how many
    __device__ int tile() const { return max(0, at - cost); }
    __device__ int head_tiles() const { return max(0, end - cost) - tile(); }
    __device__ bool next_head() {          // false: the item has no more for this run
        left -= it.tiles > 0 ? end - at : left;
        ++head;
        at = 0;
        end = min(it.tiles + cost, left);
        return left > 0;
    }
    __device__ bool next_item() {
        const long long next = begin + units;
        if (next >= u1) return false;
        ++idx;
        load(next);
        return true;
    }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) weigh_tc_kernel(const WeighArgs a, const __grid_constant__ CUtensorMap map_q, void* ws, int ntok) {
    using C = Tc<D>;
    using L = Kv4Layout<D>;
    enum { B_QF = 0, B_QE = B_QF + C::stages, B_A = B_QE + C::stages, B_DF = B_A + kHalves, B_DE = B_DF + 4, B_SEG = B_DE + 4, B_DRAIN = B_SEG + kHalves, B_N = B_DRAIN + kHalves };
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ __align__(8) uint64_t bars[B_N];
    __shared__ __align__(16) float s_z[C::stages][kMaxRows];   // -lse in powers of two
    __shared__ __align__(16) int s_p[C::stages][kMaxRows];     // the rows' places, -1 for one that adds nothing
    __shared__ int s_slow[C::stages];
    __shared__ float s_sum[kKeys];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::stages; ++i) { mbar_init(bar(B_QF + i), 2); mbar_init(bar(B_QE + i), kHalves + kEpi); }
        for (int i = 0; i < kHalves; ++i) { mbar_init(bar(B_A + i), kEpi / 2); mbar_init(bar(B_SEG + i), 1); mbar_init(bar(B_DRAIN + i), 1); }
        for (int i = 0; i < 4; ++i) { mbar_init(bar(B_DF + i), 1); mbar_init(bar(B_DE + i), kEpi / 2); }
        fence_mbar_init();
        s_abort = 0;
    }
    // rows of a stage that no token fills stay zero
    for (int i = threadIdx.x; i < C::stages * C::stage / 16; i += kThreads) reinterpret_cast<uint4*>(smem)[i] = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
    if (warp == kWarpMma) {
        tmem_alloc(smem_u32(&s_tmem), 512);                     // all columns: the first is 0
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    pdl_wait();
    pdl_trigger();
    const WeighWs w = weigh_ws(ws, max_items(a.c.S, a.c.max_pages));
    const long long total = *w.total, share = run_share(total, gridDim.x);
    const long long u0 = share * blockIdx.x, u1 = min(total, u0 + share);
    const int rows = ntok * a.group;
    bool ok = true;
    if (u0 < u1) {
        Walk k(w, a.c.n_kv, ntok, w.start[blockIdx.x], u0, u1);
        if (warp == kWarpQ) {
            // ---------------- queries ----------------
            // A tile's log-sum-exps are on their way to registers while the tile before is handed over.
            constexpr int kJ = kMaxRows / 32;
            int jt[kJ], jh[kJ];            // token and query head of the lane's rows
#pragma unroll
            for (int c = 0; c < kJ; ++c) {
                jt[c] = (lane + 32 * c) / a.group;
                jh[c] = (lane + 32 * c) % a.group;
            }
            Walk ahead = k;
            int ax = 0;                    // the tile of its head that `ahead` is at
            bool have = true;              // there is one
            auto settle = [&]() {          // goes on to the next head with tiles
                while (have && ax >= ahead.head_tiles()) {
                    ax = 0;
                    if (!ahead.next_head()) have = ahead.next_item();
                }
            };
            float l[kJ], l_next[kJ];
            auto fetch = [&]() {
                const int i = ahead.it.ia + (ahead.tile() + ax) * ntok;
#pragma unroll
                for (int c = 0; c < kJ; ++c) {
                    l_next[c] = -INFINITY;
                    if (lane + 32 * c < rows && i + jt[c] < ahead.it.ib)
                        l_next[c] = __ldg(a.lse + static_cast<long long>(ahead.it.q0 + i + jt[c]) * a.n_q + ahead.head * a.group + jh[c]);
                }
            };
            settle();
            if (have) fetch();
            uint32_t n = 0;
            while (have && ok) {
                const int st = n % C::stages, i = ahead.it.ia + (ahead.tile() + ax) * ntok, head = ahead.head;
                const int q0 = ahead.it.q0, base = ahead.it.base, key0 = ahead.it.key0;
#pragma unroll
                for (int c = 0; c < kJ; ++c) l[c] = l_next[c];
                ++ax;
                settle();
                if (have) fetch();
                ok = wait_warp(bar(B_QE + st), ((n / C::stages) & 1) ^ 1, &s_abort, a.st, kSiteQEmpty);
                if (!ok) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(bar(B_QF + st), rows * D * 2);
                    for (int b = 0; b < D / 64; ++b) tma_load_4d(smem_u32(smem + st * C::stage + b * C::box), &map_q, 64 * b, 0, head, q0 + i, bar(B_QF + st));
                }
                bool none = false;
#pragma unroll
                for (int c = 0; c < kJ; ++c) {
                    const bool sees = l[c] != -INFINITY;       // (rows that do not count have it too)
                    s_z[st][lane + 32 * c] = sees ? l[c] * -kLog2e : -INFINITY;
                    s_p[st][lane + 32 * c] = sees ? base + i + jt[c] : -1;
                    none |= lane + 32 * c < rows && !sees;
                }
                none = __any_sync(kFull, none);
                if (lane == 0) {
                    // every row sees all of the item's places, or it has to be looked at
                    const int p0 = base + i, p1 = p0 + ntok - 1;
                    s_slow[st] = none || p0 < key0 + kKeys - 1 || (a.window > 0 && key0 <= p1 - a.window);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_QF + st));
                ++n;
            }
            if (!ok && lane == 0)          // what is in flight lands before the CTA ends
                for (int i = 0; i < C::stages; ++i) {
                    mbar_drain(bar(B_QF + i), 0);
                    mbar_drain(bar(B_QF + i), 1);
                }
        } else if (warp >= kWarpMma) {
            // ---------------- products ----------------
            const int m = warp - kWarpMma;
            const uint32_t idesc = idesc_bf16_f32(128, kMaxRows);
            const uint64_t b0 = sw128_desc(smem_u32(smem));
            uint32_t n = 0, seg = 0;
            bool more = true;
            while (more && ok) {
                do {
                    const int tiles = k.head_tiles();
                    if (tiles > 0) {
                        ok = wait_warp(bar(B_A + m), seg & 1, &s_abort, a.st, kSiteA);
                        ++seg;
                    }
                    for (int x = 0; x < tiles && ok; ++x, ++n) {
                        const int st = n % C::stages, buf = n & 1;
                        ok = wait_warp(bar(B_QF + st), (n / C::stages) & 1, &s_abort, a.st, kSiteQFull) &&
                             wait_warp(bar(B_DE + m * 2 + buf), ((n >> 1) & 1) ^ 1, &s_abort, a.st, kSiteDEmpty);
                        if (!ok) break;
                        tc_fence_after();
                        if (elect_one()) {
                            const uint64_t b = b0 + static_cast<uint64_t>(st * (C::stage >> 4));
#pragma unroll
                            for (int y = 0; y < D / 16; ++y)
                                mma_ts((m * 2 + buf) * kMaxRows, C::c_a + m * (D / 2) + y * 8, b + (y / 4) * (C::box >> 4) + (y % 4) * 2, idesc, y > 0);
                            tc_commit(bar(B_DF + m * 2 + buf));
                            tc_commit(bar(B_QE + st));
                        }
                        __syncwarp();
                    }
                    if (tiles > 0 && ok && elect_one()) tc_commit(bar(B_SEG + m));
                    __syncwarp();
                } while (ok && k.next_head());
                more = ok && k.next_item();
            }
            if (!ok && n > 0) {            // the products in flight end before TMEM is freed
                if (elect_one()) tc_commit(bar(B_DRAIN + m));
                __syncwarp();
                mbar_drain(bar(B_DRAIN + m), 0);
            }
        } else {
            // ---------------- keys to bf16, and the sums ----------------
            const int m = warp >> 3, part = warp >> 2 & 1, r = (warp & 3) * 32 + lane;     // half, half of the columns, place
            const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
            uint32_t n = 0, seg = 0;
            bool more = true;
            while (more && ok) {
                const int key = k.it.key0 + m * 128 + r;
                const bool there = key < k.it.len;
                int page = -1;
                if (there) page = a.c.page_table[static_cast<long long>(k.it.s) * a.c.max_pages + key / kPage];
                const bool good = page >= 0 && page < a.c.n_pages;
                if (there && !good && key % kPage == 0) report(a.st, MOE_DEV_BAD_INDEX, page);
                const bool starts = k.starts(), ends = k.whole();
                float sum = 0.f;
                do {
                    const int tiles = k.head_tiles();
                    if (tiles == 0) continue;              // (goes on with the next head)
                    const uint8_t* base = static_cast<const uint8_t*>(a.c.pages) + (static_cast<long long>(page) * a.c.n_kv + k.head) * L::bytes;
                    // (the two warps of a place convert half of its numbers each)
                    constexpr int kRuns = D / 64;
                    uint4 run[kRuns];
                    uint32_t sc[kRuns];                    // two scales each
#pragma unroll
                    for (int x = 0; x < kRuns; ++x) { run[x] = make_uint4(0u, 0u, 0u, 0u); sc[x] = 0u; }
                    if (good) {
                        const int tok = key % kPage;
#pragma unroll
                        for (int x = 0; x < kRuns; ++x) run[x] = __ldg(reinterpret_cast<const uint4*>(base + L::k_code(tok, 32 * (part * kRuns + x))));
#pragma unroll
                        for (int x = 0; x < kRuns; ++x) {
                            const int y = 2 * (part * kRuns + x);
                            if constexpr (L::R == 2) sc[x] = __ldg(reinterpret_cast<const uint16_t*>(base + L::k_scale(tok, y)));
                            else sc[x] = __ldg(base + L::k_scale(tok, y)) | static_cast<uint32_t>(__ldg(base + L::k_scale(tok, y + 1))) << 8;
                        }
                    }
                    ok = wait_warp(bar(B_SEG + m), (seg & 1) ^ 1, &s_abort, a.st, kSiteSeg);     // the products with the keys before are over
                    ++seg;
                    if (!ok) break;
                    tc_fence_after();
#pragma unroll
                    for (int x = 0; x < kRuns; ++x) {
                        const uint32_t two = e4m3x2_to_f16(sc[x]);
                        const uint32_t s2[2] = {__byte_perm(two, 0, 0x1010), __byte_perm(two, 0, 0x3232)};
                        const uint32_t words[4] = {run[x].x, run[x].y, run[x].z, run[x].w};
                        uint32_t v[16];
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            uint32_t f[4];
                            e2m1x8_to_f16(words[y], f[0], f[1], f[2], f[3]);
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const uint32_t h = hmul2_u(f[j], s2[y / 2]);
                                __half2 h2;
                                memcpy(&h2, &h, 4);
                                const float2 lh = __half22float2(h2);
                                const __nv_bfloat162 o = __floats2bfloat162_rn(lh.x, lh.y);      // exact
                                memcpy(&v[y * 4 + j], &o, 4);
                            }
                        }
                        st_cols(C::c_a + m * (D / 2) + (part * kRuns + x) * 16 + lanes, v);
                    }
                    st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(B_A + m));
                    const float f = a.scale * kLog2e * (a.c.k_scale != nullptr ? a.c.k_scale[k.head] : 1.f);
                    const unsigned span = a.window > 0 ? a.window : 0x7fffffff;    // places from a key's own on that see it
                    float head_sum = 0.f;
                    auto at = [&](uint32_t u) { return (m * 2 + (u & 1)) * kMaxRows + part * kPart + lanes; };
                    auto wait_d = [&](uint32_t u) {
                        const uint32_t df = bar(B_DF + m * 2 + (u & 1)), qf = bar(B_QF + u % C::stages), pd = (u >> 1) & 1, pq = (u / C::stages) & 1;
                        if (!__all_sync(kFull, mbar_try_wait(qf, pq) && mbar_try_wait(df, pd)))
                            ok = wait_warp(qf, pq, &s_abort, a.st, kSiteQFull) && wait_warp(df, pd, &s_abort, a.st, kSiteDFull);
                        tc_fence_after();
                        return ok;
                    };
                    auto add = [&](const uint32_t (&v)[kPart], int st, bool slow) {
                        float2 sums[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
                        if (!slow) {
#pragma unroll
                            for (int j = 0; j < kPart; j += 4) {
                                const float4 z = *reinterpret_cast<const float4*>(&s_z[st][part * kPart + j]);
                                const float2 x2 = fma2(make_float2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), make_float2(f, f), make_float2(z.x, z.y));
                                const float2 y2 = fma2(make_float2(__uint_as_float(v[j + 2]), __uint_as_float(v[j + 3])), make_float2(f, f), make_float2(z.z, z.w));
                                sums[0] = add2(sums[0], make_float2(ex2(x2.x), ex2(x2.y)));
                                sums[1] = add2(sums[1], make_float2(ex2(y2.x), ex2(y2.y)));
                            }
                        } else {
#pragma unroll
                            for (int j = 0; j < kPart; j += 4) {
                                const float4 z = *reinterpret_cast<const float4*>(&s_z[st][part * kPart + j]);
                                const int4 p = *reinterpret_cast<const int4*>(&s_p[st][part * kPart + j]);
                                const float2 x2 = fma2(make_float2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), make_float2(f, f), make_float2(z.x, z.y));
                                const float2 y2 = fma2(make_float2(__uint_as_float(v[j + 2]), __uint_as_float(v[j + 3])), make_float2(f, f), make_float2(z.z, z.w));
                                // seen from its own place on, as far as the window goes
                                const auto seen = [&](int q, float e) { return static_cast<unsigned>(q - key) < span ? e : 0.f; };
                                sums[0] = add2(sums[0], make_float2(seen(p.x, ex2(x2.x)), seen(p.y, ex2(x2.y))));
                                sums[1] = add2(sums[1], make_float2(seen(p.z, ex2(y2.x)), seen(p.w, ex2(y2.y))));
                            }
                        }
                        head_sum += (sums[0].x + sums[0].y) + (sums[1].x + sums[1].y);
                    };
                    for (int x = 0; x < tiles && wait_d(n); ++x, ++n) {
                        const int st = n % C::stages;
                        uint32_t d[kPart];
                        ld_cols(at(n), d);
                        const bool slow = s_slow[st] != 0;
                        tmem_ld_wait();
                        tc_fence_before();                     // D is read: it may be written again
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(B_DE + m * 2 + (n & 1)));
                        add(d, st, slow);
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(B_QE + st));
                    }
                    sum += head_sum;
                } while (ok && k.next_head());
                // the warps of a half leave together where a wait has failed
                if (part == 1) s_sum[m * 128 + r] = sum;
                ok = half_sync_and(m, ok);
                if (!ok) break;
                if (part == 0) {
                    sum += s_sum[m * 128 + r];
                    if (starts && ends) {
                        WeighSeq q;
                        q.len = k.it.len;
                        q.n = k.it.len - k.it.base;
                        if (there && good) weigh_add(a, q, k.it.s, key, sum);
                    } else {
                        w.part[(blockIdx.x * 2 + (starts ? 1 : 0)) * kKeys + m * 128 + r] = sum;
                    }
                }
                more = k.next_item();
                if (more) ok = half_sync_and(m, ok);           // the sums are read
            }
        }
    }
    __syncthreads();
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(0, 512);
    }
}

// A CTA for each run: adds up the pieces of the item that starts in it and goes on.
__global__ void __launch_bounds__(kKeys) weigh_join_kernel(const WeighArgs a, void* ws, int grid) {
    const WeighWs w = weigh_ws(ws, max_items(a.c.S, a.c.max_pages));
    pdl_wait();
    pdl_trigger();
    // (loads that do not wait for one another are made together; the last run's next one is none)
    const int b = blockIdx.x, idx = b + 1 < grid ? w.start[b + 1] : 0;
    const long long total = *w.total, share = run_share(total, grid);
    const long long u1 = min(total, share * (b + 1));
    if (share * b >= total || u1 >= total) return;
    // the item of the next run's first unit, if it starts in this one
    const long long begin = w.before[idx], end = w.before[idx + 1];
    const Item it = w.items[idx];
    float v = w.part[(b * 2 + 1) * kKeys + threadIdx.x];
    if (begin >= u1 || begin < share * b) return;
    const int key = it.key0 + threadIdx.x;
    if (key >= it.len) return;
    const int page = a.c.page_table[static_cast<long long>(it.s) * a.c.max_pages + key / kPage];
    for (int i = b + 1; share * i < end; ++i) v += w.part[i * 2 * kKeys + threadIdx.x];
    if (page < 0 || page >= a.c.n_pages) return;
    WeighSeq q;
    q.len = it.len;
    q.n = it.len - it.base;
    weigh_add(a, q, it.s, key, v);
}

// q [T][n_kv][group][D] with rows ld_q numbers apart: boxes of 64 numbers, the group's heads, one key head, ntok tokens.
bool map_queries(CUtensorMap* m, const WeighArgs& a, int ntok) {
    const cuuint64_t D = a.c.head_dim;
    cuuint64_t dims[4] = {D, static_cast<cuuint64_t>(a.group), static_cast<cuuint64_t>(a.c.n_kv), static_cast<cuuint64_t>(a.T)};
    cuuint64_t strides[3] = {D * 2, D * 2 * a.group, static_cast<cuuint64_t>(a.ld_q) * 2};
    cuuint32_t box[4] = {64, static_cast<cuuint32_t>(a.group), 1, static_cast<cuuint32_t>(ntok)};
    cuuint32_t estr[4] = {1, 1, 1, 1};
    return encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<__nv_bfloat16*>(a.q), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

template <int D>
cudaError_t launch(const WeighArgs& a, void* ws, cudaStream_t s) {
    const int ntok = kMaxRows / a.group, grid = sm_count() < kMaxCtas ? sm_count() : kMaxCtas;
    CUtensorMap map;
    if (!map_queries(&map, a, ntok)) return cudaErrorInvalidValue;
    auto* k = weigh_tc_kernel<D>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Tc<D>::smem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(weigh_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, a, ws, ntok, grid);
    if (e != cudaSuccess) return e;
    e = launch_pdl(k, dim3(grid), dim3(kThreads), Tc<D>::smem, s, a, map, ws, ntok);
    if (e != cudaSuccess) return e;
    return launch_pdl(weigh_join_kernel, dim3(grid), dim3(kKeys), 0, s, a, ws, grid);
}

}  // namespace

bool weigh_tc_fits(int group) { return group <= kMaxRows; }

size_t kv4_weigh_tc_workspace(int S, int max_pages) {
    const size_t items = max_items(S, max_pages);
    return 64 * sizeof(int) + kMaxCtas * sizeof(int) + static_cast<size_t>(kMaxCtas) * 2 * kKeys * sizeof(float) + items * sizeof(Item) + (items + 1) * sizeof(long long);
}

cudaError_t launch_kv4_weigh_tc(const WeighArgs& a, void* ws, cudaStream_t s) {
    return a.c.head_dim == 64 ? launch<64>(a, ws, s) : launch<128>(a, ws, s);
}

}  // namespace moe
