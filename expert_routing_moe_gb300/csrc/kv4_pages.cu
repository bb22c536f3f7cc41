// kv4_pages.cu -- the pages of the 4-bit cache: growing and truncating
// sequences with copy on write, forking/reordering/freeing them, and packing
// the pool.  The bookkeeping is a few kilobytes of whole numbers: one CTA
// plans (prefix sums give every sequence its pages without any order of
// arrival), and a grid then copies the listed pages of all layers, which is
// bound by device memory.  Packing 4096 pages of 8 layers, half of them in holes,
// moves 561 MB in 100 us (5.6 TB/s, 0.84 of a copy's rate).  A beam search's step of 64
// sequences over 48 layers is two launches' chains of loads: assign 2.6 us,
// the plan of reserve 7 us with the launch of the copies.
#include "common.cuh"
#include "launch.h"
#include "ranges.h"
#include "tmap.h"

namespace moe {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;
constexpr int kAssignCols = 8;        // table columns of a CTA: one 32-byte sector of each row
constexpr int kAssignThreads = 256;
constexpr int kPlaceSmem = 4096;     // pages handed out through shared memory
constexpr int kHeader = 64;           // words before the lists
constexpr int kCopyThreads = 256;
constexpr int kCopyVec = 3;           // 16-byte words in flight of a thread

// Workspace: header, copy list [n_pages], three words a page.  Every call sets what it reads, so that it does not
// matter what a call on another pool has left.
struct PoolWs {
    int* header;     // [0] copies
    int2* copies;    // (from, to)
    int* a;          // reserve: growing sequences that share a page
    int* b;          // reserve: the last of them + 1
    int* place;      // reserve: the pages handed out, ascending; compact: new numbers, -1 for a page not in use
};
__host__ __device__ inline PoolWs pool_ws(void* ws, int n_pages) {
    PoolWs w;
    w.header = static_cast<int*>(ws);
    w.copies = reinterpret_cast<int2*>(w.header + kHeader);
    w.a = reinterpret_cast<int*>(w.copies + n_pages);
    w.b = w.a + n_pages;
    w.place = w.b + n_pages;
    return w;
}

// Exclusive prefix sum of (x, y) over the CTA, and their totals.
struct Sum2 {
    long long x, y;
};
__device__ __forceinline__ Sum2 scan2(Sum2 v, Sum2& total, Sum2* s_warp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Sum2 inc = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long x = __shfl_up_sync(kFull, inc.x, off), y = __shfl_up_sync(kFull, inc.y, off);
        if (lane >= off) { inc.x += x; inc.y += y; }
    }
    __syncthreads();                 // s_warp may still be read from the scan before
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    Sum2 before = {0, 0};
    total = {0, 0};
    for (int i = 0; i < kPlanWarps; ++i) {
        if (i < warp) { before.x += s_warp[i].x; before.y += s_warp[i].y; }
        total.x += s_warp[i].x;
        total.y += s_warp[i].y;
    }
    return {before.x + inc.x - v.x, before.y + inc.y - v.y};
}

// One CTA.  Thread i takes sequences [i * per, (i+1) * per).  What bounds it is
// the chain of loads (length, last page, sharers, references): each is done
// once, the references' scan is read ahead of it, and up to kPlaceSmem pages
// are handed from the threads that find them to those that take them in shared
// memory.
__global__ void __launch_bounds__(kPlanThreads, 1) kv4_reserve_plan_kernel(const moe_kv4_pool p, const int32_t* n_new,
                                                                           void* ws, moe_dev_status* st) {
    constexpr int kPer = 4;          // sequences of a thread: S <= 4096
    __shared__ Sum2 s_warp[kPlanWarps];
    __shared__ int s_bad, s_place[kPlaceSmem];
    const PoolWs w = pool_ws(ws, p.n_pages);
    const int tid = threadIdx.x;
    if (tid == 0) s_bad = -1;
    pdl_wait();
    pdl_trigger();
    const int per = (p.S + kPlanThreads - 1) / kPlanThreads;
    const int s0 = min(p.S, tid * per), s1 = min(p.S, s0 + per);
    auto row = [&](int s) { return p.page_table + static_cast<long long>(s) * p.max_pages; };
    int len[kPer], add[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const bool in = s0 + i < s1;
        len[i] = in ? p.seq_len[s0 + i] : 0;
        add[i] = in ? n_new[s0 + i] : 0;
    }
    // the thread's pages of the pool: its free ones are counted while the sequences' chain runs
    const int chunk = ((p.n_pages + kPlanThreads - 1) / kPlanThreads + 3) & ~3;
    const int g0 = min(static_cast<long long>(p.n_pages), static_cast<long long>(tid) * chunk);
    const int g1 = min(p.n_pages, g0 + chunk);
    Sum2 free_mine = {0, 0}, free_total;
    for (int g = g0; g < g1; ++g) free_mine.x += p.ref[g] == 0;
    __syncthreads();
    int part[kPer];                  // the partly filled last page of a sequence that grows, or -1
#pragma unroll
    for (int i = 0; i < kPer; ++i) part[i] = -1;
    const long long most = min(static_cast<long long>(p.max_pages) * MOE_KV4_PAGE, 0x7fffffffll);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (s0 + i >= s1) break;
        const int s = s0 + i;
        const long long after = static_cast<long long>(len[i]) + add[i];
        if (len[i] < 0 || len[i] > most || after > most) { s_bad = s; continue; }
        if (add[i] > 0 && len[i] % MOE_KV4_PAGE != 0) {
            const int g = row(s)[len[i] / MOE_KV4_PAGE];
            if (g < 0 || g >= p.n_pages) { s_bad = s; continue; }
            part[i] = g;
        }
        for (int c = pages_of(static_cast<int>(max(after, 0ll))); c < pages_of(len[i]); ++c) {
            const int id = row(s)[c];
            if (id < 0 || id >= p.n_pages) s_bad = s;
        }
        if (part[i] >= 0) {
            __stcg(&w.a[part[i]], 0);
            __stcg(&w.b[part[i]], 0);
        }
    }
    __threadfence_block();
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPer; ++i)
        if (part[i] >= 0) {
            atomicAdd(&w.a[part[i]], 1);
            atomicMax(&w.b[part[i]], s0 + i + 1);
        }
    __threadfence_block();
    __syncthreads();
    const bool bad = s_bad >= 0;
    // a sequence's copy (0 or 1) and pages in all
    int copy[kPer], fresh[kPer];
    Sum2 mine = {0, 0}, total;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        copy[i] = fresh[i] = 0;
        if (bad || s0 + i >= s1 || add[i] <= 0) continue;
        if (part[i] >= 0) {
            const int refs = p.ref[part[i]], sharers = __ldcg(&w.a[part[i]]), last = __ldcg(&w.b[part[i]]);
            copy[i] = refs > 1 && !(sharers == refs && last == s0 + i + 1);
        }
        fresh[i] = pages_of(len[i] + add[i]) - pages_of(len[i]);
        mine.x += copy[i] + fresh[i];
        mine.y += copy[i];
    }
    const Sum2 base = scan2(mine, total, s_warp);
    const long long want = total.x;
    // free pages in ascending order, as many as are wanted
    const Sum2 free_base = scan2(free_mine, free_total, s_warp);
    const bool go = !bad && want <= free_total.x;
    int* place = want <= kPlaceSmem ? s_place : w.place;
    if (go) {
        long long k = free_base.x;
        for (int g = g0; g < g1 && k < want; ++g)
            if (p.ref[g] == 0) place[k++] = g;
    }
    // decisions have read references and scratch; both change only after this barrier
    __syncthreads();
    if (go) {
        long long at = base.x, at_copy = base.y;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int s = s0 + i;
            if (s >= s1) break;
            const int held = pages_of(len[i]);
            int32_t* r = row(s);
            if (copy[i]) {
                const int g = place[at++];
                w.copies[at_copy++] = make_int2(part[i], g);
                r[len[i] / MOE_KV4_PAGE] = g;
                p.ref[g] = 1;
                atomicSub(&p.ref[part[i]], 1);
            }
            for (int c = 0; c < fresh[i]; ++c) {
                const int g = place[at++];
                r[held + c] = g;
                p.ref[g] = 1;
            }
            if (add[i] < 0) {
                const int after = max(0, len[i] + add[i]);
                for (int c = pages_of(after); c < held; ++c) {
                    atomicSub(&p.ref[r[c]], 1);
                    r[c] = -1;
                }
                p.seq_len[s] = after;
            } else if (add[i] > 0) {
                p.seq_len[s] = len[i] + add[i];
            }
        }
    }
    if (tid == 0) {
        w.header[0] = go ? static_cast<int>(total.y) : 0;
        if (bad) report(st, MOE_DEV_BAD_INDEX, s_bad);
        else if (!go) report(st, MOE_DEV_NO_PAGES, static_cast<int>(want - free_total.x));
    }
}

// Copies the listed pages of every layer; a CTA takes a part of a page at a time.
__device__ __forceinline__ void copy_pages(const moe_kv4_pool& p, const PoolWs& w) {
    const int n = w.header[0];
    const int vecs = static_cast<int>(p.page_bytes / 16);
    constexpr int kPart = kCopyThreads * kCopyVec;
    const int parts = (vecs + kPart - 1) / kPart;
    const long long items = static_cast<long long>(n) * p.n_layers * parts;
    for (long long i = blockIdx.x; i < items; i += gridDim.x) {
        const int part = static_cast<int>(i % parts);
        const long long rest = i / parts;
        const int layer = static_cast<int>(rest % p.n_layers);
        const int2 c = w.copies[rest / p.n_layers];
        uint8_t* base = static_cast<uint8_t*>(p.pages) + layer * p.layer_stride;
        const uint4* src = reinterpret_cast<const uint4*>(base + c.x * p.page_bytes);
        uint4* dst = reinterpret_cast<uint4*>(base + c.y * p.page_bytes);
        uint4 v[kCopyVec];
        const int at = part * kPart + threadIdx.x;
#pragma unroll
        for (int k = 0; k < kCopyVec; ++k)
            if (at + k * kCopyThreads < vecs) v[k] = __ldcs(src + at + k * kCopyThreads);
#pragma unroll
        for (int k = 0; k < kCopyVec; ++k)
            if (at + k * kCopyThreads < vecs) __stcs(dst + at + k * kCopyThreads, v[k]);
    }
}

__global__ void __launch_bounds__(kCopyThreads) kv4_copy_kernel(const moe_kv4_pool p, void* ws) {
    pdl_wait();
    pdl_trigger();
    copy_pages(p, pool_ws(ws, p.n_pages));
}

// A CTA takes kAssignCols columns of the table for all sequences: it reads
// them all before it writes any, so the table changes in place.
__global__ void __launch_bounds__(kAssignThreads) kv4_assign_kernel(const moe_kv4_pool p, const int32_t* parent,
                                                                    moe_dev_status* st) {
    extern __shared__ int s_old[];    // [S][kAssignCols]; the first CTA's lengths follow
    pdl_wait();
    pdl_trigger();
    const int c0 = blockIdx.x * kAssignCols, cols = min(kAssignCols, p.max_pages - c0);
    for (int x = threadIdx.x; x < p.S * kAssignCols; x += kAssignThreads) {
        const int s = x / kAssignCols, c = x % kAssignCols;
        s_old[x] = c < cols ? p.page_table[static_cast<long long>(s) * p.max_pages + c0 + c] : -1;
    }
    int* s_len = s_old + p.S * kAssignCols;
    if (blockIdx.x == 0)
        for (int s = threadIdx.x; s < p.S; s += kAssignThreads) s_len[s] = p.seq_len[s];
    __syncthreads();
    for (int x = threadIdx.x; x < p.S * kAssignCols; x += kAssignThreads) {
        const int s = x / kAssignCols, c = x % kAssignCols;
        int from = parent[s];
        if (from < -1 || from >= p.S) {
            if (c == 0 && blockIdx.x == 0) report(st, MOE_DEV_BAD_INDEX, from);
            from = s;
        }
        if (from == s) continue;
        if (c < cols) {
            const int old = s_old[x], now = from >= 0 ? s_old[from * kAssignCols + c] : -1;
            if (old != now) {
                if (old >= 0 && old < p.n_pages) atomicSub(&p.ref[old], 1);
                if (now >= 0 && now < p.n_pages) atomicAdd(&p.ref[now], 1);
                p.page_table[static_cast<long long>(s) * p.max_pages + c0 + c] = now;
            }
        }
        if (c == 0 && blockIdx.x == 0) p.seq_len[s] = from >= 0 ? s_len[from] : 0;
    }
}

__global__ void __launch_bounds__(kPlanThreads, 1) kv4_compact_plan_kernel(const moe_kv4_pool p, int32_t* n_live,
                                                                           void* ws) {
    __shared__ Sum2 s_warp[kPlanWarps];
    const PoolWs w = pool_ws(ws, p.n_pages);
    const int tid = threadIdx.x;
    pdl_wait();
    pdl_trigger();
    const int chunk = ((p.n_pages + kPlanThreads - 1) / kPlanThreads + 3) & ~3;
    const int g0 = min(static_cast<long long>(p.n_pages), static_cast<long long>(tid) * chunk);
    const int g1 = min(p.n_pages, g0 + chunk);
    Sum2 mine = {0, 0}, total;
    for (int g = g0; g < g1; ++g) mine.x += p.ref[g] != 0;
    scan2(mine, total, s_warp);
    const int n = static_cast<int>(total.x);
    // x: live pages from n on, y: free ones below n; there are as many of either
    mine = {0, 0};
    for (int g = g0; g < g1; ++g) {
        const bool live = p.ref[g] != 0;
        if (live && g >= n) ++mine.x;
        if (!live && g < n) ++mine.y;
    }
    const Sum2 base = scan2(mine, total, s_warp);
    long long x = base.x, y = base.y;
    for (int g = g0; g < g1; ++g) {
        const bool live = p.ref[g] != 0;
        if (live && g >= n) w.copies[x++].x = g;
        if (!live && g < n) w.copies[y++].y = g;
        if (!live || g < n) w.place[g] = live ? g : -1;   // the list's are set below
    }
    __threadfence_block();
    __syncthreads();
    for (int i = tid; i < static_cast<int>(total.x); i += kPlanThreads) {
        const int2 c = w.copies[i];
        w.place[c.x] = c.y;
        p.ref[c.y] = p.ref[c.x];
        p.ref[c.x] = 0;
    }
    if (tid == 0) {
        w.header[0] = static_cast<int>(total.x);
        if (n_live != nullptr) *n_live = n;
    }
}

__global__ void __launch_bounds__(kCopyThreads) kv4_compact_kernel(const moe_kv4_pool p, void* ws, moe_dev_status* st) {
    pdl_wait();
    pdl_trigger();
    const PoolWs w = pool_ws(ws, p.n_pages);
    const long long entries = static_cast<long long>(p.S) * p.max_pages;
    for (long long i = static_cast<long long>(blockIdx.x) * kCopyThreads + threadIdx.x; i < entries;
         i += static_cast<long long>(gridDim.x) * kCopyThreads) {
        const int g = p.page_table[i];
        if (g == -1) continue;
        const int to = g >= 0 && g < p.n_pages ? w.place[g] : -1;
        if (to < 0) report(st, MOE_DEV_BAD_INDEX, g);     // no page in use: the entry stays
        else if (to != g) p.page_table[i] = to;
    }
    copy_pages(p, w);
}

}  // namespace

size_t kv4_pool_workspace(int S, int n_pages) {
    (void)S;
    return kHeader * sizeof(int) + static_cast<size_t>(n_pages) * (sizeof(int2) + 3 * sizeof(int));
}

cudaError_t launch_kv4_reserve(const moe_kv4_pool& p, const int32_t* n_new, void* ws, moe_dev_status* st, cudaStream_t s) {
    cudaError_t e = launch_pdl(kv4_reserve_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, p, n_new, ws, st);
    if (e != cudaSuccess) return e;
    return launch_pdl(kv4_copy_kernel, dim3(8 * sm_count()), dim3(kCopyThreads), 0, s, p, ws);
}

cudaError_t launch_kv4_assign(const moe_kv4_pool& p, const int32_t* parent, moe_dev_status* st, cudaStream_t s) {
    if (p.max_pages < 1) return cudaSuccess;
    constexpr int seq = (kAssignCols + 1) * sizeof(int);
    const size_t smem = static_cast<size_t>(p.S) * seq;
    // (the most that there is, so that threads with pools of other sizes do not undo each other's setting)
    cudaError_t e = cudaFuncSetAttribute(kv4_assign_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPoolMaxSeqs * seq);
    if (e != cudaSuccess) return e;
    return launch_pdl(kv4_assign_kernel, dim3((p.max_pages + kAssignCols - 1) / kAssignCols), dim3(kAssignThreads), smem, s, p, parent, st);
}

cudaError_t launch_kv4_compact(const moe_kv4_pool& p, int32_t* n_live, void* ws, moe_dev_status* st, cudaStream_t s) {
    cudaError_t e = launch_pdl(kv4_compact_plan_kernel, dim3(1), dim3(kPlanThreads), 0, s, p, n_live, ws);
    if (e != cudaSuccess) return e;
    return launch_pdl(kv4_compact_kernel, dim3(8 * sm_count()), dim3(kCopyThreads), 0, s, p, ws, st);
}

}  // namespace moe
