// attn_kv4.cuh -- what the two attention kernels over the 4-bit cache share:
// the arguments, the sequences' rows and pages, the walk over the units of
// work, and the output's rounding.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "kv4.cuh"
#include "ranges.h"

namespace moe {

static_assert(kPageTokens == MOE_KV4_PAGE, "ranges.h has the page's size");
constexpr float kLog2e = 0x1.715476p+0f;
constexpr float kLn2f = 0x1.62e430p-1f;

// What both attention kernels get.
struct AttnArgs {
    const __nv_bfloat16* q;
    long long ld_q;
    int T, n_q, group;          // group: query heads of a key head
    moe_kv4_cache c;
    const int32_t* q_start;
    float scale;
    int window;
    __nv_bfloat16* out;
    long long ld_out;
    float* lse;
    int rows_lo, rows_hi;       // the kernel takes the sequences with so many rows
    int* counters;              // one of a CTA: arrivals at the tile that starts there and goes on
    float* partial;             // [CTAs][2] slots of a tile's O, m and l
    moe_dev_status* st;
};

// A sequence's rows and what they may see.
struct Seq {
    int q0, n, len;
};
__device__ __forceinline__ Seq load_seq(const AttnArgs& a, int s) {
    Seq r;
    r.q0 = a.q_start[s];
    const int q1 = a.q_start[s + 1];
    r.len = a.c.seq_len[s];
    const bool fit = rows_fit(r.q0, q1, r.len, a.T, a.c.max_pages);
    r.n = fit ? q1 - r.q0 : 0;
    if (!fit) r.len = -1;
    return r;
}

// The tile's pages [lo, hi): those that its first row's window or its last row's place reaches.
template <int NR>
__device__ __forceinline__ void tile_pages(const AttnArgs& a, const Seq& s, int tile, int& lo, int& hi) {
    const int i0 = tile * NR / a.group, i1 = min(s.n - 1, (tile * NR + NR - 1) / a.group);
    const int p0 = s.len - s.n + i0, p1 = s.len - s.n + i1;
    hi = p1 >= 0 ? p1 / kPage + 1 : 0;
    lo = a.window > 0 && p0 - a.window + 1 > 0 ? min((p0 - a.window + 1) / kPage, hi) : 0;
}
template <int NR>
__device__ __forceinline__ int seq_tiles(const AttnArgs& a, const Seq& s) {
    const int rows = s.n * a.group;
    return rows < a.rows_lo || rows > a.rows_hi ? 0 : (rows + NR - 1) / NR;
}
// Units of one key head of a sequence, and the most that a tile has; a tile
// that sees nothing still has one, to write its rows.
template <int NR>
__device__ __forceinline__ int seq_units(const AttnArgs& a, const Seq& s, int& most) {
    int u = 0;
    const int tiles = seq_tiles<NR>(a, s);
    for (int i = 0; i < tiles; ++i) {
        int lo, hi;
        tile_pages<NR>(a, s, i, lo, hi);
        const int n = max(1, hi - lo);
        most = max(most, n);
        u += n;
    }
    return u;
}

// A place in the sequence of units: sequence, key head, tile, and page of the tile.
template <int NR>
struct Cursor {
    int s, h, tile, tiles;
    int page, lo, hi;          // the tile's pages; lo == hi: one unit without a page
    int item_left;             // units of the tile from here on
    long long item_begin;      // unit of the tile's first page
    long long unit;
    Seq q;

    __device__ void set_tile(const AttnArgs& a) {
        tile_pages<NR>(a, q, tile, lo, hi);
        page = lo;
        item_left = max(1, hi - lo);
        item_begin = unit;
    }
    __device__ void next_seq(const AttnArgs& a) {   // the next sequence with rows
        do {
            ++s;
            if (s >= a.c.S) { tiles = 0; return; }
            q = load_seq(a, s);
            tiles = seq_tiles<NR>(a, q);
        } while (tiles == 0);
        h = 0;
        tile = 0;
    }
    __device__ void next_item(const AttnArgs& a) {
        if (++tile >= tiles) {
            tile = 0;
            if (++h >= a.c.n_kv) next_seq(a);
        }
        if (s < a.c.S) set_tile(a);
    }
    __device__ void advance(const AttnArgs& a) {
        ++unit;
        ++page;
        if (--item_left == 0) next_item(a);
    }
    // from the first unit of (sequence s, head 0) to unit `to` of the same sequence
    __device__ void seek(const AttnArgs& a, int seq, long long seq_begin, int seq_head_units, long long to) {
        s = seq;
        q = load_seq(a, s);
        tiles = seq_tiles<NR>(a, q);
        h = static_cast<int>(to - seq_begin) / seq_head_units;
        unit = seq_begin + static_cast<long long>(h) * seq_head_units;
        tile = 0;
        set_tile(a);
        while (unit + item_left <= to) {
            unit += item_left;
            if (++tile >= tiles) break;   // cannot happen: `to` is in this head
            set_tile(a);
        }
        const int skip = static_cast<int>(to - unit);
        page += skip;
        item_left -= skip;
        unit = to;
    }
    __device__ bool same_item(const Cursor& o) const { return item_begin == o.item_begin; }
};

__device__ __forceinline__ float ex2(float u) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(u));
    return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    uint32_t r;
    memcpy(&r, &h, 4);
    return r;
}
template <int D>
__device__ __forceinline__ void write_out4(const AttnArgs& a, const Seq& s, int h, int r, int d, float4 v) {
    __nv_bfloat16* p = a.out + static_cast<long long>(s.q0 + r / a.group) * a.ld_out +
                       static_cast<long long>(h * a.group + r % a.group) * D + d;
    const __nv_bfloat162 x = __floats2bfloat162_rn(v.x, v.y), y = __floats2bfloat162_rn(v.z, v.w);
    uint2 u;
    memcpy(&u.x, &x, 4);
    memcpy(&u.y, &y, 4);
    *reinterpret_cast<uint2*>(p) = u;
}
__device__ __forceinline__ void write_lse(const AttnArgs& a, const Seq& s, int h, int r, float m, float l) {
    if (a.lse == nullptr) return;
    a.lse[static_cast<long long>(s.q0 + r / a.group) * a.n_q + h * a.group + r % a.group] = l > 0.f || l != l ? m * kLn2f + logf(l) : -INFINITY;
}

// Workspace: the counters of both kernels, then the streaming kernel's pieces, then the prompt kernel's.  The counters
// lie where no call writes pieces, whatever its sizes: so they are zero between any two calls.
constexpr int kPromptMaxCtas = 160;
constexpr size_t kStreamCounterBytes = 2048;                          // one for each CTA
constexpr size_t kPromptCounterBytes = kPromptMaxCtas * 8 * 4;        // one for each softmax warp of each CTA
constexpr size_t kCounterBytes = kStreamCounterBytes + kPromptCounterBytes;
cudaError_t launch_attn_prefill(const AttnArgs& a, cudaStream_t s);
size_t attn_prefill_pieces(int D);

}  // namespace moe
