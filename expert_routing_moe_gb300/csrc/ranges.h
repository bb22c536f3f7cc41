// ranges.h -- the whole-number rules that keep the attention kernels and the
// pool's inside their buffers.  Nothing here needs CUDA, so that a test can run the rules on
// the host with every overflow trapped.
#pragma once

#ifdef __CUDACC__
#define MOE_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define MOE_HOST_DEVICE inline
#endif

namespace moe {

constexpr int kPageTokens = 64;   // MOE_KV4_PAGE

// Pages of a sequence of len >= 0 tokens, up to the largest number.
MOE_HOST_DEVICE int pages_of(int len) { return len / kPageTokens + (len % kPageTokens != 0); }

// Whether rows q0 .. q1-1 of T can be the last ones of a sequence of len
// tokens whose table has max_pages pages, for any four numbers.
MOE_HOST_DEVICE bool rows_fit(int q0, int q1, int len, int T, int max_pages) {
    return 0 <= q0 && q0 <= q1 && q1 <= T && 0 <= len && len <= static_cast<long long>(max_pages) * kPageTokens;
}

// The window that the kernels get for one that a caller gave (0: no window).  One that no table of max_pages pages
// is longer than hides nothing.  Places start at -T (rows before their sequence), so a place less the window stays
// above -2^31; -1 for the tables of 2^31 tokens where it would not.
MOE_HOST_DEVICE int kernel_window(int window, int T, int max_pages) {
    if (window >= static_cast<long long>(max_pages) * kPageTokens) return 0;
    return static_cast<long long>(window) + T > 0x7fffffff ? -1 : window;
}

// The CTAs that hold pieces of a tile of `units` units, the first being unit `item`, as CTA bid, which holds one of
// them and starts with unit u0, finds them.  even: each tile has per_item CTAs with `share` units each; else CTA b holds units b *
// share on, whatever tile they belong to, and per_item may be 0.  A tile's units are a 32-bit number.
struct CtaRange {
    int first, last;
};
MOE_HOST_DEVICE CtaRange tile_ctas(bool even, int bid, int per_item, long long share, long long u0, long long item, int units) {
    CtaRange r;
    if (even) {
        r.first = bid - bid % per_item;
        r.last = r.first + (units - 1) / static_cast<int>(share);
    } else {
        const unsigned sh = static_cast<unsigned>(share);
        r.first = item >= u0 ? bid : bid - static_cast<int>((static_cast<unsigned>(u0 - item) + sh - 1) / sh);
        r.last = r.first + static_cast<int>((static_cast<unsigned>(item - share * r.first) + units - 1) / sh);
    }
    return r;
}

}  // namespace moe
