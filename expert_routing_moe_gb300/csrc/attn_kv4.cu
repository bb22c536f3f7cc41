// attn_kv4.cu -- attention over the 4-bit paged cache for few query rows a
// sequence (single tokens, drafts): a streaming kernel bound by the cache's
// bytes.
//
// For one (sequence, key head) the rows are the new tokens' query heads of
// that key head, token-major.  A tile of 8 or 16 rows takes one pass over its
// pages with the running maximum m, sum l and sum O of a softmax:
//     S^T = K Q^T (64 tokens x rows),  P = 2^(f S - m),  O^T += V^T P^T
// on m16n8k16 tensor-core products with the cached numbers as the 16-row
// operand, so that eight query heads that share a key head fill the products'
// other side and no row is padding.  The layout of a page puts what a lane's
// fragments need into 16-byte runs: a warp reads a head's page (9216 bytes at
// D = 128) with 18 shared-memory loads a lane, and a fragment register is one
// conversion of a byte of codes and one multiplication by a scale, both
// exact.
//
// Work: the pages of all tiles form one sequence of units, cut into equal
// runs for the CTAs and again for their warps, whatever the contexts' lengths
// are.  A warp fetches a page ahead of the one it works on (one bulk copy each).  Tiles that
// cross warps are joined in shared memory and tiles that cross CTAs by the
// last CTA to arrive, in the order of the pages: nothing waits, and
// results do not depend on timing.
//
// P is rounded to fp16; m, l and O are fp32.  The maximum's P is 2^14, so that
// fp16 holds 11 bits of probabilities down to 2^-28 of the maximum (each is off by 2^-11
// of itself, an eighth of the bf16 output's half step) and those below by 2^-39 of
// the maximum each, which a million of them make 2^-19.  With the maximum at 1
// and the last bits at 2^-24, 100,000 keys at 2^-25 of the first lost the 0.3% that was theirs.
//
// What bounds it: a warp's pages one after the other and, for short contexts, the
// chain of dependent steps.  Above 131071 tokens of one sequence (32 heads on 4,
// other inputs from call to call) another page costs what 6.1 TB/s take, 0.91 of a copy: 26.9,
// 39.6, 52.4, 89.9 us for 131071, 262144, 400000 and 800000 tokens; some 14 us are the launch, the
// search for a CTA's first page, the first pages and the joins.  32 sequences of up to 8192
// (18.6 MB) take 15.8 us, 333 tokens 7.9 us.  fp32 arithmetic or a wider
// conversion of the codes would take the issue slots that the loads leave: a
// page costs a warp about 1000 instructions and 42% of the slots are used.
#include <cuda_bf16.h>

#include "attn_kv4.cuh"
#include "common.cuh"
#include "kv4.cuh"
#include "launch.h"
#include "tmap.h"

namespace moe {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 2;
constexpr int kMaxCtas = 160;       // one for each SM
constexpr int kAhead = 16;          // pieces in flight when a tile's are joined
constexpr int kSiteKvPage = 21;
// log2 of the largest P: m is the running maximum less this
constexpr float kRoom = 14.f;

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
template <int N>
__device__ __forceinline__ void lds(uint32_t (&v)[N], const uint8_t* p) {
    if constexpr (N == 4) {
        const uint4 x = *reinterpret_cast<const uint4*>(p);
        v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
    } else {
        const uint2 x = *reinterpret_cast<const uint2*>(p);
        v[0] = x.x; v[1] = x.y;
    }
}

// A tile's state in one warp.  Lane (g, t) = (lane / 4, lane % 4) holds, of
// row 8 n + 2 t + c, the numbers (D/8) g + 2 i + e of O in o[n][i][2 e + c].
template <int D, int NT>
struct Tile {
    static constexpr int KS = D / 16;     // products of 16 numbers of a head
    static constexpr int MD = D / 16;     // 16-row tiles of V^T
    uint32_t qf[NT][KS][2];
    float f[NT][2];                       // the scores' factor of row 8 n + 2 t + c, in powers of two
    float m[NT][2], l[NT][2];             // m: the scores' maximum less kRoom
    float o[NT][MD][4];
};

// The tile's queries as fragments: row 8 n + g, numbers (D/4) t + 4 ks + 0..3.
// A row is multiplied by a power of two that puts its largest magnitude into
// [2^10, 2^11): its bf16 numbers down to 2^-27 of that are then exact in fp16.
template <int D, int NT>
__device__ __forceinline__ void load_queries(Tile<D, NT>& w, const AttnArgs& a, const Seq& s, int h, int tile, int lane) {
    constexpr int NR = 8 * NT;
    const int g = lane >> 2, t = lane & 3;
    const float k_scale = a.c.k_scale != nullptr ? a.c.k_scale[h] : 1.f;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        const int r = tile * NR + 8 * n + g;
        const bool live = r < s.n * a.group;
        uint32_t raw[D / 8];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) raw[i] = 0u;
        if (live) {
            const __nv_bfloat16* p = a.q + static_cast<long long>(s.q0 + r / a.group) * a.ld_q +
                                     static_cast<long long>(h * a.group + r % a.group) * D + (D / 4) * t;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const uint4 v = reinterpret_cast<const uint4*>(p)[i];
                raw[4 * i] = v.x; raw[4 * i + 1] = v.y; raw[4 * i + 2] = v.z; raw[4 * i + 3] = v.w;
            }
        }
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
            top = fmaxf(top, fmaxf(fabsf(__uint_as_float(raw[i] << 16)), fabsf(__uint_as_float(raw[i] & 0xffff0000u))));
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
        top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
        // exponent of the power of two, 0 for rows that are zero or not finite
        int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
        e = (top > 0.f && e < 128) ? max(-100, min(100, 10 - e)) : 0;
        const float up = __int_as_float((e + 127) << 23);
        float f = a.scale * kLog2e * k_scale * __int_as_float((127 - e) << 23);
        f = live ? f : 0.f;
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
            w.qf[n][i / 2][i & 1] = pack_f16(__uint_as_float(raw[i] << 16) * up, __uint_as_float(raw[i] & 0xffff0000u) * up);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            w.f[n][c] = __shfl_sync(kFull, f, (2 * t + c) * 4);
            w.m[n][c] = -INFINITY;
            w.l[n][c] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) w.o[n][i][c] = 0.f;
    }
}

// One page of the tile.  `base`: the head's part of the page in shared memory.
template <int D, int NT>
__device__ __forceinline__ void do_page(Tile<D, NT>& w, const AttnArgs& a, const uint8_t* base, const Seq& s, int tile,
                                        int page, int lane) {
    using L = Kv4Layout<D>;
    constexpr int NR = 8 * NT;
    constexpr int W = D / 32;                   // code words of a lane's run
    const int g = lane >> 2, t = lane & 3;

    // S^T: rows 16 mt + 8 e + g (tokens), columns 8 n + 2 t + c (queries) in acc[mt][n][2 e + c]
    float acc[4][NT][4];
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) acc[mt][n][c] = 0.f;
    uint32_t ks[W];                             // scales of tokens g + 8 i: R bytes each
    lds<W>(ks, base + L::kScales + (t * 8 + g) * 8 * L::R);
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
        uint32_t w0[W], w1[W];
        lds<W>(w0, base + (16 * mt + g) * (D / 2) + t * (D / 8));
        lds<W>(w1, base + (16 * mt + 8 + g) * (D / 2) + t * (D / 8));
        uint32_t s0[L::R], s1[L::R];            // both halves the same scale
        if constexpr (L::R == 2) {
            const uint32_t p0 = e4m3x2_to_f16(ks[mt] & 0xffffu), p1 = e4m3x2_to_f16(ks[mt] >> 16);
            s0[0] = __byte_perm(p0, 0, 0x1010); s0[1] = __byte_perm(p0, 0, 0x3232);
            s1[0] = __byte_perm(p1, 0, 0x1010); s1[1] = __byte_perm(p1, 0, 0x3232);
        } else {
            const uint32_t p = e4m3x2_to_f16((ks[mt / 2] >> (16 * (mt & 1))) & 0xffffu);
            s0[0] = __byte_perm(p, 0, 0x1010);
            s1[0] = __byte_perm(p, 0, 0x3232);
        }
#pragma unroll
        for (int k2 = 0; k2 < W; ++k2) {        // a word: two products' worth
            uint32_t c0[4], c1[4];
            e2m1x8_to_f16(w0[k2], c0[0], c0[1], c0[2], c0[3]);
            e2m1x8_to_f16(w1[k2], c1[0], c1[1], c1[2], c1[3]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int k = 2 * k2 + e, r = k / 4;
                const uint32_t af[4] = {hmul2_u(c0[2 * e], s0[r]), hmul2_u(c1[2 * e], s1[r]),
                                        hmul2_u(c0[2 * e + 1], s0[r]), hmul2_u(c1[2 * e + 1], s1[r])};
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_f16(acc[mt][n], af, w.qf[n][k][0], w.qf[n][k][1]);
            }
        }
    }

    // softmax: scale, hide, maximum over the page
    const int key0 = page * kPage;
    const int i_last = min(s.n - 1, (tile * NR + NR - 1) / a.group);
    const int p_first = s.len - s.n + tile * NR / a.group, p_last = s.len - s.n + i_last;
    const bool edge = key0 + kPage - 1 > p_first || (a.window > 0 && key0 <= p_last - a.window);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float top[2] = {-INFINITY, -INFINITY};
        if (edge) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int p = s.len - s.n + (tile * NR + 8 * n + 2 * t + c) / a.group;
                const int last = min(p, s.len - 1), first = a.window > 0 ? p - a.window + 1 : 0;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int key = key0 + 8 * i + g;
                    float& x = acc[i >> 1][n][2 * (i & 1) + c];
                    x = key <= last && key >= first ? x * w.f[n][c] : -INFINITY;
                    top[c] = fmaxf(top[c], x);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float& x = acc[i >> 1][n][2 * (i & 1) + c];
                    x *= w.f[n][c];
                    top[c] = fmaxf(top[c], x);
                }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            top[c] = fmaxf(top[c], __shfl_xor_sync(kFull, top[c], 4));
            top[c] = fmaxf(top[c], __shfl_xor_sync(kFull, top[c], 8));
            top[c] = fmaxf(top[c], __shfl_xor_sync(kFull, top[c], 16));
            top[c] = fmaxf(top[c] - kRoom, w.m[n][c]);
        }
        if (__any_sync(kFull, top[0] > w.m[n][0] || top[1] > w.m[n][1])) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                // while nothing has been seen m is -inf and O, l are 0
                const float r = w.m[n][c] == -INFINITY ? 0.f : ex2(w.m[n][c] - top[c]);
                w.m[n][c] = top[c];
                w.l[n][c] *= r;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    w.o[n][i][c] *= r;
                    w.o[n][i][2 + c] *= r;
                }
            }
        }
        const float m0 = w.m[n][0] == -INFINITY ? 0.f : w.m[n][0], m1 = w.m[n][1] == -INFINITY ? 0.f : w.m[n][1];
        float sum0 = 0.f, sum1 = 0.f;               // of the page first: a large l loses less of small terms
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float& x0 = acc[i >> 1][n][2 * (i & 1)];
            float& x1 = acc[i >> 1][n][2 * (i & 1) + 1];
            x0 = ex2(x0 - m0);
            x1 = ex2(x1 - m1);
            sum0 += x0;
            sum1 += x1;
        }
        w.l[n][0] += sum0;
        w.l[n][1] += sum1;
    }

    // O^T += V^T P^T, 16 tokens at a time
    uint32_t vs[4];                             // scale pairs of tokens 8 i + 2 t, 8 i + 2 t + 1
    lds<4>(vs, base + L::vScales + (((D == 128 ? g : g / 2) * 4 + t) * 8) * 2);
    // tokens that the sequence does not have: their bytes may be anything, a NaN scale among it
    const int left = s.len - key0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t sc[2], v[2][W];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int i = 2 * k + e;
            uint32_t two = (vs[i / 2] >> (16 * (i & 1))) & 0xffffu;
            if (left < kPage) {
                const int tok = 8 * i + 2 * t;
                two = tok + 1 < left ? two : (tok < left ? (two & 0xffu) : 0u);
            }
            sc[e] = e4m3x2_to_f16(two);
            lds<W>(v[e], base + L::vCodes + ((i * 8 + g) * 4 + t) * L::U);
        }
        uint32_t pf[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                pf[n][e] = transpose8x8(pack_f16(acc[k][n][2 * e], acc[k][n][2 * e + 1]));
#pragma unroll
        for (int j = 0; j < W; ++j) {           // a word: four numbers of two tokens, i.e. two tiles of V^T
            uint32_t c0[4], c1[4];
            e2m1x8_to_f16(v[0][j], c0[0], c0[1], c0[2], c0[3]);
            e2m1x8_to_f16(v[1][j], c1[0], c1[1], c1[2], c1[3]);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t af[4] = {hmul2_u(c0[2 * e], sc[0]), hmul2_u(c0[2 * e + 1], sc[0]),
                                        hmul2_u(c1[2 * e], sc[1]), hmul2_u(c1[2 * e + 1], sc[1])};
#pragma unroll
                for (int n = 0; n < NT; ++n) mma_f16(w.o[n][2 * j + e], af, pf[n][0], pf[n][1]);
            }
        }
    }
}

// The tile's sums over the lanes of a row.
template <int D, int NT>
__device__ __forceinline__ void sum_lanes(Tile<D, NT>& w) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            w.l[n][c] += __shfl_xor_sync(kFull, w.l[n][c], 4);
            w.l[n][c] += __shfl_xor_sync(kFull, w.l[n][c], 8);
            w.l[n][c] += __shfl_xor_sync(kFull, w.l[n][c], 16);
        }
}

// Where a tile's pieces lie in shared memory: O [NR][D + 4], then m [NR], l [NR].
template <int D, int NR>
struct Piece {
    static constexpr int ld = D + 4;
    static constexpr int m = NR * ld, l = m + NR, floats = l + NR;
};
struct PieceInfo {
    long long item;            // first unit of the tile, -1: none
    int h, tile, units;        // units of the whole tile
    float v_scale;
    Seq q;
};

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, 1) attn_kv4_stream_kernel(const AttnArgs a) {
    using L = Kv4Layout<D>;
    constexpr int NR = 8 * NT;
    using P = Piece<D, NR>;
    constexpr int kRing = kStages * L::bytes;
    static_assert(P::floats * 4 <= kRing, "a warp's last piece fits its ring");
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ __align__(8) uint64_t bars[kWarps * kStages];
    __shared__ PieceInfo info[2 * kWarps];
    __shared__ long long s_scan[kWarps], w_begin[kWarps], s_u0, s_u1;
    __shared__ int s_items[kWarps], s_most[kWarps], w_units[kWarps], w_seq[kWarps];
    __shared__ PieceInfo s_piece[2];
    __shared__ int s_last[2], s_b0[2], s_n[2];
    __shared__ volatile int s_abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kWarps * kStages; ++i) mbar_init(smem_u32(&bars[i]), 1);
        fence_mbar_init();
        s_abort = 0;
        s_last[0] = s_last[1] = 0;
        s_n[0] = s_n[1] = 0;
    }
    pdl_wait();
    pdl_trigger();

    // The units of all sequences; every CTA adds them up for itself.  (A
    // sequence's own are a 32-bit number: its pages fit the device's memory.)
    const int per = (a.c.S + kThreads - 1) / kThreads;
    const int sa = min(a.c.S, static_cast<int>(threadIdx.x) * per), sb = min(a.c.S, sa + per);
    long long mine = 0;
    int items = 0, most = 0, hu = 0;
    Seq q0 = {0, 0, 0};
    for (int s = sa; s < sb; ++s) {
        q0 = load_seq(a, s);
        if (q0.len < 0 && blockIdx.x == 0) report(a.st, MOE_DEV_BAD_INDEX, s);
        hu = seq_units<NR>(a, q0, most);
        mine += static_cast<long long>(hu) * a.c.n_kv;
        items += seq_tiles<NR>(a, q0) * a.c.n_kv;
    }
    long long inc = mine;
    int inc_items = items;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const long long v = __shfl_up_sync(kFull, inc, off);
        const int k = __shfl_up_sync(kFull, inc_items, off);
        if (lane >= off) { inc += v; inc_items += k; }
    }
    most = __reduce_max_sync(kFull, most);
    if (lane == 31) {
        s_scan[warp] = inc;
        s_items[warp] = inc_items;
        s_most[warp] = most;
    }
    __syncthreads();
    long long before = 0, total = 0;
    int items_before = 0, all_items = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
        if (i < warp) { before += s_scan[i]; items_before += s_items[i]; }
        total += s_scan[i];
        all_items += s_items[i];
        most = max(most, s_most[i]);
    }
    before += inc - mine;
    items_before += inc_items - items;
    if (total == 0) return;
    // Few short tiles: one for each CTA, so that none is joined across CTAs.  Else equal runs
    // of units for the CTAs, at least a page for each warp.  (Four heads of keys; batches of 4, 16 and 32 sequences
    // with 333, 500 and 1000 tokens: 8.3, 8.6, 10.6 us by tiles, 10.6, 11.2, 12.8 by runs; one of 333: 8.3, 8.2.)
    const bool by_item = all_items <= static_cast<int>(gridDim.x) && most <= 2 * kWarps;
    // Few tiles of one size (a batch of one or two): as many CTAs for each, so that no CTA has two tiles to join.
    // (Four tiles of 32, 47, 141, 625, 2048 pages: 10.7, 10.7, 11.6, 15.8, 25.0 us; with runs across tiles 10.1, 11.6,
    // 12.2, 17.0, 28.3.  16 and 32 tiles of 141 pages: 12.3, 12.7, with runs 12.1, 12.3.)
    const int per_item = static_cast<int>(gridDim.x) / max(1, all_items);
    const bool even = !by_item && per_item >= 16 && most > 4 * kWarps && total == static_cast<long long>(most) * all_items;
    const int bid = static_cast<int>(blockIdx.x);
    long long share = 0, u0, u1;
    if (by_item) {
        if (bid >= all_items) return;
        if (bid >= items_before && bid < items_before + items) {
            long long b = before;
            int k = items_before;
            for (int s = sa; s < sb; ++s) {
                const Seq q = per == 1 ? q0 : load_seq(a, s);
                const int tiles = seq_tiles<NR>(a, q), n = tiles * a.c.n_kv;
                if (bid >= k + n) {
                    int unused = 0;
                    b += static_cast<long long>(per == 1 ? hu : seq_units<NR>(a, q, unused)) * a.c.n_kv;
                    k += n;
                    continue;
                }
                const int h = (bid - k) / tiles, tile = (bid - k) - h * tiles;
                int unused = 0, lo, hi;
                b += static_cast<long long>(h) * (per == 1 ? hu : seq_units<NR>(a, q, unused));
                for (int i = 0; i < tile; ++i) {
                    tile_pages<NR>(a, q, i, lo, hi);
                    b += max(1, hi - lo);
                }
                tile_pages<NR>(a, q, tile, lo, hi);
                s_u0 = b;
                s_u1 = b + max(1, hi - lo);
                break;
            }
        }
        __syncthreads();
        u0 = s_u0;
        u1 = s_u1;
    } else if (even) {
        share = max(kWarps, (most + per_item - 1) / per_item);
        if (bid >= per_item * all_items) return;
        const long long begin = static_cast<long long>(bid / per_item) * most;
        u0 = begin + share * (bid % per_item);
        u1 = min(begin + most, u0 + share);
        if (u0 >= u1) return;
    } else {
        const int grid = static_cast<int>(gridDim.x);
        share = total < 0x7fffffff - grid ? (static_cast<int>(total) + grid - 1) / grid : (total + grid - 1) / grid;
        share = share < kWarps ? kWarps : share;
        u0 = min(total, share * bid);
        u1 = min(total, u0 + share);
        if (u0 >= u1) return;
    }
    const long long n_cta = u1 - u0;
    const long long w0 = u0 + n_cta * warp / kWarps, w1 = u0 + n_cta * (warp + 1) / kWarps;
    // The sequence that a warp's run starts in is found by the thread that added it up.
    if (mine > 0 && before < u1 && before + mine > u0) {
        long long b = before;
        for (int s = sa; s < sb; ++s) {
            int unused = 0;
            const int h_units = per == 1 ? hu : seq_units<NR>(a, load_seq(a, s), unused);
            const long long u = static_cast<long long>(h_units) * a.c.n_kv;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                const long long at = u0 + n_cta * i / kWarps;
                if (at >= b && at < b + u) {
                    w_seq[i] = s;
                    w_begin[i] = b;
                    w_units[i] = h_units;
                }
            }
            b += u;
        }
    }
    if (lane < 2) info[2 * warp + lane].item = -1;
    __syncthreads();

    uint8_t* ring = smem + warp * kRing;
    float* pieces = reinterpret_cast<float*>(ring);
    const uint32_t bar0 = smem_u32(&bars[warp * kStages]);
    if (w0 < w1) {
        Cursor<NR> rd, wr;      // the unit being computed, and the next one to fetch
        rd.seek(a, w_seq[warp], w_begin[warp], w_units[warp], w0);
        wr = rd;
        uint32_t fetched = 0;   // bit st: the stage holds a page
        auto page_of = [&](const Cursor<NR>& c) {
            return c.page < c.hi ? a.c.page_table[static_cast<long long>(c.s) * a.c.max_pages + c.page] : -1;
        };
        int next_id = page_of(wr);
        auto fetch = [&](int stage) {
            if (wr.unit >= w1) { fetched &= ~(1u << stage); return; }
            const int id = next_id;
            const bool ok = wr.page < wr.hi && id >= 0 && id < a.c.n_pages;
            if (!ok && wr.page < wr.hi && lane == 0) report(a.st, MOE_DEV_BAD_INDEX, id);
            if (ok) {
                if (lane == 0) {
                    const uint8_t* src = static_cast<const uint8_t*>(a.c.pages) + (static_cast<long long>(id) * a.c.n_kv + wr.h) * L::bytes;
                    mbar_arrive_expect_tx(bar0 + 8 * stage, L::bytes);
                    bulk_copy_g2s(smem_u32(ring + stage * L::bytes), src, L::bytes, bar0 + 8 * stage);
                }
                fetched |= 1u << stage;
            } else {
                fetched &= ~(1u << stage);
            }
            wr.advance(a);
            if (wr.unit < w1) next_id = page_of(wr);
        };
        for (int st = 0; st < kStages; ++st) fetch(st);

        Tile<D, NT> w;
        load_queries(w, a, rd.q, rd.h, rd.tile, lane);
        bool piece_open = rd.page != rd.lo;     // began in an earlier run
        int stage = 0;
        uint32_t phases = 0;                    // bit st: parity that the stage completes next
        bool ok = true;
        while (ok) {
            if (fetched & (1u << stage)) {
                ok = mbar_wait(bar0 + 8 * stage, (phases >> stage) & 1u, &s_abort, a.st, kSiteKvPage);
                ok = __all_sync(kFull, ok);
                phases ^= 1u << stage;
                if (!ok) break;
                do_page<D, NT>(w, a, ring + stage * L::bytes, rd.q, rd.tile, rd.page, lane);
                __syncwarp();
            }
            const Cursor<NR> was = rd;
            rd.advance(a);
            const bool item_done = rd.unit >= w1 || !rd.same_item(was);
            fetch(stage);
            stage = stage + 1 == kStages ? 0 : stage + 1;
            if (!item_done) continue;
            sum_lanes(w);
            const bool complete = !piece_open && was.item_left == 1;
            const int g = lane >> 2, t = lane & 3;
            if (complete) {
                const float vs = a.c.v_scale != nullptr ? a.c.v_scale[was.h] : 1.f;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int r = was.tile * NR + 8 * n + 2 * t + c;
                        if (r >= was.q.n * a.group) continue;
                        const float inv = w.l[n][c] == 0.f ? 0.f : vs / w.l[n][c];
#pragma unroll
                        for (int i = 0; i < D / 16; i += 2)
                            write_out4<D>(a, was.q, was.h, r, (D / 8) * g + 2 * i,
                                          make_float4(w.o[n][i][c] * inv, w.o[n][i][2 + c] * inv, w.o[n][i + 1][c] * inv,
                                                      w.o[n][i + 1][2 + c] * inv));
                        if (g == 0) write_lse(a, was.q, was.h, r, w.m[n][c], w.l[n][c]);
                    }
            } else {
                // only a run's first and last tile can be incomplete: the first has a place after the
                // rings, the last takes the ring, which is free by then
                float* dst = rd.unit >= w1 ? pieces : reinterpret_cast<float*>(smem + kWarps * kRing) + warp * P::floats;
                const int which = rd.unit >= w1 ? 1 : 0;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const int r = 8 * n + 2 * t + c;
#pragma unroll
                        for (int i = 0; i < D / 16; i += 2)
                            *reinterpret_cast<float4*>(dst + r * P::ld + (D / 8) * g + 2 * i) =
                                make_float4(w.o[n][i][c], w.o[n][i][2 + c], w.o[n][i + 1][c], w.o[n][i + 1][2 + c]);
                        if (g == 0) {
                            dst[P::m + r] = w.m[n][c];
                            dst[P::l + r] = w.l[n][c];
                        }
                    }
                if (lane == 0) {
                    PieceInfo& p = info[2 * warp + which];
                    p.item = was.item_begin;
                    p.h = was.h;
                    p.tile = was.tile;
                    p.units = max(1, was.hi - was.lo);
                    p.v_scale = a.c.v_scale != nullptr ? a.c.v_scale[was.h] : 1.f;
                    p.q = was.q;
                }
            }
            if (rd.unit >= w1) break;
            load_queries(w, a, rd.q, rd.h, rd.tile, lane);
            piece_open = false;
        }
        if (!ok) {
            // copies still in flight land before the CTA's shared memory is given up
            for (int st = 0; st < kStages; ++st)
                if (fetched & (1u << st)) mbar_drain(bar0 + 8 * st, (phases >> st) & 1u);
        }
    }
    __syncthreads();
    if (s_abort) return;

    // Join the pieces of each tile, in the order of the pages: a thread's part
    // is four numbers of a row at a time.
    const float* first_pieces = reinterpret_cast<const float*>(smem + kWarps * kRing);
    auto piece = [&](int i) {
        return (i & 1) ? reinterpret_cast<const float*>(smem + (i >> 1) * kRing) : first_pieces + (i >> 1) * P::floats;
    };
    constexpr int kPieces = 2 * kWarps, kRowW = kPieces + 2;
    float* const weight = reinterpret_cast<float*>(smem + kWarps * kRing) + kWarps * P::floats;   // [NR][kMaxCtas] at the end
    static_assert(kWarps * kRowW <= kMaxCtas, "the warps' weights fit");
    float* const mine_w = weight + warp * NR * kRowW;
    uint32_t have = 0, starts = 0;           // pieces that there are, and those that are a tile's first
    long long seen = -1;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        const long long id = info[i].item;
        if (id < 0) continue;
        have |= 1u << i;
        if (id != seen) starts |= 1u << i;
        seen = id;
    }
    // one tile: all threads; several: the threads in two, four or eight groups that take them in turn
    const int tiles_here = __popc(starts);
    const int groups = tiles_here <= 1 ? 1 : tiles_here == 2 ? 2 : tiles_here <= 4 ? 4 : 8;
    const int g_threads = kThreads / groups, g_tid = static_cast<int>(threadIdx.x) % g_threads;
    int turn = static_cast<int>(threadIdx.x) / g_threads;
    for (uint32_t left = starts; left != 0; left &= left - 1) {
        if (turn-- != 0) continue;
        turn = groups - 1;
        const int i = __ffs(left) - 1;
        const PieceInfo p = info[i];
        // the tile's pieces: from its first to the next tile's
        const uint32_t rest = left & (left - 1);
        const uint32_t set = have & ~((1u << i) - 1) & (rest != 0 ? (1u << (__ffs(rest) - 1)) - 1 : ~0u);
        const Seq q = p.q;
        const float vs = p.v_scale;
        const bool here = p.item >= u0 && p.item + p.units <= u1;   // the whole tile is this CTA's
        const int my_slot = p.item < u0 ? 0 : 1;
        float* part = a.partial + (static_cast<long long>(bid) * 2 + my_slot) * (NR * (D + 2));
        // each row's weights 2^(m - max) of the pieces, and its sum; every warp for itself, a lane for a row and
        // every (32 / NR)th piece
        {
            constexpr int kStep = 32 / NR;
            const int r = lane % NR;
            float mk[kPieces / kStep], lk[kPieces / kStep], m = -INFINITY, l = 0.f;
#pragma unroll
            for (int i = 0; i < kPieces / kStep; ++i) {
                const int k = lane / NR + i * kStep;
                const bool in = (set >> k) & 1;
                mk[i] = in ? piece(k)[P::m + r] : -INFINITY;
                lk[i] = in ? piece(k)[P::l + r] : 0.f;
                m = fmaxf(m, mk[i]);
            }
#pragma unroll
            for (int off = NR; off < 32; off <<= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, off));
#pragma unroll
            for (int i = 0; i < kPieces / kStep; ++i) {
                // a piece that has seen nothing has l = 0, or a NaN that stays
                const float e = mk[i] == -INFINITY ? (lk[i] == lk[i] ? 0.f : 1.f) : ex2(mk[i] - m);
                mine_w[r * kRowW + lane / NR + i * kStep] = e;
                l = fmaf(e, lk[i], l);
            }
#pragma unroll
            for (int off = NR; off < 32; off <<= 1) l += __shfl_xor_sync(kFull, l, off);
            if (lane < NR) {
                mine_w[r * kRowW + kPieces] = m;
                mine_w[r * kRowW + kPieces + 1] = l;
            }
        }
        __syncwarp();
        for (int x = g_tid; x < NR * (D / 4); x += g_threads) {
            const int r = x / (D / 4), d = x % (D / 4) * 4;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (uint32_t b = set; b != 0; b &= b - 1) {
                const int k = __ffs(b) - 1;
                const float e = mine_w[r * kRowW + k];
                const float4 v = *reinterpret_cast<const float4*>(piece(k) + r * P::ld + d);
                o.x = fmaf(e, v.x, o.x); o.y = fmaf(e, v.y, o.y);
                o.z = fmaf(e, v.z, o.z); o.w = fmaf(e, v.w, o.w);
            }
            const float m = mine_w[r * kRowW + kPieces], l = mine_w[r * kRowW + kPieces + 1];
            if (here) {
                const int row = p.tile * NR + r;
                if (row < q.n * a.group) {
                    const float inv = l == 0.f ? 0.f : vs / l;
                    write_out4<D>(a, q, p.h, row, d, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
                    if (d == 0) write_lse(a, q, p.h, row, m, l);
                }
            } else {
                __stcg(reinterpret_cast<float4*>(part + r * D + d), o);
                if (d == 0) {
                    __stcg(part + NR * D + r, m);
                    __stcg(part + NR * D + NR + r, l);
                }
            }
        }
        __syncwarp();                        // the next tile's weights take the same memory
        if (here) continue;
        // the CTAs that hold pieces of this tile: the first in its slot 1, the others in their slots 0
        const CtaRange ctas = tile_ctas(even, bid, per_item, share, u0, p.item, p.units);
        if (g_tid == 0) {
            s_b0[my_slot] = ctas.first;
            s_n[my_slot] = ctas.last - ctas.first + 1;
            s_piece[my_slot] = p;
        }
    }
    __syncthreads();
    if (lane == 0 && warp < 2 && s_n[warp] > 0) {
        const bool last = atom_add_acq_rel_gpu(a.counters + s_b0[warp], 1) == s_n[warp] - 1;
        s_last[warp] = last;
        if (last) a.counters[s_b0[warp]] = 0;
    }
    __syncthreads();
    // Tiles whose last piece was this CTA's: at most the one that came in and the one that goes on.
    float* sums = reinterpret_cast<float*>(smem);                                           // [NR]; the rings are free
    for (int which = 0; which < 2; ++which) {
        if (!s_last[which]) continue;
        const PieceInfo p = s_piece[which];
        const int b0 = s_b0[which], n = s_n[which], pad = (n + kAhead - 1) / kAhead * kAhead;
        const float* base = a.partial + static_cast<long long>(b0) * 2 * (NR * (D + 2));
        auto slot = [&](int k) { return base + (2 * k + (k == 0 ? 1 : 0)) * (NR * (D + 2)); };
        // the first pieces' numbers are on their way while the weights are found
        float4 v[kAhead];
        auto load = [&](int x, int k0) {
            const int at = x / (D / 4) * D + x % (D / 4) * 4;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) v[k] = __ldcg(reinterpret_cast<const float4*>(slot(min(k0 + k, n - 1)) + at));
        };
        if (threadIdx.x < NR * (D / 4)) load(threadIdx.x, 0);
        // a warp for each row: the pieces' weights 2^(m - max) and the sum of their l
        for (int r = warp; r < NR; r += kWarps) {
            float m = -INFINITY, l = 0.f;
            float mk[kMaxCtas / 32], lk[kMaxCtas / 32];
#pragma unroll
            for (int i = 0; i < kMaxCtas / 32; ++i) {
                const int k = 32 * i + lane;
                mk[i] = k < n ? __ldcg(slot(k) + NR * D + r) : -INFINITY;
                lk[i] = k < n ? __ldcg(slot(k) + NR * D + NR + r) : 0.f;
                m = fmaxf(m, mk[i]);
            }
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, off));
#pragma unroll
            for (int i = 0; i < kMaxCtas / 32; ++i) {
                const int k = 32 * i + lane;
                // a piece that has seen nothing counts for nothing; a NaN sum stays
                const float e = mk[i] == -INFINITY ? (lk[i] == lk[i] ? 0.f : 1.f) : ex2(mk[i] - m);
                l = fmaf(e, lk[i], l);
                if (k < pad) weight[r * kMaxCtas + k] = e;
            }
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) l += __shfl_xor_sync(kFull, l, off);
            if (lane == 0) {
                sums[r] = l;
                const int row = p.tile * NR + r;
                if (row < p.q.n * a.group) write_lse(a, p.q, p.h, row, m, l);
            }
        }
        __syncthreads();
        for (int x = threadIdx.x; x < NR * (D / 4); x += kThreads) {
            const int r = x / (D / 4), d = x % (D / 4) * 4;
            const int row = p.tile * NR + r;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int k0 = 0; k0 < n; k0 += kAhead) {
                if (k0 > 0 || x >= kThreads) load(x, k0);
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const float e = weight[r * kMaxCtas + k0 + k];
                    o.x = fmaf(e, v[k].x, o.x); o.y = fmaf(e, v[k].y, o.y);
                    o.z = fmaf(e, v[k].z, o.z); o.w = fmaf(e, v[k].w, o.w);
                }
            }
            if (row >= p.q.n * a.group) continue;
            const float l = sums[r], inv = l == 0.f ? 0.f : p.v_scale / l;
            write_out4<D>(a, p.q, p.h, row, d, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
        }
        __syncthreads();                     // the next tile's weights take the same memory
    }
}

static_assert(kMaxCtas * 4 <= kStreamCounterBytes && kCounterBytes % 256 == 0, "places of the counters");

template <int D, int NT>
cudaError_t launch_stream(const AttnArgs& a, cudaStream_t s) {
    constexpr int smem = kWarps * kStages * Kv4Layout<D>::bytes + kWarps * Piece<D, 8 * NT>::floats * 4 + kMaxCtas * 8 * NT * 4;
    static_assert(smem <= 226 * 1024, "shared memory of a CTA");
    auto* k = attn_kv4_stream_kernel<D, NT>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(k, dim3(min(sm_count(), kMaxCtas)), dim3(kThreads), smem, s, a);
}

}  // namespace

// Rows of a sequence that the streaming kernel takes, for `rows` of all sequences; more go to the prompt
// kernel.  Streaming costs a pass over the pages for each 16 rows, the prompt kernel a start of some 30 us.
// us of the two (streaming/prompt), 8 query heads a key head, 4 key heads, contexts of 300, 2000, 9000:
//     128 rows,  1 sequence  13/34 17/33 27/77     8: 22/36 25/35 43/79    32: 23/37 40/40 96/54
//     256 rows,  1 sequence  15/38 25/36 41/57     8: 24/36 29/37 71/58    32: 32/38 63/39 187/58
constexpr int stream_rows(long long rows) { return rows <= 1024 ? 256 : 128; }

constexpr size_t stream_workspace(int D) {
    return kCounterBytes + static_cast<size_t>(kMaxCtas) * 2 * 16 * (D + 2) * sizeof(float);
}

size_t attention_kv4_workspace(int T, int n_q, int n_kv, int D) {
    const long long rows = static_cast<long long>(T) * (n_q / n_kv);
    const bool prefill = rows > stream_rows(rows);
    return (stream_workspace(D) + 255) / 256 * 256 + (prefill ? attn_prefill_pieces(D) : 0);
}

cudaError_t launch_attention_kv4(const void* q, long long ld_q, int T, int n_q, const moe_kv4_cache& c,
                                 const int32_t* q_start, int max_new, float scale, int window, void* out,
                                 long long ld_out, float* lse, void* ws, moe_dev_status* st, cudaStream_t s) {
    AttnArgs a = {};
    a.q = static_cast<const __nv_bfloat16*>(q); a.ld_q = ld_q; a.T = T; a.n_q = n_q; a.group = n_q / c.n_kv;
    a.c = c; a.q_start = q_start; a.scale = scale; a.window = window;
    a.out = static_cast<__nv_bfloat16*>(out); a.ld_out = ld_out; a.lse = lse;
    a.counters = static_cast<int*>(ws);
    a.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kCounterBytes);
    a.st = st;
    a.rows_lo = 1;
    a.rows_hi = 0x7fffffff;
    // Without a sequence of many rows (as max_new promises) the streaming kernel is launched alone;
    // sequences that have more all the same are right there, only slower.
    const long long rows = static_cast<long long>(T) * a.group;
    const int few = stream_rows(rows);
    const bool prefill = static_cast<long long>(max_new) * a.group > few && rows > few;
    if (prefill) {
        a.rows_hi = few;
        AttnArgs b = a;
        b.rows_lo = few + 1;
        b.rows_hi = 0x7fffffff;
        b.counters = reinterpret_cast<int*>(static_cast<uint8_t*>(ws) + kStreamCounterBytes);
        b.partial = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + (stream_workspace(c.head_dim) + 255) / 256 * 256);
        cudaError_t e = launch_attn_prefill(b, s);
        if (e != cudaSuccess) return e;
    }
    const bool one = static_cast<long long>(max_new) * a.group <= 8;
    if (c.head_dim == 128) return one ? launch_stream<128, 1>(a, s) : launch_stream<128, 2>(a, s);
    return one ? launch_stream<64, 1>(a, s) : launch_stream<64, 2>(a, s);
}

}  // namespace moe
