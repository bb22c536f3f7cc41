// attn_kv4_prefill.cu -- attention over the 4-bit paged cache for many query
// rows a sequence (prompt chunks): tcgen05 products bound by the tensor cores.
//
// For one (sequence, key head) the rows are the new tokens' query heads of
// that key head, token-major; a work item is 256 of them, in two tiles of 128
// (TMEM lanes) that share every page of keys and values:
//     S = Q K^T (128 x 64, fp32 in TMEM),  P = 2^(f S - m) (fp16, over S),
//     O += P V (128 x D, fp32 in TMEM)
// Q and P are the products' A operands in TMEM, so shared memory feeds only
// the 64-token operands and the conversion that writes them: with Q there
// too its reads alone would take the products' time.  TMEM of a tile: S/P 64
// columns, Q D/2, O D; two tiles fill the 512 columns.
//
// Warps: 0-3 and 4-7 the softmax of tile 0 and 1 (a thread is a row), 8-11
// convert 4-bit pages to fp16 operands (exact), 12 issues the products, 13
// copies pages (one bulk copy each).  While one tile's softmax runs, the
// other tile's products do.  O is scaled only when a row's maximum grows by
// more than 2^8, which fp16's range allows for P.
//
// The pages of all items form one sequence of units, cut into equal runs for
// the CTAs; an item that crosses CTAs is joined by the last to arrive,
// in the order of the pages.
#include <cuda_bf16.h>
#include <type_traits>

#include "attn_kv4.cuh"
#include "common.cuh"
#include "kv4.cuh"
#include "launch.h"
#include "tmap.h"

namespace moe {

namespace {

constexpr int kRows = 256;          // of an item
constexpr int kTile = 128;
constexpr int kPfThreads = 14 * 32;
constexpr int kPfWarps = kPfThreads / 32;
constexpr int kRaw = 3;             // pages in 4 bits in flight
constexpr int kBuf = 2;             // pages as fp16 operands
constexpr int kMaxCtasPf = 160;
constexpr int kCounterBytesPf = 2048;
constexpr int kChunk = 1024;        // sequences whose units are held in shared memory
constexpr float kGrow = 8.f;        // log2 of the growth that O waits for

enum Site : int { kSiteRaw = 31, kSiteRawFree, kSiteKFree, kSiteVFree, kSiteKFull, kSiteVFull, kSiteQ, kSiteP, kSiteS, kSiteO };

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
          "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
          "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// D[tmem] (+)= A[tmem] * B[smem]^T, kind::f16 (fp16 inputs, fp32 accumulate).
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// One lane of the converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}
// fp16 A and B, fp32 D, both K-major: as idesc_bf16_f32 with the operand formats 0.
__host__ __device__ constexpr uint32_t idesc_f16_f32(int M, int N) {
    return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

template <int D>
struct Pf {
    static constexpr int raw = Kv4Layout<D>::bytes;
    static constexpr int k_tile = kPage * D * 2;      // D/64 halves of [64 tokens][64 numbers], 128-byte rows
    static constexpr int v_tile = kPage * D * 2;      // [D numbers][64 tokens], 128-byte rows
    static constexpr int o_k = 0;
    static constexpr int o_v = o_k + kBuf * k_tile;
    static constexpr int o_raw = o_v + kBuf * v_tile;
    static constexpr int smem = o_raw + kRaw * raw + 1024;   // slack for 1024-byte alignment
    // TMEM columns of a tile; all 512 are taken, so the first is column 0
    static constexpr int c_s = 0, c_q = 64, c_o = 128, tile_cols = 256;
};

// Where a run starts.
struct Start {
    int s, h, tile, skip;
    long long item_begin;
};

// The units of a run, item by item: the same walk in every role.
struct Walk {
    int s, h, tile, tiles;
    long long unit;
    Seq q;
    int lo, hi;        // pages of the item
    int pa, pb;        // those of this run's piece
    __device__ void begin(const AttnArgs& a, const Start& st, long long u0, long long u1) {
        s = st.s; h = st.h; tile = st.tile;
        q = load_seq(a, s);
        tiles = seq_tiles<kRows>(a, q);
        unit = u0;
        tile_pages<kRows>(a, q, tile, lo, hi);
        pa = lo + st.skip;
        pb = static_cast<int>(min(static_cast<long long>(hi), pa + (u1 - unit)));
    }
    __device__ void next(const AttnArgs& a, long long u1) {
        unit += max(1, pb - pa);
        if (unit >= u1) return;
        if (++tile >= tiles) {
            tile = 0;
            if (++h >= a.c.n_kv) {
                h = 0;
                do {
                    ++s;
                    q = load_seq(a, s);
                    tiles = seq_tiles<kRows>(a, q);
                } while (tiles == 0);      // a later sequence has rows: unit < u1 <= total
            }
        }
        tile_pages<kRows>(a, q, tile, lo, hi);
        pa = lo;
        pb = static_cast<int>(min(static_cast<long long>(hi), pa + (u1 - unit)));
    }
    // pages of half t (128 rows) within the piece
    __device__ void half(const AttnArgs& a, int t, int& x, int& y) const {
        const int r0 = tile * kRows + t * kTile;
        if (r0 >= q.n * a.group) { x = y = pa; return; }
        int l, e;
        tile_pages<kTile>(a, q, 2 * tile + t, l, e);
        x = max(pa, l);
        y = max(x, min(pb, e));
    }
};

template <int D>
__global__ void __launch_bounds__(kPfThreads, 1) attn_kv4_prefill_kernel(const AttnArgs a) {
    using L = Kv4Layout<D>;
    using C = Pf<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    enum { B_RAWF = 0, B_RAWE = B_RAWF + kRaw, B_KF = B_RAWE + kRaw, B_KE = B_KF + kBuf, B_VF = B_KE + kBuf, B_VE = B_VF + kBuf,
           B_Q = B_VE + kBuf, B_S = B_Q + 2, B_P = B_S + 2, B_O = B_P + 2, B_DRAIN = B_O + 2, B_N };
    __shared__ __align__(8) uint64_t bars[B_N];
    __shared__ uint32_t s_tmem;
    __shared__ long long s_units[kChunk], s_warp[kPfWarps];
    __shared__ int s_list[kChunk], s_list_n, s_ticket;
    __shared__ Start s_start;
    __shared__ uint8_t s_bad[kRaw];
    __shared__ volatile int s_abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto bar = [&](int i) { return smem_u32(&bars[i]); };

    if (threadIdx.x == 0) {
        for (int i = 0; i < kRaw; ++i) { mbar_init(bar(B_RAWF + i), 1); mbar_init(bar(B_RAWE + i), 4); }
        for (int i = 0; i < kBuf; ++i) {
            mbar_init(bar(B_KF + i), 4); mbar_init(bar(B_KE + i), 1);
            mbar_init(bar(B_VF + i), 4); mbar_init(bar(B_VE + i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(B_Q + i), 4); mbar_init(bar(B_S + i), 1);
            mbar_init(bar(B_P + i), 4); mbar_init(bar(B_O + i), 1);
        }
        mbar_init(bar(B_DRAIN), 1);
        s_abort = 0;
        fence_mbar_init();
    }
    pdl_wait();
    pdl_trigger();

    // ---- the units of all sequences, added up by every CTA for itself ----
    // s_units of a chunk of sequences; long ones take a whole warp each
    auto fill_units = [&](int c0) {
        const int n = min(kChunk, a.c.S - c0);
        if (threadIdx.x == 0) s_list_n = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < n; i += kPfThreads) {
            const Seq q = load_seq(a, c0 + i);
            if (seq_tiles<kRows>(a, q) <= 4) s_units[i] = seq_units<kRows>(a, q) * a.c.n_kv;
            else s_list[atomicAdd(&s_list_n, 1)] = i;
        }
        __syncthreads();
        for (int k = warp; k < s_list_n; k += kPfWarps) {
            const int i = s_list[k];
            const Seq q = load_seq(a, c0 + i);
            const int tiles = seq_tiles<kRows>(a, q);
            long long u = 0;
            for (int x = lane; x < tiles; x += 32) {
                int lo, hi;
                tile_pages<kRows>(a, q, x, lo, hi);
                u += max(1, hi - lo);
            }
#pragma unroll
            for (int off = 16; off >= 1; off >>= 1) u += __shfl_xor_sync(kFull, u, off);
            if (lane == 0) s_units[i] = u * a.c.n_kv;
        }
        __syncthreads();
        return n;
    };
    long long total = 0;
    for (int c0 = 0; c0 < a.c.S; c0 += kChunk) {
        const int n = fill_units(c0);
        long long mine = 0;
        for (int i = threadIdx.x; i < n; i += kPfThreads) mine += s_units[i];
#pragma unroll
        for (int off = 16; off >= 1; off >>= 1) mine += __shfl_xor_sync(kFull, mine, off);
        if (lane == 0) s_warp[warp] = mine;
        __syncthreads();
        for (int i = 0; i < kPfWarps; ++i) total += s_warp[i];
        __syncthreads();
    }
    const long long share = max(4ll, (total + gridDim.x - 1) / gridDim.x);
    const long long u0 = min(total, share * blockIdx.x), u1 = min(total, u0 + share);
    if (u0 >= u1) return;
    // warp 0 finds the sequence, head, tile and page of unit u0
    {
        long long before = 0;
        for (int c0 = 0; c0 < a.c.S; c0 += kChunk) {
            const int n = a.c.S > kChunk ? fill_units(c0) : a.c.S;
            if (warp == 0) {
                for (int i0 = 0; i0 < n; i0 += 32) {
                    const long long v = i0 + lane < n ? s_units[i0 + lane] : 0;
                    long long inc = v;
#pragma unroll
                    for (int off = 1; off < 32; off <<= 1) {
                        const long long o = __shfl_up_sync(kFull, inc, off);
                        if (lane >= off) inc += o;
                    }
                    const long long b = before + inc - v;
                    const unsigned hit = __ballot_sync(kFull, v > 0 && u0 >= b && u0 < b + v);
                    if (hit != 0) {
                        const int src = __ffs(hit) - 1;
                        const long long sb = __shfl_sync(kFull, b, src), sv = __shfl_sync(kFull, v, src);
                        const int s = c0 + i0 + src;
                        const Seq q = load_seq(a, s);
                        const int tiles = seq_tiles<kRows>(a, q);
                        const long long per_head = sv / a.c.n_kv;
                        const int h = static_cast<int>((u0 - sb) / per_head);
                        long long at = sb + h * per_head;
                        for (int x0 = 0; x0 < tiles; x0 += 32) {
                            long long w = 0;
                            if (x0 + lane < tiles) {
                                int lo, hi;
                                tile_pages<kRows>(a, q, x0 + lane, lo, hi);
                                w = max(1, hi - lo);
                            }
                            long long wi = w;
#pragma unroll
                            for (int off = 1; off < 32; off <<= 1) {
                                const long long o = __shfl_up_sync(kFull, wi, off);
                                if (lane >= off) wi += o;
                            }
                            const long long tb = at + wi - w;
                            if (w > 0 && u0 >= tb && u0 < tb + w) s_start = {s, h, x0 + lane, static_cast<int>(u0 - tb), tb};
                            at += __shfl_sync(kFull, wi, 31);
                        }
                    }
                    before += __shfl_sync(kFull, inc, 31);
                }
            }
            __syncthreads();
        }
    }
    if (warp == 12) {
        tmem_alloc(smem_u32(&s_tmem), 512);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    const Start start = s_start;

    bool ok = true;
    if (warp == 13) {
        // ---------------- pages from device memory ----------------
        Walk w;
        w.begin(a, start, u0, u1);
        int st = 0;
        uint32_t ph = 1;             // the stages start out free
        for (; ok;) {
            for (int p0 = w.pa; p0 < w.pb && ok; p0 += 32) {
                // the table's entries of 32 pages at once
                const int mine = p0 + lane < w.pb ? a.c.page_table[static_cast<long long>(w.s) * a.c.max_pages + p0 + lane] : 0;
                const int n = min(32, w.pb - p0);
                for (int i = 0; i < n; ++i) {
                    const int id = __shfl_sync(kFull, mine, i);
                    ok = mbar_wait(bar(B_RAWE + st), ph, &s_abort, a.st, kSiteRawFree);
                    ok = __all_sync(kFull, ok);
                    if (!ok) break;
                    if (lane == 0) {
                        const bool good = id >= 0 && id < a.c.n_pages;
                        s_bad[st] = !good;
                        if (good) {
                            mbar_arrive_expect_tx(bar(B_RAWF + st), L::bytes);
                            bulk_copy_g2s(smem_u32(smem + C::o_raw + st * C::raw),
                                          static_cast<const uint8_t*>(a.c.pages) + (static_cast<long long>(id) * a.c.n_kv + w.h) * L::bytes,
                                          L::bytes, bar(B_RAWF + st));
                        } else {
                            report(a.st, MOE_DEV_BAD_INDEX, id);
                            mbar_arrive(bar(B_RAWF + st));
                        }
                    }
                    __syncwarp();
                    if (++st == kRaw) { st = 0; ph ^= 1; }
                }
            }
            if (!ok) break;
            w.next(a, u1);
            if (w.unit >= u1) break;
        }
        // copies in flight land before the CTA gives its shared memory up: on
        // success the converters have waited for all of them
        if (!ok) {
            for (int i = 0; i < kRaw; ++i) {
                mbar_drain(bar(B_RAWF + i), 0);
                mbar_drain(bar(B_RAWF + i), 1);
            }
        }
    } else if (warp == 12) {
        // ---------------- products ----------------
        // The warp walks together and one elected lane issues: addresses and
        // descriptors then stay in uniform registers.
        constexpr uint32_t id_s = idesc_f16_f32(kTile, kPage), id_o = idesc_f16_f32(kTile, D);
        const uint64_t k_desc = sw128_desc(smem_u32(smem + C::o_k)), v_desc = sw128_desc(smem_u32(smem + C::o_v));
        Walk w;
        w.begin(a, start, u0, u1);
        uint32_t kb = 0, kp = 0, vb = 0, vp = 0;     // buffer and parity of the next keys and values
        uint32_t pp0 = 0, pp1 = 0, qp0 = 0, qp1 = 0;
        auto wait = [&](int i, uint32_t parity, int site) {
            ok = mbar_wait(bar(i), parity, &s_abort, a.st, site);
            ok = __all_sync(kFull, ok);
            return ok;
        };
        auto issue_s = [&](auto tc) {
            constexpr uint32_t t = decltype(tc)::value;
            const uint64_t d = k_desc + kb * (C::k_tile >> 4);
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k)
                    tc_mma_ts(t * C::tile_cols + C::c_s, t * C::tile_cols + C::c_q + 8 * k, d + (k / 4) * (kPage * 128 >> 4) + (k % 4) * 2, id_s, k > 0);
                tc_commit(bar(B_S + t));
            }
            __syncwarp();
        };
        auto issue_o = [&](auto tc, bool add, bool last) {
            constexpr uint32_t t = decltype(tc)::value;
            const uint64_t d = v_desc + vb * (C::v_tile >> 4);
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    tc_mma_ts(t * C::tile_cols + C::c_o, t * C::tile_cols + C::c_s + 8 * k, d + 2 * k, id_o, add || k > 0);
                if (last) tc_commit(bar(B_O + t));
            }
            __syncwarp();
        };
        constexpr std::integral_constant<uint32_t, 0> T0{};
        constexpr std::integral_constant<uint32_t, 1> T1{};
        while (ok) {
            int x0, y0, x1, y1;
            w.half(a, 0, x0, y0);
            w.half(a, 1, x1, y1);
            if (w.pa < w.pb) {
                if (!wait(B_KF + kb, kp, kSiteKFull)) break;
                if (x0 < y0) { if (!wait(B_Q, qp0, kSiteQ)) break; qp0 ^= 1; tc_fence_after(); if (x0 == w.pa) issue_s(T0); }
                if (x1 < y1) { if (!wait(B_Q + 1, qp1, kSiteQ)) break; qp1 ^= 1; tc_fence_after(); if (x1 == w.pa) issue_s(T1); }
                if (elect_one()) tc_commit(bar(B_KE + kb));
                __syncwarp();
                kb ^= 1; kp ^= kb == 0;
                for (int j = w.pa; j < w.pb; ++j) {
                    const bool more = j + 1 < w.pb;
                    if (!wait(B_VF + vb, vp, kSiteVFull)) break;
                    if (x0 <= j && j < y0) {
                        if (!wait(B_P, pp0, kSiteP)) break;
                        pp0 ^= 1;
                        tc_fence_after();
                        issue_o(T0, j > x0, j + 1 == y0);
                    }
                    if (more) {
                        if (!wait(B_KF + kb, kp, kSiteKFull)) break;
                        tc_fence_after();
                        if (x0 <= j + 1 && j + 1 < y0) issue_s(T0);
                    }
                    if (x1 <= j && j < y1) {
                        if (!wait(B_P + 1, pp1, kSiteP)) break;
                        pp1 ^= 1;
                        tc_fence_after();
                        issue_o(T1, j > x1, j + 1 == y1);
                    }
                    if (elect_one()) tc_commit(bar(B_VE + vb));
                    __syncwarp();
                    vb ^= 1; vp ^= vb == 0;
                    if (more) {
                        if (x1 <= j + 1 && j + 1 < y1) issue_s(T1);
                        if (elect_one()) tc_commit(bar(B_KE + kb));
                        __syncwarp();
                        kb ^= 1; kp ^= kb == 0;
                    }
                }
                if (!ok) break;
            }
            w.next(a, u1);
            if (w.unit >= u1) break;
        }
        // every product is done before TMEM and shared memory are given up
        if (elect_one()) tc_commit(bar(B_DRAIN));
        __syncwarp();
        mbar_drain(bar(B_DRAIN), 0);
    } else if (warp >= 8) {
        // ---------------- 4 bits to fp16 operands ----------------
        const int cw = warp - 8;
        Walk w;
        w.begin(a, start, u0, u1);
        uint32_t n = 0, st = 0, ph = 0;
        const int i8 = lane >> 2, t = lane & 3;
        uint32_t v_off[8];           // byte of (row k of an 8-row group, 8-token chunk i8, token pair t)
#pragma unroll
        for (int k = 0; k < 8; ++k) v_off[k] = static_cast<uint32_t>(k * 128 + ((i8 ^ k) * 16) + t * 4);
        while (ok) {
            for (int j = w.pa; j < w.pb && ok; ++j) {
                ok = mbar_wait(bar(B_RAWF + st), ph, &s_abort, a.st, kSiteRaw);
                if (ok) ok = mbar_wait(bar(B_KE + n % kBuf), ((n / kBuf) & 1) ^ 1, &s_abort, a.st, kSiteKFree);
                ok = __all_sync(kFull, ok);
                if (!ok) break;
                const uint8_t* raw = smem + C::o_raw + st * C::raw;
                const bool bad = s_bad[st];
                uint8_t* kt = smem + C::o_k + (n % kBuf) * C::k_tile;
                // keys: a thread converts runs of D/4 numbers of a token
                constexpr int W = D / 32;           // words of a run
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int x = u * 128 + cw * 32 + lane, tok = x >> 2, kt4 = x & 3;
                    uint32_t c[W], sc[L::R];
                    const uint8_t* p = raw + tok * (D / 2) + kt4 * (D / 8);
                    if constexpr (W == 4) {
                        const uint4 v = *reinterpret_cast<const uint4*>(p);
                        c[0] = v.x; c[1] = v.y; c[2] = v.z; c[3] = v.w;
                        const uint32_t two = e4m3x2_to_f16(*reinterpret_cast<const uint16_t*>(raw + L::kScales + ((kt4 * 8 + (tok & 7)) * 8 + (tok >> 3)) * 2));
                        sc[0] = __byte_perm(two, 0, 0x1010);
                        sc[1] = __byte_perm(two, 0, 0x3232);
                    } else {
                        const uint2 v = *reinterpret_cast<const uint2*>(p);
                        c[0] = v.x; c[1] = v.y;
                        sc[0] = __byte_perm(e4m3x2_to_f16(raw[L::kScales + (kt4 * 8 + (tok & 7)) * 8 + (tok >> 3)]), 0, 0x1010);
                    }
                    if (bad) {
#pragma unroll
                        for (int i = 0; i < L::R; ++i) sc[i] = 0u;
                    }
                    // numbers (D/4) kt4 + 8 i ..: half, 16-byte chunk of the row
                    const int half = D == 128 ? kt4 >> 1 : 0;
                    const int chunk0 = D == 128 ? (kt4 & 1) * 4 : kt4 * 2;
#pragma unroll
                    for (int i0 = 0; i0 < W; ++i0) {
                        // the upper half's runs go in another order, so that eight threads' chunks differ in their banks
                        const int i = D == 128 ? i0 ^ (half * 2) : i0;
                        const uint32_t cw_ = D == 128 ? (half ? c[(i0 ^ 2) % W] : c[i0]) : c[i0];
                        const uint32_t sr = D == 128 ? (i < 2 ? sc[0] : sc[L::R - 1]) : sc[0];
                        uint32_t f[4];
                        e2m1x8_to_f16(cw_, f[0], f[1], f[2], f[3]);
                        const uint4 v = make_uint4(hmul2_u(f[0], sr), hmul2_u(f[1], sr), hmul2_u(f[2], sr), hmul2_u(f[3], sr));
                        *reinterpret_cast<uint4*>(kt + half * (kPage * 128) + tok * 128 + (((chunk0 + i) ^ (tok & 7)) * 16)) = v;
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_KF + n % kBuf));
                ok = mbar_wait(bar(B_VE + n % kBuf), ((n / kBuf) & 1) ^ 1, &s_abort, a.st, kSiteVFree);
                ok = __all_sync(kFull, ok);
                if (!ok) break;
                // values: a thread converts a token pair's run of D/8 numbers, for two of the eight runs
                uint8_t* vt = smem + C::o_v + (n % kBuf) * C::v_tile;
                const int left = w.q.len - j * kPage;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int g = 2 * cw + u;
                    constexpr int WV = D / 32;      // words of a run of D/8 bytes
                    uint32_t c[WV];
                    const uint8_t* p = raw + L::vCodes + ((i8 * 8 + g) * 4 + t) * L::U;
                    if constexpr (WV == 4) {
                        const uint4 v = *reinterpret_cast<const uint4*>(p);
                        c[0] = v.x; c[1] = v.y; c[2] = v.z; c[3] = v.w;
                    } else {
                        const uint2 v = *reinterpret_cast<const uint2*>(p);
                        c[0] = v.x; c[1] = v.y;
                    }
                    uint32_t two = *reinterpret_cast<const uint16_t*>(raw + L::vScales + (((D == 128 ? g : g / 2) * 4 + t) * 8 + i8) * 2);
                    // tokens that the sequence does not have: their bytes may be anything
                    if (left < kPage) {
                        const int tok = 8 * i8 + 2 * t;
                        two = tok + 1 < left ? two : (tok < left ? (two & 0xffu) : 0u);
                    }
                    uint32_t sc = e4m3x2_to_f16(two);
                    if (bad) sc = 0u;
                    uint8_t* row = vt + g * (L::U * 128);
#pragma unroll
                    for (int i = 0; i < WV; ++i) {
                        uint32_t f[4];
                        e2m1x8_to_f16(c[i], f[0], f[1], f[2], f[3]);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            *reinterpret_cast<uint32_t*>(row + (i / 2) * 1024 + v_off[(4 * i + k) % 8]) = hmul2_u(f[k], sc);
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(B_VF + n % kBuf));
                    mbar_arrive(bar(B_RAWE + st));
                }
                ++n;
                if (++st == kRaw) { st = 0; ph ^= 1; }
            }
            if (!ok) break;
            w.next(a, u1);
            if (w.unit >= u1) break;
        }
    } else {
        // ---------------- softmax: a thread is a row ----------------
        const int t = warp >> 2;                              // tile
        const int r_tile = (warp & 3) * 32 + lane;            // row of the tile = TMEM lane
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tb = tmem + t * C::tile_cols + lanes;
        Walk w;
        w.begin(a, start, u0, u1);
        uint32_t n_s = 0, n_o = 0;
        // after a wait that ran out (ok = false) the items are walked to the end all the same, without
        // waiting: the two tiles' warps meet at barriers below
        while (true) {
            int x, y;
            w.half(a, t, x, y);
            const int r = w.tile * kRows + t * kTile + r_tile;   // row of the (sequence, head)
            const bool live = r < w.q.n * a.group;
            const int p_row = w.q.len - w.q.n + r / a.group;     // place of the row
            float m = -INFINITY, l = 0.f;                        // m in powers of two
            if (x < y && ok) {
                // queries to TMEM, scaled by a power of two of the row (see the streaming kernel)
                // (read twice, once for the row's largest magnitude: the row would take D/2 registers)
                const uint4* src = reinterpret_cast<const uint4*>(a.q + static_cast<long long>(w.q.q0 + r / a.group) * a.ld_q +
                                                                  static_cast<long long>(w.h * a.group + r % a.group) * D);
                float top = 0.f;
                if (live) {
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {
                        const uint4 v = src[i];
                        const uint32_t c[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            top = fmaxf(top, fmaxf(fabsf(__uint_as_float(c[k] << 16)), fabsf(__uint_as_float(c[k] & 0xffff0000u))));
                    }
                }
                int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
                e = (top > 0.f && e < 128) ? max(-100, min(100, 10 - e)) : 0;
                float up = __int_as_float((e + 127) << 23);
                float f = a.scale * kLog2e * (a.c.k_scale != nullptr ? a.c.k_scale[w.h] : 1.f) * __int_as_float((127 - e) << 23);
                // the maximum is taken before the factor: it has to be positive
                if (f < 0.f) { f = -f; up = -up; }
                f = fmaxf(f, 1e-37f);
#pragma unroll 1
                for (int i = 0; i < D / 64; ++i) {
                    uint32_t h[32];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint4 v = live ? src[8 * i + k] : make_uint4(0u, 0u, 0u, 0u);
                        const uint32_t c[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int z = 0; z < 4; ++z)
                            h[4 * k + z] = pack_f16(__uint_as_float(c[z] << 16) * up, __uint_as_float(c[z] & 0xffff0000u) * up);
                    }
                    tmem_st32(tb + C::c_q + 32 * i, h);
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_Q + t));

                // places of the tile's first and last row, for the pages that need no mask
                const int rt0 = w.tile * kRows + t * kTile, rt1 = min(w.q.n * a.group, rt0 + kTile) - 1;
                const int p_first = w.q.len - w.q.n + rt0 / a.group, p_last = w.q.len - w.q.n + rt1 / a.group;
                const int first_key = a.window > 0 ? p_row - a.window + 1 : 0;
                float mf = -INFINITY;                            // the maximum in use, before the factor
                for (int j = x; j < y; ++j) {
                    ok = mbar_wait(bar(B_S + t), n_s++ & 1, &s_abort, a.st, kSiteS);
                    ok = __all_sync(kFull, ok);
                    if (!ok) break;
                    tc_fence_after();
                    uint32_t s0[32], s1[32];
                    tmem_ld32(tb + C::c_s, s0);
                    tmem_ld32(tb + C::c_s + 32, s1);
                    tmem_ld_wait();
                    const int key0 = j * kPage;
                    if (key0 + kPage - 1 > p_first || (a.window > 0 && key0 <= p_last - a.window)) {
                        const int last = p_row - key0, first = first_key - key0;
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            if (k > last || k < first) s0[k] = 0xff800000u;
                            if (k + 32 > last || k + 32 < first) s1[k] = 0xff800000u;
                        }
                    }
                    float t0 = __uint_as_float(s0[0]), t1 = __uint_as_float(s1[0]);
#pragma unroll
                    for (int k = 1; k < 32; ++k) {
                        t0 = fmaxf(t0, __uint_as_float(s0[k]));
                        t1 = fmaxf(t1, __uint_as_float(s1[k]));
                    }
                    const float now = fmaxf(t0, t1);
                    // in use: the maximum so far, unless it has grown by more than 2^kGrow
                    if (__any_sync(kFull, now > mf && (mf == -INFINITY || (now - mf) * f > kGrow))) {
                        const float nm = fmaxf(mf, now);
                        const float sc = mf == -INFINITY ? 0.f : ex2((mf - nm) * f);
                        mf = nm;
                        l *= sc;
                        if (j > x) {
#pragma unroll 1
                            for (int i = 0; i < D / 32; ++i) {
                                uint32_t o[32];
                                tmem_ld32(tb + C::c_o + 32 * i, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * sc);
                                tmem_st32(tb + C::c_o + 32 * i, o);
                            }
                        }
                    }
                    const float base = mf == -INFINITY ? 0.f : -mf * f;
                    uint32_t h[32];
                    float l0 = 0.f, l1 = 0.f;
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const float e0 = ex2(fmaf(__uint_as_float(s0[2 * k]), f, base)), e1 = ex2(fmaf(__uint_as_float(s0[2 * k + 1]), f, base));
                        const float e2 = ex2(fmaf(__uint_as_float(s1[2 * k]), f, base)), e3 = ex2(fmaf(__uint_as_float(s1[2 * k + 1]), f, base));
                        l0 += e0 + e1;
                        l1 += e2 + e3;
                        h[k] = pack_f16(e0, e1);
                        h[16 + k] = pack_f16(e2, e3);
                    }
                    l += l0 + l1;
                    tmem_st32(tb + C::c_s, h);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(B_P + t));
                }
                m = mf == -INFINITY ? -INFINITY : mf * f;
                if (ok) ok = mbar_wait(bar(B_O + t), n_o++ & 1, &s_abort, a.st, kSiteO);
                ok = __all_sync(kFull, ok);
                tc_fence_after();
            }
            // ---- the piece's result ----
            const bool whole = w.pa == w.lo && w.pb == w.hi;
            const long long item = w.unit - (w.pa - w.lo);
            const int units = max(1, w.hi - w.lo);
            const float vs = a.c.v_scale != nullptr ? a.c.v_scale[w.h] : 1.f;
            float* part = nullptr;
            constexpr int kSlot = kRows * (D + 2);
            if (!whole) part = a.partial + (static_cast<long long>(blockIdx.x) * 2 + (item < u0 ? 0 : 1)) * kSlot;
            const float inv = l == 0.f ? 0.f : vs / l;
#pragma unroll 1
            for (int i = 0; i < D / 32; ++i) {
                uint32_t o[32];
                if (x < y && ok) {
                    tmem_ld32(tb + C::c_o + 32 * i, o);
                    tmem_ld_wait();
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = 0u;
                }
                if (whole) {
                    if (live) {
                        uint4* out = reinterpret_cast<uint4*>(a.out + static_cast<long long>(w.q.q0 + r / a.group) * a.ld_out +
                                                              static_cast<long long>(w.h * a.group + r % a.group) * D + 32 * i);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            uint32_t v[4];
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                // a row that has seen nothing has l = 0: its O is not a number only if the page's is
                                const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(o[8 * k + 2 * c]) * inv, __uint_as_float(o[8 * k + 2 * c + 1]) * inv);
                                memcpy(&v[c], &b, 4);
                            }
                            out[k] = make_uint4(v[0], v[1], v[2], v[3]);
                        }
                    }
                } else {
                    // columns in fours, rows side by side: a warp's stores are dense
                    float4* dst = reinterpret_cast<float4*>(part) + (static_cast<long long>(8 * i) * kRows + t * kTile + r_tile);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        __stcg(dst + k * kRows, make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]),
                                                            __uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3])));
                }
            }
            tc_fence_before();      // O and S are read: the next item's products may follow (through B_Q and B_P)
            if (whole) {
                if (live) write_lse(a, w.q, w.h, r, m, l);
            } else {
                __stcg(part + kRows * D + t * kTile + r_tile, m);
                __stcg(part + kRows * D + kRows + t * kTile + r_tile, l);
                const int b0 = static_cast<int>(item / share), b1 = static_cast<int>((item + units - 1) / share);
                asm volatile("bar.sync 2, 256;" ::: "memory");
                if (threadIdx.x == 0) {
                    __threadfence();
                    s_ticket = atom_add_acq_rel_gpu(a.counters + b0, 1);
                }
                asm volatile("bar.sync 2, 256;" ::: "memory");
                if (s_ticket == b1 - b0) {
                    __threadfence();
                    if (threadIdx.x == 0) a.counters[b0] = 0;
                    const int row = t * kTile + r_tile;
                    auto slot = [&](int b) { return a.partial + (static_cast<long long>(b) * 2 + (b == b0 ? 1 : 0)) * kSlot; };
                    float gm = -INFINITY, gl = 0.f;
                    for (int b = b0; b <= b1; ++b) gm = fmaxf(gm, __ldcg(slot(b) + kRows * D + row));
                    for (int b = b0; b <= b1; ++b) {
                        const float mk = __ldcg(slot(b) + kRows * D + row);
                        gl += mk == -INFINITY ? 0.f : ex2(mk - gm) * __ldcg(slot(b) + kRows * D + kRows + row);
                    }
                    const float ginv = gl == 0.f ? 0.f : vs / gl;
#pragma unroll 1
                    for (int i = 0; i < D / 8; ++i) {
                        float4 o0 = make_float4(0.f, 0.f, 0.f, 0.f), o1 = o0;
                        for (int b = b0; b <= b1; ++b) {
                            const float mk = __ldcg(slot(b) + kRows * D + row);
                            const float ek = mk == -INFINITY ? 0.f : ex2(mk - gm) * ginv;
                            const float4* src = reinterpret_cast<const float4*>(slot(b)) + static_cast<long long>(2 * i) * kRows + row;
                            const float4 v0 = __ldcg(src), v1 = __ldcg(src + kRows);
                            o0.x = fmaf(ek, v0.x, o0.x); o0.y = fmaf(ek, v0.y, o0.y); o0.z = fmaf(ek, v0.z, o0.z); o0.w = fmaf(ek, v0.w, o0.w);
                            o1.x = fmaf(ek, v1.x, o1.x); o1.y = fmaf(ek, v1.y, o1.y); o1.z = fmaf(ek, v1.z, o1.z); o1.w = fmaf(ek, v1.w, o1.w);
                        }
                        if (live) {
                            write_out4<D>(a, w.q, w.h, r, 8 * i, o0);
                            write_out4<D>(a, w.q, w.h, r, 8 * i + 4, o1);
                        }
                    }
                    if (live) write_lse(a, w.q, w.h, r, gm, gl);
                }
            }
            w.next(a, u1);
            if (w.unit >= u1) break;
        }
    }
    __syncthreads();
    if (warp == 12) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D>
cudaError_t launch_pf(const AttnArgs& a, cudaStream_t s) {
    auto* k = attn_kv4_prefill_kernel<D>;
    cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, Pf<D>::smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(k, dim3(min(sm_count(), kMaxCtasPf)), dim3(kPfThreads), Pf<D>::smem, s, a);
}

}  // namespace

size_t attn_prefill_workspace(int D) {
    return kCounterBytesPf + static_cast<size_t>(kMaxCtasPf) * 2 * kRows * (D + 2) * sizeof(float);
}

cudaError_t launch_attn_prefill(const AttnArgs& a, cudaStream_t s) {
    return a.c.head_dim == 128 ? launch_pf<128>(a, s) : launch_pf<64>(a, s);
}

}  // namespace moe
