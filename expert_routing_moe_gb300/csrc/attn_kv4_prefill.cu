// attn_kv4_prefill.cu -- attention over the 4-bit paged cache for many query
// rows a sequence (prompt chunks): tcgen05 products.
//
// For one (sequence, key head) the rows are the new tokens' query heads of
// that key head, token-major; a work item is 256 of them, in two tiles of 128
// (TMEM lanes) that share every page of keys and values:
//     S = Q K^T (128 x 64, fp32 in TMEM),  P = 2^(f S - m) (fp16, over S),
//     O += P V (128 x D, fp32 in TMEM; P is the A operand in TMEM)
// S has two buffers a tile: the next page's scores are computed while the
// softmax is at this one's.  TMEM of a tile: S/P 2 x 64 columns, O D.
//
// Warps: 0-3 and 4-7 the softmax of tile 0 and 1 (a thread is a row), 8-9
// convert the keys' pages and 10-11 the values' to fp16 operands (exact), 12-13
// issue the tiles' products, 14 copies pages (one bulk copy each), 15 walks the
// items and copies the next one's queries, which the softmax warps turn to fp16
// between two items.
//
// P is fp16, and sums of it are taken in fp32 before it is rounded.  O is scaled
// only when a row's maximum grows by more than 2^kGrow over the one in use, whose P
// is 2^kRoom: P reaches 2^15 of fp16's 2^16.  A probability down to 2^-20 of the
// maximum in use is off by 2^-11 of itself (an eighth of the bf16 output's half step),
// one below by 2^-31 of that maximum: 100,000 of them by 2^-14, a million by 2^-11.
//
// The pages of all items form one sequence of units, cut into equal runs for
// the CTAs.  An item of few pages goes whole to one of them; a longer one that
// crosses CTAs is joined by the last to arrive, in the order of the pages.
//
// What bounds it: a page of an item (256 rows x 64 keys, D = 128) takes about
// 1650 clocks.  The products alone are 1280 (scores with both operands in shared
// memory run at two thirds of the tensor cores' rate, 384 clocks a tile: operands of
// 48 KB at 128 bytes a clock), the softmax warps' chain (load 300, exponentials
// 700 with the other tile's warp on the same scheduler, store 135) about 1200,
// and the two meet once a page; an item costs another 11,000 clocks (queries
// 4000, outputs 5500).  A prompt of 8192 tokens, 32 heads on 4 (550 GFLOP):
// 441-449 us from card to card, 1225-1247 TFLOP/s.
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
constexpr int kPfThreads = 16 * 32;
constexpr int kPfWarps = kPfThreads / 32;
constexpr int kRaw = 3;             // pages in 4 bits in flight
constexpr int kBuf = 2;             // pages as fp16 operands
constexpr int kChunk = 256;         // sequences whose units are held in shared memory
// log2 of the P of the maximum in use, and of the growth that O waits for: 15 in all.  Room keeps small probabilities, growth saves
// scalings of O: (0, 14), (5, 10), (6, 9), (7, 8), (10, 5), (12, 3) took 443, 444, 449, 455, 493, 542 us for a prompt of 8192 tokens
// and 102, 102, 103, 104, 113, 125 us for chunks behind long contexts.  With no room, 100,000 keys at 2^-25 of the first
// lost the 0.3% of the output that was theirs.
constexpr float kRoom = 6.f;
constexpr float kGrow = 9.f;
static_assert(kRoom + kGrow <= 15.f, "P fits fp16");
// What an item costs beside its pages (its queries, its outputs, the pipeline's
// start and end), in pages: the runs are cut by cost, so that a CTA with many
// short items gets fewer pages.  Costs of 2, 4, 6, 8, 10 took 553, 491, 452, 441, 445 us
// for a prompt of 8192 tokens and 143, 116, 103, 100, 102 us for chunks behind long contexts.
constexpr int kItemCost = 8;
// Pages of an item that is not cut: joining its pieces costs more (5 us; 64 new tokens behind 236 took 32 us
// with every item cut where a run ends, 20 with limits of 8 to 32).
constexpr int kUncut = 16;

enum Site : int { kSiteRaw = 31, kSiteRawFree, kSiteKFree, kSiteVFree, kSiteKFull, kSiteVFull, kSiteQ, kSiteP, kSiteS, kSiteO, kSiteQFree };

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
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// The largest of three.
__device__ __forceinline__ float max3(float x, float y, float z) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}

// Four 8 x 8 matrices of 16-bit numbers to shared memory; lane 8 m + r gives the address of row r of matrix m.
__device__ __forceinline__ void stmatrix4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d)
                 : "memory");
}
// The larger magnitudes of two packed bf16 pairs (a NaN gives way to a number:
// the row's products are NaN whatever its power of two is).
__device__ __forceinline__ uint32_t bf2_max_abs(uint32_t x, uint32_t y) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x & 0x7fff7fffu), "r"(y & 0x7fff7fffu));
    return r;
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
    // queries: groups of 8 rows, in each D/64 halves of [8 rows][64 numbers], 128-byte rows; a group takes
    // the bytes that its rows have in device memory, so that they are turned to fp16 in place
    static constexpr int q_group = 8 * D * 2;
    static constexpr int q_tile = kTile * D * 2;
    static constexpr int q_slot = 2 * q_tile;         // an item's
    static constexpr int o_q = 0;                     // two items: the one at hand and the next
    static constexpr int o_k = o_q + 2 * q_slot;
    static constexpr int o_v = o_k + kBuf * k_tile;
    static constexpr int o_raw = o_v + kBuf * v_tile;
    static constexpr int smem = o_raw + kRaw * raw + 1024;   // slack for 1024-byte alignment
    // TMEM columns of a tile (S: two buffers); all 512 are taken, so the first is column 0
    static constexpr int c_s = 0, c_o = 128, tile_cols = 256;
};

// Units of an item: its own cost, then one for each page.
template <int NR>
__device__ __forceinline__ int item_units(const AttnArgs& a, const Seq& s, int tile) {
    int lo, hi;
    tile_pages<NR>(a, s, tile, lo, hi);
    return kItemCost + hi - lo;
}

// What the warps of an item's products and softmax get to know of it.
struct Item {
    int q0, n, len;      // the sequence
    int h, tile;
    int pa, pb;          // pages of this run's piece
    int x[2], y[2];      // of each tile
    int b0, b1;          // runs with pages of the item
    int kind;            // kPart, kWhole or kEnd
};
enum Kind : int { kPart, kWhole, kEnd };

// The queries of 8-row groups g0 .. g1 - 1 (an even number) from bf16 rows to fp16 operands, in place, by
// one warp: four lanes hold a row, scaled by a power of two of its own (see the streaming kernel).
template <int D>
__device__ __forceinline__ void convert_queries(uint8_t* q, float* fs, int g0, int g1, int rows, float f_all, int lane) {
    constexpr int Z = D / 32;                          // 16-byte chunks of a lane
    const int rr = lane >> 2, q4 = lane & 3;
#pragma unroll 1
    for (int g = g0; g < g1; g += 2) {
        uint4 v[2][Z];
        float up[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int rt = 8 * (g + u) + rr;
            uint32_t top2 = 0u;                        // the largest magnitudes, as two bf16
#pragma unroll
            for (int z = 0; z < Z; ++z) {
                // neighbouring rows take their chunks in another order: no two lanes of a load share a bank
                const int c = (z ^ (rr & 1)) * 4 + q4;
                v[u][z] = rt < rows ? *reinterpret_cast<const uint4*>(q + rt * (D * 2) + c * 16) : make_uint4(0u, 0u, 0u, 0u);
                top2 = bf2_max_abs(top2, bf2_max_abs(bf2_max_abs(v[u][z].x, v[u][z].y), bf2_max_abs(v[u][z].z, v[u][z].w)));
            }
            float top = fmaxf(__uint_as_float(top2 << 16), __uint_as_float(top2 & 0xffff0000u));
            top = fmaxf(top, __shfl_xor_sync(kFull, top, 1));
            top = fmaxf(top, __shfl_xor_sync(kFull, top, 2));
            int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
            e = (top > 0.f && e < 128) ? max(-100, min(100, 10 - e)) : 0;
            up[u] = __int_as_float((e + 127) << 23);
            float fr = f_all * __int_as_float((127 - e) << 23);
            // the maximum is taken before the factor: it has to be positive
            if (fr < 0.f) { fr = -fr; up[u] = -up[u]; }
            if (q4 == 0) fs[rt] = fmaxf(fr, 1e-37f);
        }
        __syncwarp();                                  // the rows are read
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int z = 0; z < Z; ++z) {
                const int c = (z ^ (rr & 1)) * 4 + q4;
                const uint32_t in[4] = {v[u][z].x, v[u][z].y, v[u][z].z, v[u][z].w};
                uint32_t h[4];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    h[k] = pack_f16(__uint_as_float(in[k] << 16) * up[u], __uint_as_float(in[k] & 0xffff0000u) * up[u]);
                *reinterpret_cast<uint4*>(q + (g + u) * (8 * D * 2) + (c / 8) * 1024 + rr * 128 + (((c % 8) ^ rr) * 16)) =
                    make_uint4(h[0], h[1], h[2], h[3]);
            }
    }
    fence_proxy_async_smem();
    __syncwarp();
}

// Where a run starts.
struct Start {
    int s, h, tile, skip;
};

// The units of a run, item by item: the same walk in every role.
struct Walk {
    int s, h, tile, tiles;
    long long item;    // first unit of the item
    Seq q;
    int lo, hi;        // pages of the item
    int pa, pb;        // those of this run's piece
    bool end, own;     // own: an item that is not cut is this run's
    // A run's piece of the item: a page belongs to the run that holds its unit, and an item of few pages or
    // none to the run that holds its middle unit.
    __device__ void piece(const AttnArgs& a, long long u0, long long u1) {
        tile_pages<kRows>(a, q, tile, lo, hi);
        own = false;
        if (hi - lo <= kUncut) {
            const long long mid = item + (kItemCost + hi - lo) / 2;
            own = mid >= u0 && mid < u1;
            pa = lo;
            pb = own ? hi : lo;
            return;
        }
        const long long first = item + kItemCost;
        pa = static_cast<int>(min(static_cast<long long>(hi), lo + max(0ll, u0 - first)));
        pb = static_cast<int>(min(static_cast<long long>(hi), lo + max(0ll, u1 - first)));
    }
    __device__ void begin(const AttnArgs& a, const Start& st, long long u0, long long u1) {
        s = st.s; h = st.h; tile = st.tile;
        q = load_seq(a, s);
        tiles = seq_tiles<kRows>(a, q);
        item = u0 - st.skip;
        end = false;
        piece(a, u0, u1);
    }
    __device__ void next(const AttnArgs& a, long long u0, long long u1) {
        item += kItemCost + hi - lo;
        if (item >= u1) { end = true; return; }
        if (++tile >= tiles) {
            tile = 0;
            if (++h >= a.c.n_kv) {
                h = 0;
                do {
                    ++s;
                    q = load_seq(a, s);
                    tiles = seq_tiles<kRows>(a, q);
                } while (tiles == 0);      // a later sequence has rows: item < u1 <= total
            }
        }
        piece(a, u0, u1);
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
           B_QF = B_VE + kBuf, B_QE = B_QF + 2, B_QRF = B_QE + 2, B_S = B_QRF + 2, B_P = B_S + 4, B_O = B_P + 4, B_DRAIN = B_O + 4, B_N = B_DRAIN + 2 };
    __shared__ __align__(8) uint64_t bars[B_N];
    __shared__ uint32_t s_tmem;
    __shared__ long long s_units[kChunk], s_warp[kPfWarps];
    __shared__ int s_list[kChunk], s_list_n;
    __shared__ Start s_start;
    __shared__ uint8_t s_bad[kRaw];
    __shared__ float s_f[2][kRows];      // the rows' factors, of the item at hand and the next
    __shared__ Item s_item[2];
    __shared__ volatile int s_abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto bar = [&](int i) { return smem_u32(&bars[i]); };

    if (threadIdx.x == 0) {
        for (int i = 0; i < kRaw; ++i) { mbar_init(bar(B_RAWF + i), 1); mbar_init(bar(B_RAWE + i), 4); }
        for (int i = 0; i < kBuf; ++i) {
            mbar_init(bar(B_KF + i), 2); mbar_init(bar(B_KE + i), 2);
            mbar_init(bar(B_VF + i), 2); mbar_init(bar(B_VE + i), 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(B_QF + i), 8);
            mbar_init(bar(B_QE + i), 10);
            mbar_init(bar(B_QRF + i), 1);
            mbar_init(bar(B_DRAIN + i), 1);
        }
        for (int i = 0; i < 4; ++i) { mbar_init(bar(B_S + i), 1); mbar_init(bar(B_P + i), 4); mbar_init(bar(B_O + i), 1); }
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
            const int tiles = seq_tiles<kRows>(a, q);
            if (tiles <= 4) {
                long long u = 0;
                for (int x = 0; x < tiles; ++x) u += item_units<kRows>(a, q, x);
                s_units[i] = u * a.c.n_kv;
            }
            else s_list[atomicAdd(&s_list_n, 1)] = i;
        }
        __syncthreads();
        for (int k = warp; k < s_list_n; k += kPfWarps) {
            const int i = s_list[k];
            const Seq q = load_seq(a, c0 + i);
            const int tiles = seq_tiles<kRows>(a, q);
            long long u = 0;
            for (int x = lane; x < tiles; x += 32) u += item_units<kRows>(a, q, x);
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
    // (no run is shorter than an item's own cost: short items then have a CTA each)
    const long long share = max(static_cast<long long>(kItemCost), (total + gridDim.x - 1) / gridDim.x);
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
                            if (x0 + lane < tiles) w = item_units<kRows>(a, q, x0 + lane);
                            long long wi = w;
#pragma unroll
                            for (int off = 1; off < 32; off <<= 1) {
                                const long long o = __shfl_up_sync(kFull, wi, off);
                                if (lane >= off) wi += o;
                            }
                            const long long tb = at + wi - w;
                            if (w > 0 && u0 >= tb && u0 < tb + w) s_start = {s, h, x0 + lane, static_cast<int>(u0 - tb)};
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

    // The roles deal the 512 x 128 registers anew: 256 x 176 + 256 x 80 = 65,536.
    bool ok = true;
    if (warp == 15) {
        // ---------------- the items and their queries ----------------
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        // This warp alone walks the items for the warps of products and softmax, an item ahead of them.
        Walk w;
        w.begin(a, start, u0, u1);
        uint32_t it = 0;
        auto free_slot = [&]() {
            ok = mbar_wait(bar(B_QE + (it & 1)), ((it >> 1) & 1) ^ 1, &s_abort, a.st, kSiteQFree);
            ok = __all_sync(kFull, ok);
            return ok;
        };
        while (true) {
            const bool pages = w.pa < w.pb;
            // (a run that holds only units of the item's own cost has no piece)
            if (pages || w.own) {
                if (!free_slot()) break;
                Item m;
                m.q0 = w.q.q0; m.n = w.q.n; m.len = w.q.len;
                m.h = w.h; m.tile = w.tile; m.pa = w.pa; m.pb = w.pb;
                w.half(a, 0, m.x[0], m.y[0]);
                w.half(a, 1, m.x[1], m.y[1]);
                // the runs with pages of the item: b0 (its slot 1) .. b1 (their slots 0)
                m.b0 = static_cast<int>((w.item + kItemCost) / share);
                m.b1 = static_cast<int>((w.item + kItemCost + w.hi - w.lo - 1) / share);
                m.kind = w.pa == w.lo && w.pb == w.hi ? kWhole : kPart;
                if (lane == 0) s_item[it & 1] = m;
                const uint32_t q = smem_u32(smem + C::o_q) + (it & 1) * C::q_slot;
                const int r0 = w.tile * kRows, r1 = min(w.q.n * a.group, r0 + kRows);
                if (lane == 0) {
                    if (pages) mbar_arrive_expect_tx(bar(B_QRF + (it & 1)), (r1 - r0) * (D * 2));
                    else mbar_arrive(bar(B_QRF + (it & 1)));
                }
                __syncwarp();
                // a token's query heads of the key head lie side by side: one copy for each token
                if (pages) {
                    for (int i = r0 / a.group + lane; i * a.group < r1; i += 32) {
                        const int x = max(r0, i * a.group), y = min(r1, (i + 1) * a.group);
                        bulk_copy_g2s(q + (x - r0) * (D * 2),
                                      a.q + static_cast<long long>(w.q.q0 + i) * a.ld_q + static_cast<long long>(w.h * a.group + x - i * a.group) * D,
                                      (y - x) * (D * 2), bar(B_QRF + (it & 1)));
                    }
                }
                ++it;
            }
            w.next(a, u0, u1);
            if (w.end) break;
        }
        if (ok && free_slot() && lane == 0) {
            s_item[it & 1].kind = kEnd;
            mbar_arrive(bar(B_QRF + (it & 1)));
        }
        if (!ok) {       // copies in flight land before the CTA gives its shared memory up
            for (int i = 0; i < 2; ++i) {
                mbar_drain(bar(B_QRF + i), 0);
                mbar_drain(bar(B_QRF + i), 1);
            }
        }
    } else if (warp == 14) {
        // ---------------- pages from device memory ----------------
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
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
            w.next(a, u0, u1);
            if (w.end) break;
        }
        // copies in flight land before the CTA gives its shared memory up: on
        // success the converters have waited for all of them
        if (!ok) {
            for (int i = 0; i < kRaw; ++i) {
                mbar_drain(bar(B_RAWF + i), 0);
                mbar_drain(bar(B_RAWF + i), 1);
            }
        }
    } else if (warp >= 12) {
        // ---------------- products ----------------
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        // A warp for each tile: waits and commits cost issue time, which the
        // other tile's products then fill.  The warp walks together and one
        // elected lane issues: addresses and descriptors stay in uniform registers.
        constexpr uint32_t id_s = idesc_f16_f32(kTile, kPage), id_o = idesc_f16_f32(kTile, D);
        const uint32_t t = warp - 12;
        // a group of the queries is followed by the next after both halves
        const uint64_t q_desc = sw128_desc(smem_u32(smem + C::o_q) + t * C::q_tile) + (static_cast<uint64_t>((C::q_group - 1024) >> 4) << 32), k_desc = sw128_desc(smem_u32(smem + C::o_k)),
                       v_desc = sw128_desc(smem_u32(smem + C::o_v));
        const uint32_t ts = t * C::tile_cols + C::c_s, to = t * C::tile_cols + C::c_o;
        const uint32_t bar_s = bar(B_S + 2 * t), bar_o = bar(B_O + 2 * t);
        auto wait = [&](int i, uint32_t parity, int site) {
            ok = mbar_wait(bar(i), parity, &s_abort, a.st, site);
            ok = __all_sync(kFull, ok);
            return ok;
        };
        uint32_t kv = 0, vv = 0;                       // pages of keys and values so far
        uint32_t ns = 0, no = 0;                       // scores and outputs issued
        uint64_t qd = 0;
        auto scores = [&](bool active) {               // of the next page of keys
            if (!wait(B_KF + kv % kBuf, (kv / kBuf) & 1, kSiteKFull)) return;
            tc_fence_after();
            if (elect_one()) {
                if (active) {
                    const uint64_t d = k_desc + (kv % kBuf) * (C::k_tile >> 4);
#pragma unroll
                    for (int k = 0; k < D / 16; ++k)
                        tc_mma_bf16(ts + 64 * (ns & 1), qd + (k / 4) * (1024 >> 4) + (k % 4) * 2,
                                    d + (k / 4) * (kPage * 128 >> 4) + (k % 4) * 2, id_s, k > 0);
                    tc_commit(bar_s + 8 * (ns & 1));
                }
                tc_commit(bar(B_KE + kv % kBuf));
            }
            __syncwarp();
            ns += active;
            ++kv;
        };
        auto outputs = [&](bool active, bool add) {    // of the next page of values
            if (!wait(B_VF + vv % kBuf, (vv / kBuf) & 1, kSiteVFull)) return;
            if (active && !wait(B_P + 2 * t + (no & 1), (no >> 1) & 1, kSiteP)) return;
            tc_fence_after();
            if (elect_one()) {
                if (active) {
                    const uint64_t d = v_desc + (vv % kBuf) * (C::v_tile >> 4);
#pragma unroll
                    for (int k = 0; k < 4; ++k) tc_mma_ts(to, ts + 64 * (no & 1) + 8 * k, d + 2 * k, id_o, add || k > 0);
                    tc_commit(bar_o + 8 * (no & 1));
                }
                tc_commit(bar(B_VE + vv % kBuf));
            }
            __syncwarp();
            no += active;
            ++vv;
        };
        // The scores run a page ahead of the outputs within an item.
        for (uint32_t it = 0; ok; ++it) {
            const uint32_t slot = it & 1;
            if (!wait(B_QF + slot, (it >> 1) & 1, kSiteQ)) break;
            const Item& w = s_item[slot];
            if (w.kind == kEnd) break;
            const int pa = w.pa, pb = w.pb, x = w.x[t], y = w.y[t];
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_QE + slot));
            if (pa < pb) {
                qd = q_desc + slot * (C::q_slot >> 4);
                scores(x <= pa && pa < y);
                for (int p = pa; ok && p < pb; ++p) {
                    if (p + 1 < pb) scores(x <= p + 1 && p + 1 < y);
                    if (ok) outputs(x <= p && p < y, p > x);
                }
            }
        }
        // every product is done before TMEM and shared memory are given up
        if (elect_one()) tc_commit(bar(B_DRAIN + t));
        __syncwarp();
        mbar_drain(bar(B_DRAIN + t), 0);
    } else if (warp >= 8 && warp < 12) {
        // ---------------- 4 bits to fp16 operands ----------------
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        const bool keys = warp < 10;
        const int cw = (warp - 8) & 1;        // which of the two warps
        Walk w;
        w.begin(a, start, u0, u1);
        uint32_t n = 0, st = 0, ph = 0;
        const int i8 = lane >> 2, t = lane & 3;
        // A byte of value codes is a number of two tokens; over a warp, the 8 x 8 matrix (token chunk i8, token of
        // the chunk) of one number.  Four of them are stored at once: this lane gives the address of row
        // lane % 8 of matrix lane / 8, for numbers 0-3 and 4-7 of an 8-row group.
        const uint32_t vm = lane >> 3, vr = lane & 7;
        const uint32_t v_off[2] = {vm * 128 + ((vr ^ vm) * 16), (vm + 4) * 128 + ((vr ^ (vm + 4)) * 16)};
        const int b_free = keys ? B_KE : B_VE, b_full = keys ? B_KF : B_VF;
        while (ok) {
            for (int j = w.pa; j < w.pb && ok; ++j) {
                ok = mbar_wait(bar(B_RAWF + st), ph, &s_abort, a.st, kSiteRaw);
                if (ok) ok = mbar_wait(bar(b_free + n % kBuf), ((n / kBuf) & 1) ^ 1, &s_abort, a.st, keys ? kSiteKFree : kSiteVFree);
                ok = __all_sync(kFull, ok);
                if (!ok) break;
                const uint8_t* raw = smem + C::o_raw + st * C::raw;
                const bool bad = s_bad[st];
                constexpr int W = D / 32;           // words of a run
                if (keys) {
                    uint8_t* kt = smem + C::o_k + (n % kBuf) * C::k_tile;
                    // a thread converts runs of D/4 numbers of four tokens
                    uint32_t c[4][W], sc[4][L::R];
                    const int kt4 = lane & 3;
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const int tok = u * 16 + cw * 8 + i8;
                        const uint8_t* p = raw + tok * (D / 2) + kt4 * (D / 8);
                        if constexpr (W == 4) {
                            const uint4 v = *reinterpret_cast<const uint4*>(p);
                            c[u][0] = v.x; c[u][1] = v.y; c[u][2] = v.z; c[u][3] = v.w;
                            sc[u][0] = *reinterpret_cast<const uint16_t*>(raw + L::kScales + ((kt4 * 8 + i8) * 8 + (tok >> 3)) * 2);
                        } else {
                            const uint2 v = *reinterpret_cast<const uint2*>(p);
                            c[u][0] = v.x; c[u][1] = v.y;
                            sc[u][0] = raw[L::kScales + (kt4 * 8 + i8) * 8 + (tok >> 3)];
                        }
                    }
                    // numbers (D/4) kt4 + 8 i ..: half, 16-byte chunk of the row
                    const int half = D == 128 ? kt4 >> 1 : 0;
                    const int chunk0 = D == 128 ? (kt4 & 1) * 4 : kt4 * 2;
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const uint32_t two = e4m3x2_to_f16(bad ? 0u : sc[u][0]);
                        sc[u][0] = __byte_perm(two, 0, 0x1010);
                        if constexpr (L::R == 2) sc[u][1] = __byte_perm(two, 0, 0x3232);
                        uint8_t* row = kt + half * (kPage * 128) + (u * 16 + cw * 8 + i8) * 128;
#pragma unroll
                        for (int i0 = 0; i0 < W; ++i0) {
                            // the upper half's runs go in another order, so that eight threads' chunks differ in their banks
                            const int i = D == 128 ? i0 ^ (half * 2) : i0;
                            const uint32_t word = D == 128 ? (half ? c[u][(i0 ^ 2) % W] : c[u][i0]) : c[u][i0];
                            const uint32_t sr = D == 128 ? (i < 2 ? sc[u][0] : sc[u][L::R - 1]) : sc[u][0];
                            uint32_t f[4];
                            e2m1x8_to_f16(word, f[0], f[1], f[2], f[3]);
                            *reinterpret_cast<uint4*>(row + (((chunk0 + i) ^ i8) * 16)) =
                                make_uint4(hmul2_u(f[0], sr), hmul2_u(f[1], sr), hmul2_u(f[2], sr), hmul2_u(f[3], sr));
                        }
                    }
                } else {
                    const uint32_t vt = smem_u32(smem + C::o_v) + (n % kBuf) * C::v_tile;
                    // a thread converts a token pair's runs of D/8 numbers, four of the eight
                    uint32_t c[4][W], sc[4];
                    const int left = w.q.len - j * kPage;
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const int g = 4 * cw + u;
                        const uint8_t* p = raw + L::vCodes + ((i8 * 8 + g) * 4 + t) * L::U;
                        if constexpr (W == 4) {
                            const uint4 v = *reinterpret_cast<const uint4*>(p);
                            c[u][0] = v.x; c[u][1] = v.y; c[u][2] = v.z; c[u][3] = v.w;
                        } else {
                            const uint2 v = *reinterpret_cast<const uint2*>(p);
                            c[u][0] = v.x; c[u][1] = v.y;
                        }
                        sc[u] = *reinterpret_cast<const uint16_t*>(raw + L::vScales + (((D == 128 ? g : g / 2) * 4 + t) * 8 + i8) * 2);
                    }
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        uint32_t two = bad ? 0u : sc[u];
                        // tokens that the sequence does not have: their bytes may be anything
                        if (left < kPage) {
                            const int tok = 8 * i8 + 2 * t;
                            two = tok + 1 < left ? two : (tok < left ? (two & 0xffu) : 0u);
                        }
                        const uint32_t s2 = e4m3x2_to_f16(two);
                        const uint32_t row = vt + (4 * cw + u) * (L::U * 128);
#pragma unroll
                        for (int i = 0; i < W; ++i) {
                            uint32_t f[4];
                            e2m1x8_to_f16(c[u][i], f[0], f[1], f[2], f[3]);
                            stmatrix4(row + (i / 2) * 1024 + v_off[i & 1], hmul2_u(f[0], s2), hmul2_u(f[1], s2), hmul2_u(f[2], s2), hmul2_u(f[3], s2));
                        }
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(bar(b_full + n % kBuf));
                    mbar_arrive(bar(B_RAWE + st));
                }
                ++n;
                if (++st == kRaw) { st = 0; ph ^= 1; }
            }
            if (!ok) break;
            w.next(a, u0, u1);
            if (w.end) break;
        }
    } else {
        // ---------------- softmax: a thread is a row ----------------
        asm volatile("setmaxnreg.inc.sync.aligned.u32 176;");
        const int t = warp >> 2;                              // tile
        const int r_tile = (warp & 3) * 32 + lane;            // row of the tile = TMEM lane
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tb = tmem + t * C::tile_cols + lanes;
        uint32_t n = 0;              // pages of this tile so far
        // The warp's rows of an item's queries to fp16, when its tile's scores of the item before are done.
        auto prepare = [&](uint32_t it) {
            const uint32_t slot = it & 1;
            ok = mbar_wait(bar(B_QRF + slot), (it >> 1) & 1, &s_abort, a.st, kSiteQ);
            ok = __all_sync(kFull, ok);
            if (!ok) return;
            const Item& w = s_item[slot];
            if (w.kind != kEnd && w.pa < w.pb)
                convert_queries<D>(smem + C::o_q + slot * C::q_slot, s_f[slot], 4 * warp, 4 * warp + 4, w.n * a.group - w.tile * kRows,
                                   a.scale * kLog2e * (a.c.k_scale != nullptr ? a.c.k_scale[w.h] : 1.f), lane);
            if (lane == 0) mbar_arrive(bar(B_QF + slot));
        };
        prepare(0);
        for (uint32_t it = 0; ok; ++it) {
            const uint32_t slot = it & 1;
            uint8_t* q = smem + C::o_q + slot * C::q_slot;
            const Item& w = s_item[slot];
            if (w.kind == kEnd) break;
            const int x = w.x[t], y = w.y[t];
            const int r = w.tile * kRows + t * kTile + r_tile;   // row of the (sequence, head)
            const bool live = r < w.n * a.group;
            const int tok = r / a.group, head = w.h * a.group + r - tok * a.group;
            const float f = s_f[slot][t * kTile + r_tile];
            float m = -INFINITY, l = 0.f;                        // m in powers of two
            // Outputs of pages n - 1 and n - 2 may both be outstanding (the scores run ahead), so they
            // signal two barriers in turn: the one waited on is never two phases behind.
            if (x < y) {
                // places of the row and of the tile's first and last row, for the pages that need no mask
                const int p_row = w.len - w.n + tok;
                const int rt0 = w.tile * kRows + t * kTile, rt1 = min(w.n * a.group, rt0 + kTile) - 1;
                const int p_first = w.len - w.n + rt0 / a.group, p_last = w.len - w.n + rt1 / a.group;
                const int first_key = a.window > 0 ? p_row - a.window + 1 : 0;
                float mf = -INFINITY;                            // the maximum in use, before the factor
                float2 l2 = make_float2(0.f, 0.f);
                auto base_of = [&](float top) { return fmaf(top, f, -kRoom); };
                uint32_t s0[32], s1[32];                         // a page's scores
                auto wait_s = [&](uint32_t i) {
                    ok = mbar_wait(bar(B_S + 2 * t + (i & 1)), (i >> 1) & 1, &s_abort, a.st, kSiteS);
                    ok = __all_sync(kFull, ok);
                    tc_fence_after();
                    return ok;
                };
                auto load_s = [&](uint32_t i) {
                    tmem_ld32(tb + C::c_s + 64 * (i & 1), s0);
                    tmem_ld32(tb + C::c_s + 64 * (i & 1) + 32, s1);
                };
                auto hide = [&](int j) {
                    const int key0 = j * kPage;
                    if (key0 + kPage - 1 > p_first || (a.window > 0 && key0 <= p_last - a.window)) {
                        const int last = p_row - key0, first = first_key - key0;
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            if (k > last || k < first) s0[k] = 0xff800000u;
                            if (k + 32 > last || k + 32 < first) s1[k] = 0xff800000u;
                        }
                    }
                };
                if (wait_s(n)) {
                    load_s(n);
                    tmem_ld_wait();
                    hide(x);
                    float t0 = __uint_as_float(s0[0]), t1 = __uint_as_float(s1[0]);
#pragma unroll
                    for (int k = 1; k < 31; k += 2) {
                        t0 = max3(t0, __uint_as_float(s0[k]), __uint_as_float(s0[k + 1]));
                        t1 = max3(t1, __uint_as_float(s1[k]), __uint_as_float(s1[k + 1]));
                    }
                    mf = fmaxf(max3(t0, t1, __uint_as_float(s0[31])), __uint_as_float(s1[31]));
                }
                for (int j = x; j < y && ok; ++j, ++n) {
                    // The exponentials use the maximum so far and the page's own is found beside them: only
                    // when it is more than 2^kGrow above is the page done over, with O and l scaled.
                    uint32_t h[32];
                    float2 sum;
                    auto exponentials = [&]() {
                        const float base = mf == -INFINITY ? 0.f : -base_of(mf);
                        const float2 f2 = make_float2(f, f), b2 = make_float2(base, base);
                        float t0 = -INFINITY, t1 = -INFINITY;
                        sum = make_float2(0.f, 0.f);
                        float2 sum1 = sum;
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            t0 = max3(t0, __uint_as_float(s0[2 * k]), __uint_as_float(s0[2 * k + 1]));
                            t1 = max3(t1, __uint_as_float(s1[2 * k]), __uint_as_float(s1[2 * k + 1]));
                            float2 p0 = fma2(make_float2(__uint_as_float(s0[2 * k]), __uint_as_float(s0[2 * k + 1])), f2, b2);
                            float2 p1 = fma2(make_float2(__uint_as_float(s1[2 * k]), __uint_as_float(s1[2 * k + 1])), f2, b2);
                            p0.x = ex2(p0.x); p0.y = ex2(p0.y);
                            p1.x = ex2(p1.x); p1.y = ex2(p1.y);
                            sum = add2(sum, p0);
                            sum1 = add2(sum1, p1);
                            h[k] = pack_f16(p0.x, p0.y);
                            h[16 + k] = pack_f16(p1.x, p1.y);
                        }
                        sum = add2(sum, sum1);
                        return fmaxf(t0, t1);
                    };
                    const float now = exponentials();
                    if (__any_sync(kFull, now > mf && (mf == -INFINITY || (now - mf) * f > kGrow))) {
                        const float nm = fmaxf(mf, now);
                        const float sc = mf == -INFINITY ? 0.f : ex2((mf - nm) * f);
                        mf = nm;
                        l2.x *= sc;
                        l2.y *= sc;
                        if (j > x) {
                            // the outputs so far are complete when page n - 1's are
                            ok = mbar_wait(bar(B_O + 2 * t + ((n - 1) & 1)), ((n - 1) >> 1) & 1, &s_abort, a.st, kSiteO);
                            ok = __all_sync(kFull, ok);
                            if (!ok) break;
                            tc_fence_after();
#pragma unroll 1
                            for (int i = 0; i < D / 16; ++i) {
                                uint32_t o[16];
                                tmem_ld16(tb + C::c_o + 16 * i, o);
                                tmem_ld_wait();
#pragma unroll
                                for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * sc);
                                tmem_st16(tb + C::c_o + 16 * i, o);
                            }
                        }
                        load_s(n);
                        tmem_ld_wait();
                        hide(j);
                        exponentials();
                    }
                    l2 = add2(l2, sum);
                    // P goes out before the wait for the next page's scores: the tensor cores have work in between
                    // (the other way round, with those loads beside this store, took 547 us for 8192 tokens, not 472)
                    const bool more = j + 1 < y;
                    tmem_st32(tb + C::c_s + 64 * (n & 1), h);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(B_P + 2 * t + (n & 1)));
                    if (more) {
                        if (!wait_s(n + 1)) break;
                        load_s(n + 1);
                        tmem_ld_wait();
                        hide(j + 1);
                    }
                }
                l = l2.x + l2.y;
                m = mf == -INFINITY ? -INFINITY : base_of(mf);
            }
            if (ok) prepare(it + 1);
            if (ok && x < y) {
                ok = mbar_wait(bar(B_O + 2 * t + ((n - 1) & 1)), ((n - 1) >> 1) & 1, &s_abort, a.st, kSiteO);
                ok = __all_sync(kFull, ok);
                tc_fence_after();
            }
            if (!ok) break;
            // ---- the piece's result ----
            // Rows leave through shared memory, so that a warp stores whole rows and not 32 bytes of each of 32
            // (an item's 64 KB of outputs: 5500 clocks, 6700 the other way): the warp's rows of queries are not
            // needed any more once its tile's last scores are there.
            uint8_t* stage = q + (t * kTile + (warp & 3) * 32) * (D * 2);
            auto put = [&](int i, const float (&o)[32], float by) {   // numbers 32 i .. of the lane's row
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    uint32_t v[4];
#pragma unroll
                    for (int z = 0; z < 4; ++z) {
                        const __nv_bfloat162 b = __floats2bfloat162_rn(o[8 * k + 2 * z] * by, o[8 * k + 2 * z + 1] * by);
                        memcpy(&v[z], &b, 4);
                    }
                    *reinterpret_cast<uint4*>(stage + lane * (D * 2) + (((4 * i + k) ^ (lane & 7)) * 16)) = make_uint4(v[0], v[1], v[2], v[3]);
                }
            };
            auto flush = [&](float m, float l) {
                const long long at = live ? static_cast<long long>(w.q0 + tok) * a.ld_out + static_cast<long long>(head) * D : -1;
                constexpr int LR = D / 8, RP = 32 / LR;              // lanes of a row, rows of a pass
                const int c = lane % LR;
                __syncwarp();
#pragma unroll 8
                for (int k = 0; k < LR; ++k) {
                    const int row = k * RP + lane / LR;
                    const uint4 v = *reinterpret_cast<const uint4*>(stage + row * (D * 2) + ((c ^ (row & 7)) * 16));
                    const long long to = __shfl_sync(kFull, at, row);
                    if (to >= 0) *reinterpret_cast<uint4*>(a.out + to + c * 8) = v;
                }
                if (live && a.lse != nullptr)
                    a.lse[static_cast<long long>(w.q0 + tok) * a.n_q + head] = l > 0.f || l != l ? m * kLn2f + logf(l) : -INFINITY;
            };
            const float vs = a.c.v_scale != nullptr ? a.c.v_scale[w.h] : 1.f;
            constexpr int kSlot = kRows * (D + 2);
            const int row = t * kTile + r_tile;
            auto part = [&](int b) { return a.partial + (static_cast<long long>(b) * 2 + (b == w.b0 ? 1 : 0)) * kSlot; };
            const float inv = l == 0.f ? 0.f : vs / l;
#pragma unroll 1
            for (int i = 0; i < D / 32; ++i) {
                uint32_t o[32];
                if (x < y) {
                    tmem_ld32(tb + C::c_o + 32 * i, o);
                    tmem_ld_wait();
                } else {
#pragma unroll
                    for (int k = 0; k < 32; ++k) o[k] = 0u;
                }
                if (w.kind == kWhole) {
                    float v[32];
#pragma unroll
                    for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(o[k]);
                    put(i, v, inv);
                } else {
                    // columns in fours, rows side by side: a warp's stores are dense
                    float4* dst = reinterpret_cast<float4*>(part(blockIdx.x)) + (8 * i * kRows + row);
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        __stcg(dst + k * kRows, make_float4(__uint_as_float(o[4 * k]), __uint_as_float(o[4 * k + 1]),
                                                            __uint_as_float(o[4 * k + 2]), __uint_as_float(o[4 * k + 3])));
                }
            }
            tc_fence_before();      // O is read: the next item's products follow through B_P
            if (w.kind == kWhole) {
                flush(m, l);
            } else {
                // A warp's rows are joined by the warp that is the last to arrive with them.
                __stcg(part(blockIdx.x) + kRows * D + row, m);
                __stcg(part(blockIdx.x) + kRows * D + kRows + row, l);
                __syncwarp();
                int* counter = a.counters + w.b0 * 8 + warp;
                int ticket = 0;
                if (lane == 0) {
                    __threadfence();
                    ticket = atom_add_acq_rel_gpu(counter, 1);
                    if (ticket == w.b1 - w.b0) *counter = 0;
                }
                ticket = __shfl_sync(kFull, ticket, 0);
                if (ticket == w.b1 - w.b0) {
                    __threadfence();
                    float gm = -INFINITY, gl = 0.f;
                    for (int b = w.b0; b <= w.b1; ++b) gm = fmaxf(gm, __ldcg(part(b) + kRows * D + row));
                    for (int b = w.b0; b <= w.b1; ++b) {
                        const float mk = __ldcg(part(b) + kRows * D + row), lk = __ldcg(part(b) + kRows * D + kRows + row);
                        // a piece that has seen nothing has l = 0, or a NaN that stays
                        gl += mk == -INFINITY ? lk : ex2(mk - gm) * lk;
                    }
                    const float ginv = gl == 0.f ? 0.f : vs / gl;
                    // 32 numbers of a piece at a time, and the next 32 on their way
                    float4 v[8];
                    float mk;
                    auto load = [&](int i, int b) {
                        mk = __ldcg(part(b) + kRows * D + row);
                        const float4* src = reinterpret_cast<const float4*>(part(b)) + (8 * i * kRows + row);
#pragma unroll
                        for (int k = 0; k < 8; ++k) v[k] = __ldcg(src + k * kRows);
                    };
                    load(0, w.b0);
#pragma unroll 1
                    for (int i = 0; i < D / 32; ++i) {
                        float o[32];
#pragma unroll
                        for (int k = 0; k < 32; ++k) o[k] = 0.f;
#pragma unroll 1
                        for (int b = w.b0; b <= w.b1; ++b) {
                            float4 u[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k) u[k] = v[k];
                            const float ek = mk == -INFINITY ? 0.f : ex2(mk - gm);
                            if (b < w.b1) load(i, b + 1);
                            else if (i + 1 < D / 32) load(i + 1, w.b0);
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                o[4 * k] = fmaf(ek, u[k].x, o[4 * k]); o[4 * k + 1] = fmaf(ek, u[k].y, o[4 * k + 1]);
                                o[4 * k + 2] = fmaf(ek, u[k].z, o[4 * k + 2]); o[4 * k + 3] = fmaf(ek, u[k].w, o[4 * k + 3]);
                            }
                        }
                        put(i, o, ginv);
                    }
                    flush(gm, gl);
                }
            }
            // the slot's bytes were read and written here; the next copy into them follows
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_QE + slot));
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
    return launch_pdl(k, dim3(min(sm_count(), kPromptMaxCtas)), dim3(kPfThreads), Pf<D>::smem, s, a);
}

}  // namespace

size_t attn_prefill_pieces(int D) {
    return static_cast<size_t>(kPromptMaxCtas) * 2 * kRows * (D + 2) * sizeof(float);
}

cudaError_t launch_attn_prefill(const AttnArgs& a, cudaStream_t s) {
    return a.c.head_dim == 128 ? launch_pf<128>(a, s) : launch_pf<64>(a, s);
}

}  // namespace moe
