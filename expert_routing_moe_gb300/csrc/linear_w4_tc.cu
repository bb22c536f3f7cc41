// linear_w4_tc.cu -- products with weights in 4 bits for many tokens: tcgen05.
//
// A tile of the output is 256 weight rows (two halves of 128 TMEM lanes) and up
// to 192 tokens.  For 64 columns at a time, four warps turn each half's codes
// to bf16 in TMEM (a thread is a row), where they are the products' A
// operand, and the tokens' numbers come to shared memory by TMA as the B operand:
//     D[row][token] += A[row][64] B[token][64]^T      (fp32 in TMEM)
//
// 2001 tokens through 5120 x 2048 take 29.3 us (1430 TFLOP/s of the 1910 that a
// large bf16 product of the library reaches), 8192 tokens 98 us (1750): the
// products are fed without a pause but for the first and last step of a tile.  Few
// tokens are bound by the conversion, 630 clocks for 256 rows of 64 columns.
//
// Where there are fewer tiles than SMs, clusters of two, four or eight CTAs
// share a tile's columns and add up their parts through each other's shared
// memory: 300 tokens through 8192 x 2048 30.4 -> 18.6 us, 100 44.7 -> 14.1.
//
// Rows of x that start anywhere are loaded by eight warps, which costs a step 1150 clocks instead of 630: 43 tokens
// through 6847 x 36585 70 us (6848: 41), 1000 through 2049 x 5120 42 (2056: 17).  (Four warps a unit of eight numbers at a
// time: 256 us; eight lanes a token, four turns ahead: 118; warps whose rows begin alike, so that only halves
// are shifted: 69.)
//
// Warps: 0-15 convert (eight for each half, in two groups that take the steps in
// turn) and write the outputs, 16 and 17 issue a half's products each, 18 copies the
// weights' tiles, 19 the tokens (or 19-26, with plain loads, where rows of x do not start at 16-byte boundaries).
// TMEM columns: D 2 x 192, A 2 halves x 2 buffers x 32.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "launch.h"
#include "linear_w4.cuh"
#include "tc_ts.cuh"
#include "tmap.h"
#include "w4.cuh"

namespace moe {

namespace cg = cooperative_groups;

namespace {

constexpr int kHalves = 2;
constexpr int kTileRows = kHalves * kW4Tile;
constexpr int kStep = 64;                 // columns of a step
constexpr int kMaxTok = 192;
constexpr int kRaw = 3;                   // weights' tiles in flight, of a half
constexpr int kB = 6;                     // steps of tokens in flight
constexpr int kBBytes = kMaxTok * kStep * 2;
constexpr int kRawOff = kB * kBBytes;
constexpr int kSmem = kRawOff + kHalves * kRaw * kW4Bytes + 1024;   // slack for 1024-byte alignment
constexpr int kColA = kHalves * kMaxTok;  // TMEM column of the A buffers
constexpr int kTeams = 2;                 // of warps that load x where TMA cannot: they take the steps in turn
constexpr int kTeam = 4;                  // warps of one
constexpr int kLoaders = kTeams * kTeam;
constexpr int kLoadTok = kTeam * 16;      // tokens of a team at a time
constexpr int kConv = 16;                 // warps that convert
constexpr int kWarpMma = kConv, kWarpW = kConv + 2, kWarpX = kConv + 3;

constexpr int kMaxSplit = 8;              // CTAs that share a tile
// Clusters of that many CTAs that run at a time: some groups of SMs have too few left for another one.
int clusters_of(int split) { return sm_count() / split - (split == 8 ? 4 : split == 4 ? 2 : 0); }

enum Bar : int { B_WF = 0, B_WE = B_WF + kHalves * kRaw, B_AF = B_WE + kHalves * kRaw, B_AE = B_AF + 4, B_BF = B_AE + 4, B_BE = B_BF + kB,
                 B_DF = B_BE + kB, B_DE, B_DRAIN, B_N = B_DRAIN + kHalves };
enum Site : int { kSiteWFull = 41, kSiteWEmpty, kSiteAFull, kSiteAEmpty, kSiteBFull, kSiteBEmpty, kSiteDFull, kSiteDEmpty };

__device__ __forceinline__ void st32(uint32_t taddr, const uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
        "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(v[16]), "r"(v[17]), "r"(v[18]),
        "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]), "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]),
        "r"(v[28]), "r"(v[29]), "r"(v[30]), "r"(v[31])
        : "memory");
}

long long tiles_of(const LinearArgs& a, int tok) { return static_cast<long long>((a.N + kTileRows - 1) / kTileRows) * ((a.T + tok - 1) / tok); }

// The tiles of a CTA: row tile and first token.
struct Tiles {
    int tok_tiles, total, tok;
    __device__ int row(int i) const { return i / tok_tiles; }
    __device__ int t0(int i) const { return i % tok_tiles * tok; }
};

template <bool TMA, bool SPLIT>
__global__ void __launch_bounds__((kWarpX + (TMA ? 1 : kLoaders)) * 32, 1) linear_w4_tc_kernel(const LinearArgs a, const __grid_constant__ CUtensorMap map_x, int tok, int ctas) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    __shared__ __align__(8) uint64_t bars[B_N];
    __shared__ uint32_t s_tmem;
    __shared__ volatile int s_abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    if (threadIdx.x == 0) {
        for (int i = 0; i < kHalves * kRaw; ++i) { mbar_init(bar(B_WF + i), 1); mbar_init(bar(B_WE + i), 8); }
        for (int i = 0; i < 4; ++i) { mbar_init(bar(B_AF + i), 4); mbar_init(bar(B_AE + i), 1); }
        for (int i = 0; i < kB; ++i) { mbar_init(bar(B_BF + i), TMA ? 1 : kTeam); mbar_init(bar(B_BE + i), kHalves); }
        mbar_init(bar(B_DF), kHalves);
        mbar_init(bar(B_DE), kConv);
        for (int i = 0; i < kHalves; ++i) mbar_init(bar(B_DRAIN + i), 1);
        fence_mbar_init();
        s_abort = 0;
    }
    if (warp == kWarpMma) {
        tmem_alloc(smem_u32(&s_tmem), 512);
        tmem_relinquish();
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;             // all 512 columns are taken, so it is 0
    Tiles w;
    w.tok = tok;
    w.tok_tiles = (a.T + tok - 1) / tok;
    const int halves = (a.N + kW4Tile - 1) / kW4Tile;
    w.total = (halves + kHalves - 1) / kHalves * w.tok_tiles;
    // a cluster of `split` CTAs has a tile, each a part of its columns; without one a CTA has every gridDim.x-th tile
    const int split = SPLIT ? ctas : 1;
    const int part = SPLIT ? static_cast<int>(blockIdx.x) % split : 0;
    const int first = blockIdx.x / split, by = gridDim.x / split;
    const int c0 = a.kt * part / split, c1 = a.kt * (part + 1) / split;
    bool ok = true;

    pdl_wait();
    pdl_trigger();
    if (warp == kWarpW) {
        // ---------------- weights ----------------
        if (lane == 0) {
            uint32_t n = 0;            // tiles of a half copied
            for (int i = first; i < w.total && ok; i += by)
                for (int c = c0; c < c1 && ok; ++c, ++n) {
                    const int st = n % kRaw;
                    for (int m = 0; m < kHalves && ok; ++m) {
                        ok = mbar_wait(bar(B_WE + m * kRaw + st), ((n / kRaw) & 1) ^ 1, &s_abort, a.st, kSiteWEmpty);
                        if (!ok) break;
                        // the last tile's second half may be none: its rows are not written
                        const int half = min(w.row(i) * kHalves + m, halves - 1);
                        mbar_arrive_expect_tx(bar(B_WF + m * kRaw + st), kW4Bytes);
                        bulk_copy_g2s(smem_u32(smem + kRawOff + (m * kRaw + st) * kW4Bytes), a.tiles + (static_cast<long long>(half) * a.kt + c) * kW4Bytes, kW4Bytes,
                                      bar(B_WF + m * kRaw + st));
                    }
                }
            if (!ok)                   // what is in flight lands before the CTA ends
                for (int i = 0; i < kHalves * kRaw; ++i) {
                    mbar_drain(bar(B_WF + i), 0);
                    mbar_drain(bar(B_WF + i), 1);
                }
        }
    } else if (warp >= kWarpX) {
        // ---------------- tokens ----------------
        uint32_t n = 0;
        if (TMA) {
            if (lane == 0) {
                tma_prefetch_desc(&map_x);
                const uint64_t policy = l2_policy_evict_last();
                for (int i = first; i < w.total && ok; i += by)
                    for (int k = 2 * c0; k < 2 * c1 && ok; ++k, ++n) {
                        const int st = n % kB;
                        ok = mbar_wait(bar(B_BE + st), ((n / kB) & 1) ^ 1, &s_abort, a.st, kSiteBEmpty);
                        if (!ok) break;
                        mbar_arrive_expect_tx(bar(B_BF + st), tok * kStep * 2);
                        tma_load_2d(smem_u32(smem + st * kBBytes), &map_x, k * kStep, w.t0(i), bar(B_BF + st), policy);
                    }
                if (!ok)
                    for (int i = 0; i < kB; ++i) {
                        mbar_drain(bar(B_BF + i), 0);
                        mbar_drain(bar(B_BF + i), 1);
                    }
            }
        } else {
            // A thread has half of a token's 64 numbers, 64 tokens at a time: five 16-byte words that hold them, shifted into
            // place.  The words of the two turns to come are on their way meanwhile.
            const int team = (warp - kWarpX) / kTeam, half = threadIdx.x & 1, r = (threadIdx.x - kWarpX * 32) % (kTeam * 32) >> 1;
            const int turns = (tok + kLoadTok - 1) / kLoadTok, k0 = 2 * c0 + team;      // (a tile has an even number of steps)
            n = team;
            struct At {
                int i, k, turn, t;                         // t: token of the thread's first turn
            };
            auto next = [&](At& at) {
                if (++at.turn < turns) return;
                at.turn = 0;
                if ((at.k += kTeams) < 2 * c1) return;
                at.k = k0;
                at.i += by;
                at.t = w.t0(at.i) + r;
            };
            const __nv_bfloat16* x0 = a.x + half * 32;
            auto place = [&](const At& at, const __nv_bfloat16*& p, int& left) {
                const int t = at.t + at.turn * kLoadTok;
                p = x0 + (t * a.ld_x + at.k * kStep);
                left = t < a.T ? max(0, min(32, a.K - half * 32 - at.k * kStep)) : 0;       // numbers that there are
            };
            auto fetch = [&](uint32_t (&v)[20], const At& at) {
                if (at.i >= w.total) return;
                const __nv_bfloat16* p;
                int left;
                place(at, p, left);
                const uintptr_t from = reinterpret_cast<uintptr_t>(p);
                const uint4* words = reinterpret_cast<const uint4*>(from & ~static_cast<uintptr_t>(15));
                const int bytes = left > 0 ? static_cast<int>(from & 15) + 2 * left : 0;
#pragma unroll
                for (int x = 0; x < 5; ++x) {
                    const uint4 q = 16 * x < bytes ? __ldg(words + x) : make_uint4(0u, 0u, 0u, 0u);
                    v[4 * x] = q.x; v[4 * x + 1] = q.y; v[4 * x + 2] = q.z; v[4 * x + 3] = q.w;
                }
            };
            At here = {first, k0, 0, w.t0(first) + r}, ahead = here;
            auto turn = [&](uint32_t (&v)[20]) {
                const int st = n % kB;
                if (here.turn == 0) ok = wait_warp(bar(B_BE + st), ((n / kB) & 1) ^ 1, &s_abort, a.st, kSiteBEmpty);
                if (!ok) return;
                const __nv_bfloat16* p;
                int left;
                place(here, p, left);
                const int off = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 15), to = here.turn * kLoadTok + r;
                // whole words, two and one at a time, then half a word
#pragma unroll
                for (int x = 0; x < 18; ++x) v[x] = off & 8 ? v[x + 2] : v[x];
#pragma unroll
                for (int x = 0; x < 17; ++x) v[x] = off & 4 ? v[x + 1] : v[x];
#pragma unroll
                for (int x = 0; x < 16; ++x) v[x] = __funnelshift_r(v[x], v[x + 1], (off & 2) * 8);
                if (left < 32) {
#pragma unroll
                    for (int x = 0; x < 16; ++x) v[x] = left >= 2 * x + 2 ? v[x] : left == 2 * x + 1 ? v[x] & 0xffffu : 0u;
                }
                if (to < tok) {
                    uint8_t* dst = smem + st * kBBytes + to * 128;
#pragma unroll
                    for (int x = 0; x < 4; ++x)
                        *reinterpret_cast<uint4*>(dst + (((half * 4 + x) ^ (to & 7)) * 16)) = make_uint4(v[4 * x], v[4 * x + 1], v[4 * x + 2], v[4 * x + 3]);
                }
                if (here.turn == turns - 1) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(B_BF + st));
                    n += kTeams;
                }
                next(here);
                fetch(v, ahead);
                next(ahead);
            };
            uint32_t even[20], odd[20];
            fetch(even, ahead);
            next(ahead);
            fetch(odd, ahead);
            next(ahead);
            while (ok && here.i < w.total) {
                turn(even);
                if (ok && here.i < w.total) turn(odd);
            }
        }
    } else if (warp >= kWarpMma && warp < kWarpMma + kHalves) {
        // ---------------- products: a warp for each half ----------------
        const int m = warp - kWarpMma;
        const uint32_t idesc = idesc_bf16_f32(kW4Tile, tok);
        const uint64_t b0 = sw128_desc(smem_u32(smem));
        uint32_t n = 0, done = 0;
        for (int i = first; i < w.total && ok; i += by, ++done) {
            ok = wait_warp(bar(B_DE), (done & 1) ^ 1, &s_abort, a.st, kSiteDEmpty);
            for (int k = 2 * c0; k < 2 * c1 && ok; ++k, ++n) {
                const int st = n % kB, buf = n & 1;
                ok = wait_warp(bar(B_BF + st), (n / kB) & 1, &s_abort, a.st, kSiteBFull) &&
                     wait_warp(bar(B_AF + m * 2 + buf), (n >> 1) & 1, &s_abort, a.st, kSiteAFull);
                if (!ok) break;
                tc_fence_after();
                if (elect_one()) {
                    const uint64_t b = b0 + static_cast<uint64_t>(st * (kBBytes >> 4));
                    const uint32_t at = kColA + (m * 2 + buf) * 32;
#pragma unroll
                    for (int x = 0; x < 4; ++x) mma_ts(m * kMaxTok, at + x * 8, b + x * 2, idesc, k > 2 * c0 || x > 0);
                    tc_commit(bar(B_AE + m * 2 + buf));
                    tc_commit(bar(B_BE + st));
                }
                __syncwarp();
            }
            if (ok && elect_one()) tc_commit(bar(B_DF));
            __syncwarp();
        }
        if (!ok && n > 0) {            // the products in flight end before TMEM is freed
            if (elect_one()) tc_commit(bar(B_DRAIN + m));
            __syncwarp();
            mbar_drain(bar(B_DRAIN + m), 0);
        }
    } else {
        // ---------------- weights to bf16, and the outputs ----------------
        // A group takes every other step, so its own half of the columns of each tile of weights.
        const int m = warp >> 3, g = (warp >> 2) & 1, r = (warp & 3) * 32 + lane;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        uint32_t raw = 0, done = 0;
        for (int i = first; i < w.total && ok; i += by, ++done) {
            for (int c = c0; c < c1 && ok; ++c, ++raw) {
                const int st = raw % kRaw;
                ok = wait_warp(bar(B_WF + m * kRaw + st), (raw / kRaw) & 1, &s_abort, a.st, kSiteWFull);
                if (!ok) break;
                const uint8_t* tile = smem + kRawOff + (m * kRaw + st) * kW4Bytes;
                const uint32_t four = *reinterpret_cast<const uint32_t*>(tile + w4_scale(r, 4 * g));
                const uint4 run[2] = {*reinterpret_cast<const uint4*>(tile + w4_run(r, 2 * g)), *reinterpret_cast<const uint4*>(tile + w4_run(r, 2 * g + 1))};
                uint32_t v[32];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    uint32_t s[2];
                    w4_scales(x == 0 ? four & 0xffffu : four >> 16, s[0], s[1]);
                    const uint32_t words[4] = {run[x].x, run[x].y, run[x].z, run[x].w};
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        uint32_t f[4];
                        w4_values(words[y], f);
#pragma unroll
                        for (int j = 0; j < 4; ++j) v[x * 16 + y * 4 + j] = bmul2(f[j], s[y / 2]);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_WE + m * kRaw + st));
                ok = wait_warp(bar(B_AE + m * 2 + g), (raw & 1) ^ 1, &s_abort, a.st, kSiteAEmpty);
                if (!ok) break;
                tc_fence_after();
                st32(kColA + (m * 2 + g) * 32 + lanes, v);
                st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_AF + m * 2 + g));
            }
            if (!ok) break;
            ok = wait_warp(bar(B_DF), done & 1, &s_abort, a.st, kSiteDFull);
            if (!ok) break;
            tc_fence_after();
            if constexpr (SPLIT) {
                // what is not yet the whole sum waits in shared memory, whose operands are used up: [token][row]
                for (int c = 16 * g; c < tok; c += 32) {
                    uint32_t d[16];
                    tmem_ld16(m * kMaxTok + lanes + c, d);
                    tmem_ld_wait();
#pragma unroll
                    for (int x = 0; x < 16; ++x) reinterpret_cast<float*>(smem)[(c + x) * kTileRows + m * kW4Tile + r] = __uint_as_float(d[x]);
                }
                break;                 // (the CTA's only tile)
            }
            const int row = w.row(i) * kTileRows + m * kW4Tile + r, t0 = w.t0(i);
            const bool live = row < a.N;
            const float scale = (live && a.row_scale != nullptr ? a.row_scale[row] : 1.f) * kW4Up;
            const float bias = live && a.bias != nullptr ? a.bias[row] : 0.f;
            // the groups share the tokens, 16 at a time
            auto put = [&](auto* y, auto add) {
                auto* p = y + static_cast<long long>(t0 + 16 * g) * a.ld_y + row;
                for (int c = 16 * g; c < tok; c += 32, p += 32 * a.ld_y) {
                    const int left = live ? a.T - (t0 + c) : 0;      // tokens of the 16 that there are
                    auto* q = p;
                    // (all on their way at once: a store could be to what a later load reads)
                    float old[16];
                    if constexpr (decltype(add)::value) {
#pragma unroll
                        for (int x = 0; x < 16; ++x, q += a.ld_y) old[x] = x < left ? *q : 0.f;
                        q = p;
                    }
                    uint32_t d[16];
                    tmem_ld16(m * kMaxTok + lanes + c, d);
                    tmem_ld_wait();
#pragma unroll
                    for (int x = 0; x < 16; ++x, q += a.ld_y) {
                        float v = fmaf(__uint_as_float(d[x]), scale, bias);
                        if (x < left) {
                            if constexpr (decltype(add)::value) v += old[x];
                            if constexpr (sizeof(*q) == 2) *q = __float2bfloat16_rn(v);
                            else *q = v;
                        }
                    }
                }
            };
            if (a.y_bf16) put(static_cast<__nv_bfloat16*>(a.y), std::false_type());
            else if (a.add) put(static_cast<float*>(a.y), std::true_type());
            else put(static_cast<float*>(a.y), std::false_type());
            tc_fence_before();         // D is read: the next tile's products may begin
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_DE));
        }
    }
    __syncthreads();
    if (warp == kWarpMma) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
    if constexpr (SPLIT) {
        // each CTA adds up the parts of some of the tile's tokens, in the order of the columns
        cg::cluster_group cluster = cg::this_cluster();
        cluster.sync();
        const float* parts[kMaxSplit];
#pragma unroll
        for (int i = 0; i < kMaxSplit; ++i) parts[i] = cluster.map_shared_rank(reinterpret_cast<const float*>(smem), i < split ? i : 0);
        const int x0 = tok * part / split, x1 = min(tok * (part + 1) / split, a.T - w.t0(first));
        for (int u = warp; u < (x1 - x0) * kHalves; u += blockDim.x / 32) {
            const int x = x0 + u / kHalves, r = u % kHalves * kW4Tile + lane * 4, row = w.row(first) * kTileRows + r;
            float4 v[kMaxSplit], sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int i = 0; i < kMaxSplit; ++i)
                if (i < split) v[i] = *reinterpret_cast<const float4*>(parts[i] + x * kTileRows + r);
#pragma unroll
            for (int i = 0; i < kMaxSplit; ++i)
                if (i < split) { sum.x += v[i].x; sum.y += v[i].y; sum.z += v[i].z; sum.w += v[i].w; }
            const float of[4] = {sum.x, sum.y, sum.z, sum.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (row + i >= a.N) break;
                const float scale = (a.row_scale != nullptr ? a.row_scale[row + i] : 1.f) * kW4Up;
                put_y(a, w.t0(first) + x, row + i, fmaf(of[i], scale, a.bias != nullptr ? a.bias[row + i] : 0.f));
            }
        }
        cluster.sync();                // no CTA leaves while its shared memory is read
    }
}

// [T][K] bf16 with rows `ld` numbers apart, boxes of 64 columns and `tok` rows with the 128-byte swizzle.
bool map_tokens(CUtensorMap* m, const LinearArgs& a, int tok) {
    cuuint64_t dims[2] = {static_cast<cuuint64_t>(a.K), static_cast<cuuint64_t>(a.T)};
    cuuint64_t strides[1] = {static_cast<cuuint64_t>(a.ld_x) * 2};
    cuuint32_t box[2] = {kStep, static_cast<cuuint32_t>(tok)};
    cuuint32_t estr[2] = {1, 1};
    return encode_tiled(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<__nv_bfloat16*>(a.x), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

template <bool TMA, bool SPLIT>
cudaError_t launch(const LinearArgs& a, const LinearTile& t, cudaStream_t s) {
    CUtensorMap map = {};
    if (TMA && !map_tokens(&map, a, t.tok)) return cudaErrorInvalidValue;
    auto* k = linear_w4_tc_kernel<TMA, SPLIT>;
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    const long long ctas = tiles_of(a, t.tok) * t.split;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(SPLIT || ctas < sm_count() ? ctas : sm_count()));
    cfg.blockDim = dim3((kWarpX + (TMA ? 1 : kLoaders)) * 32);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = t.split;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = SPLIT ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, k, a, static_cast<const CUtensorMap>(map), t.tok, t.split);
}

}  // namespace

// Tokens of a tile, and CTAs that share one: those that make the longest CTA's time shortest.  A step of 64 columns takes 4 clocks
// a token and some 100 more, or 630 for the conversion of its weights (1150 where x is loaded without TMA), whichever is longer, and a tile its outputs; parts
// meet in 2000 clocks more, and clusters of four and eight leave some SMs without work.  (2001 tokens through 5120 x 2048 with 64,
// 96, 128, 144, 160 tokens a tile: 58.0, 37.6, 39.2, 28.1, 29.8 us; 8192 tokens with 128, 144, 160: 112, 104, 98 us.)
static LinearTile best_tile(const LinearArgs& a, double least, int only) {
    LinearTile best = {16, 1, 1e300};
    for (int tok = 16; tok <= kMaxTok && tok < a.T + 16; tok += 16) {
        const long long tiles = tiles_of(a, tok);
        const double step = std::max(4.0 * tok + 100.0, least);
        for (int split = 1; split <= kMaxSplit && split <= a.kt; split *= 2) {
            if (split > 1 && tiles > clusters_of(split)) break;
            if (only > 0 && split != only) continue;
            const long long waves = split > 1 ? 1 : (tiles + sm_count() - 1) / sm_count();
            const double clocks = static_cast<double>(waves) * (2.0 * ((a.kt + split - 1) / split) * step + 1500.0 + 12.0 * tok) + (split > 1 ? 2000.0 + 8.0 * tok : 0.0);
            if (clocks < best.clocks) best = {tok, split, clocks};
        }
    }
    return best;
}
// The order of the sums goes by the kernel and by how many CTAs share a tile, so both are chosen as if x's rows started at
// 16-byte boundaries; only a tile's tokens go by where they do start.
LinearTile linear_w4_tile(const LinearArgs& a) {
    LinearTile t = best_tile(a, 630.0, 0);
    if (!a.wide) t.tok = best_tile(a, 1150.0, t.split).tok;
    return t;
}

cudaError_t launch_linear_w4_tc(const LinearArgs& a, const LinearTile& t, cudaStream_t s) {
    if (t.split > 1) return a.wide ? launch<true, true>(a, t, s) : launch<false, true>(a, t, s);
    return a.wide ? launch<true, false>(a, t, s) : launch<false, false>(a, t, s);
}

}  // namespace moe
