// linear_w4.cu -- products with weights in 4 bits, and their packing.
//
//   y[t][n] = r[n] * sum_k x[t][k] c[n][k] s[n][k/16]  (+ bias[n]) (+ y[t][n])
//
// c * s has at most six significant bits, so it is exact in bf16, and so are the
// products of the tensor cores; sums are fp32.
//
// Few tokens (more: linear_w4_tc.cu): the weights are the 16-row operand of
// mma.sync.m16n8k16, eight tokens the other.  A CTA takes 16 or 32 rows a step;
// its warps share their columns, 128 at a time, and join their sums in shared
// memory in a fixed order.  A piece of weights is on its way while the one
// before is multiplied, the first one's bytes before the kernel before has ended.
//
// What bounds it: one token through 5120 x 2048 takes 3.7 us (a chain of
// loads; 3.1 us of host time), a head of 128001 x 2048 for five tokens 36.6 us for 148 MB (4.0 TB/s;
// 22 us at the rate of a copy).  No unit is full: issue slots 64%, ALUs 55%, DRAM
// 43%.  443 instructions go with a piece of 32 x 128, of which 240 turn codes into bf16 (15
// for eight); with 2048 columns a warp has two pieces, then eight warps
// store their sums, meet and add up eight, which is much of the rest.  (Two pieces ahead: 41.5 us, a CTA less fits; four
// CTAs an SM: 39.5 with spills; sums of two steps joined at a time: 38.4;
// pieces of all steps in equal runs for the warps, without a join a step: 43.7.)
#include <cuda_bf16.h>

#include "common.cuh"
#include "kv4.cuh"
#include "launch.h"
#include "linear_w4.cuh"
#include "tmap.h"
#include "w4.cuh"

namespace moe {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxStaged = 128 * 1024;   // bytes of x in shared memory

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint4 ldg_stream(const void* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

__device__ __forceinline__ void store_y(const LinearArgs& a, int t, int n, float v) {
    v *= a.row_scale == nullptr ? kW4Up : a.row_scale[n] * kW4Up;
    put_y(a, t, n, a.bias != nullptr ? v + a.bias[n] : v);
}

// What a lane holds of 16 MT rows and 128 columns: rows g + 8 i, columns 32 t .. 32 t + 31.
template <int MT>
struct Piece {
    uint4 w[2 * MT];
    uint32_t s[2 * MT];     // two scales each
};
template <int MT>
__device__ __forceinline__ const uint8_t* piece_at(const LinearArgs& a, int row0, int c) {
    return a.tiles + (static_cast<long long>(row0 / kW4Tile) * a.kt + c) * kW4Bytes;
}
template <int MT>
__device__ __forceinline__ void load_piece(Piece<MT>& p, const LinearArgs& a, int row0, int c, int lane) {
    const int g = lane >> 2, t = lane & 3, r = row0 % kW4Tile + g;
    const uint8_t* tile = piece_at<MT>(a, row0, c);
#pragma unroll
    for (int i = 0; i < 2 * MT; ++i) {
        p.w[i] = ldg_stream(tile + w4_run(r + 8 * i, t));
        p.s[i] = __ldg(reinterpret_cast<const uint16_t*>(tile + w4_scale(r + 8 * i, 2 * t)));
    }
}

// NT: groups of eight tokens.  MT: groups of 16 rows of a step.  STAGED: x lies in shared memory as operands (a CTA with more
// than one step), else each warp loads its columns as it goes.
template <int NT, int MT, bool STAGED>
__global__ void __launch_bounds__(kThreads) linear_w4_kernel(const LinearArgs a) {
    constexpr int kRows = 16 * MT, kRedLd = kRows + 4;                 // padded: no two lanes of a store share a bank
    constexpr int kRed = kWarps * 8 * NT * kRedLd;
    extern __shared__ __align__(16) uint8_t smem[];
    float* red = reinterpret_cast<float*>(smem);                       // [STAGED ? 2 : 1][warps][tokens][kRedLd]
    uint4* xs = reinterpret_cast<uint4*>(smem + 2 * kRed * sizeof(float));   // [column tile][word][NT][lane]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int t0 = blockIdx.y * 8 * NT;
    const int stride = gridDim.x * kRows;
    int row = blockIdx.x * kRows, c = warp;                            // the next piece
    // weights on their way to L2 while the kernel before ends (L2 is where everybody's writes meet, so nothing stale is kept)
    for (int k = warp; k < a.kt; k += kWarps) {
        const uint8_t* tile = piece_at<MT>(a, row, k) + row % kW4Tile / 8 * 512;
        for (int i = lane * 128; i < 2 * MT * 512; i += 32 * 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(tile + i));
        if (lane == 31) asm volatile("prefetch.global.L2 [%0];" ::"l"(piece_at<MT>(a, row, k) + w4_scale(row % kW4Tile, 0)));
    }
    pdl_wait();
    pdl_trigger();
    Piece<MT> next;
    if (c < a.kt) load_piece<MT>(next, a, row, c, lane);
    if constexpr (STAGED) {
        const int per = a.kt * 16;                                     // runs of eight columns of a token
        for (int i = threadIdx.x; i < per * 8 * NT; i += kThreads) {
            const int tok = i / per, k8 = i % per;
            const uint4 v = load_x8(a, t0 + tok, 8 * k8);
            xs[((k8 / 16 * 4 + k8 % 4) * NT + tok / 8) * 32 + (tok % 8) * 4 + k8 / 4 % 4] = v;
        }
        __syncthreads();
    }
    int buf = 0;
    for (int row0 = row; row0 < a.N; row0 += stride, buf ^= 1) {
        float acc[MT][NT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[m][n][i] = 0.f;
        for (int cc = warp; cc < a.kt; cc += kWarps) {
            const Piece<MT> p = next;
            c += kWarps;
            if (c >= a.kt) { c = warp; row += stride; }
            if (row < a.N) load_piece<MT>(next, a, row, c, lane);
            uint4 x[STAGED ? 1 : 4][NT];
            if constexpr (!STAGED) {
#pragma unroll
                for (int w = 0; w < 4; ++w)
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const int k = cc * kW4Tile + 32 * t + 8 * w, tok = t0 + 8 * n + g;
                        if (a.wide && (cc + 1) * kW4Tile <= a.K)
                            x[w][n] = tok < a.T ? __ldg(reinterpret_cast<const uint4*>(a.x + tok * a.ld_x + k)) : make_uint4(0u, 0u, 0u, 0u);
                        else
                            x[w][n] = load_x8(a, tok, k);
                    }
            }
            uint32_t s[2 * MT][2];
#pragma unroll
            for (int i = 0; i < 2 * MT; ++i) w4_scales(p.s[i], s[i][0], s[i][1]);
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                uint32_t f[2 * MT][4];
#pragma unroll
                for (int i = 0; i < 2 * MT; ++i) {
                    w4_values(w == 0 ? p.w[i].x : w == 1 ? p.w[i].y : w == 2 ? p.w[i].z : p.w[i].w, f[i]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) f[i][j] = bmul2(f[i][j], s[i][w / 2]);
                }
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint4 b = STAGED ? xs[((cc * 4 + w) * NT + n) * 32 + lane] : x[STAGED ? 0 : w][n];
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        mma_bf16(acc[m][n], f[2 * m][0], f[2 * m + 1][0], f[2 * m][1], f[2 * m + 1][1], b.x, b.y);
                        mma_bf16(acc[m][n], f[2 * m][2], f[2 * m + 1][2], f[2 * m][3], f[2 * m + 1][3], b.z, b.w);
                    }
                }
            }
        }
        float* mine = red + buf * kRed + warp * 8 * NT * kRedLd;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 4; ++i) mine[(8 * n + 2 * t + (i & 1)) * kRedLd + 16 * m + g + 8 * (i >> 1)] = acc[m][n][i];
        __syncthreads();                 // the other buffer is free: its readers are through before this barrier's next use
        for (int i = threadIdx.x; i < kRows * 8 * NT; i += kThreads) {
            const int tok = i / kRows, r = i % kRows;
            if (t0 + tok >= a.T || row0 + r >= a.N) continue;
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v += red[buf * kRed + (w * 8 * NT + tok) * kRedLd + r];
            store_y(a, t0 + tok, row0 + r, v);
        }
    }
}

// ---------------------------------------------------------------------------
// Packing: a warp for each row (of the padded ones too, whose tiles are zero).  5120 x 2048 take 25 us in bf16 and 45 in fp32
// (4 and 7 us of bytes): a lane's columns lie 32 apart from the next one's.  It runs once a weight.
// ---------------------------------------------------------------------------
template <typename W>
__device__ __forceinline__ float load_w(const W* w, int k, int K) {
    return k < K ? static_cast<float>(w[k]) : 0.f;
}
__device__ __forceinline__ bool finite(float v) { return v - v == 0.f; }

template <typename W>
__global__ void __launch_bounds__(kThreads) w4_pack_kernel(const W* w, long long ld, int N, int K, uint8_t* tiles, float* row_scale, moe_dev_status* st) {
    const int row = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const int kt = (K + kW4Tile - 1) / kW4Tile, rows = (N + kW4Tile - 1) / kW4Tile * kW4Tile;
    pdl_wait();
    pdl_trigger();
    if (row >= rows) return;
    const bool live = row < N;
    const W* p = w + row * ld;
    float top = 0.f;
    bool bad = false;
    if (live)
        for (int k = lane; k < K; k += 32) {
            const float v = load_w(p, k, K);
            if (finite(v)) top = fmaxf(top, fabsf(v));
            else bad = true;
        }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
    if (__any_sync(kFull, bad) && lane == 0) report(st, MOE_DEV_NONFINITE, row);
    float hs = __fmul_rn(top, 1.f / 2688.f);
    if (!(hs >= 0x1p-100f)) hs = 1.f;
    const float inv = __fdiv_rn(1.f, hs);
    if (live && lane == 0) row_scale[row] = hs;
    for (int run = lane; run < kt * 4; run += 32) {                    // runs of 32 columns
        uint8_t* tile = tiles + (static_cast<long long>(row / kW4Tile) * kt + run / 4) * kW4Bytes;
        const int r = row % kW4Tile, c = run % 4;
        uint32_t words[4] = {0u, 0u, 0u, 0u}, scales = 0u;
        if (live)
#pragma unroll 1
            for (int b = 0; b < 2; ++b) {
                float z[16], most = 0.f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float v = load_w(p, run * 32 + b * 16 + i, K);
                    z[i] = finite(v) ? __fmul_rn(v, inv) : 0.f;
                    most = fmaxf(most, fabsf(z[i]));
                }
                const uint32_t s = f32_to_e4m3(__fmul_rn(most, 1.f / 6.f));
                const float sv = e4m3_to_f32(s), up = sv > 0.f ? __fdiv_rn(1.f, sv) : 0.f;
                scales |= s << (8 * b);
#pragma unroll
                for (int i = 0; i < 16; i += 2) {
                    const uint32_t two = f32_to_e2m1x2(__fmul_rn(z[i], up), __fmul_rn(z[i + 1], up));
                    const int j = i % 8 / 2;
                    const uint32_t bits = w4_half_bits(two & 15u, j) | w4_half_bits(two >> 4 & 15u, j) << 16;
                    words[2 * b + i / 8] |= bits;
                }
            }
        *reinterpret_cast<uint4*>(tile + w4_run(r, c)) = make_uint4(words[0], words[1], words[2], words[3]);
        *reinterpret_cast<uint16_t*>(tile + w4_scale(r, 2 * c)) = static_cast<uint16_t>(scales);
    }
}

template <int NT, int MT, bool STAGED>
cudaError_t launch_few(const LinearArgs& a, int sms, cudaStream_t s) {
    constexpr int rows = 16 * MT;
    constexpr int red = kWarps * 8 * NT * (rows + 4) * sizeof(float);
    const size_t smem = 2 * red + (STAGED ? static_cast<size_t>(a.kt) * kW4Tile * 16 * NT : 0);
    // (a call of some 0.3 us that a short product can do without; it sets the most that there is, so that threads do not undo each
    // other's setting)
    if (smem > 48 * 1024) {
        constexpr int room = 2 * red + (STAGED ? kMaxStaged : 0);
        const cudaError_t e = cudaFuncSetAttribute(linear_w4_kernel<NT, MT, STAGED>, cudaFuncAttributeMaxDynamicSharedMemorySize, room);
        if (e != cudaSuccess) return e;
    }
    const int steps = (a.N + rows - 1) / rows, fit = static_cast<int>((227 * 1024) / (smem + 1024));
    const int most = STAGED ? (fit < 3 ? fit : 3) * sms : steps;
    return launch_pdl(linear_w4_kernel<NT, MT, STAGED>, dim3(steps < most ? steps : most, (a.T + 8 * NT - 1) / (8 * NT)), dim3(kThreads), smem, s, a);
}

template <int NT>
cudaError_t launch_few(const LinearArgs& a, cudaStream_t s) {
    // Few rows: every CTA has one step, of 16 rows where 32 would leave SMs without any; many: persistent CTAs with x in
    // shared memory.  Through 2048 x N, 16 rows / 32 rows / persistent, 1 token: N = 2048 2.7 / 2.9 / 3.5 us, 8192 5.3 / 3.9 /
    // 6.4, 14000 7.0 / 6.4 / 6.8, 32000 14.2 / 12.1 / 11.9; 16 tokens: 3.7 / 4.3 / 7.0, 9.0 / 6.2 / 8.6, 12.9 / 11.3 / 11.5,
    // 26.4 / 18.4 / 16.8.
    const int sms = sm_count();
    if (a.N <= 16 * sms * 2) return launch_few<NT, 1, false>(a, sms, s);
    // (more than 16 tokens through that many rows go to the kernel for many)
    if constexpr (NT < 4)
        if (a.N > 32 * sms * 3 && static_cast<size_t>(a.kt) * kW4Tile * 16 * NT <= kMaxStaged) return launch_few<NT, 2, true>(a, sms, s);
    return launch_few<NT, 2, false>(a, sms, s);
}

}  // namespace

// Clocks that the kernel for few tokens should take, for 9 to 64 of them.  (Both sides, few / many: through 2048 x 2048 16
// tokens 3.7 / 6.2 us, 32 5.1 / 6.8, 48 8.6 / 7.4, 64 9.6 / 8.1; 8192 x 2048: 9.6 / 10.3, 15.2 / 10.9, 25.6 / 11.5, 29.5 / 12.2; 2048 x
// 5120: 6.0 / 7.5, 11.4 / 8.2, 15.6 / 8.8, 17.0 / 9.3; 2048 x 32000: 16.9 / 13.9, 28.4 / 14.2, 51 / 14.6, 55 / 15.0.  Rows of x that
// start anywhere, where the choice is the same: 32 tokens, 4096 x 2048 25.5 / 10.1; 15 tokens, 5391 x 26969 68 / 52.)
static double few_clocks(const LinearArgs& a) {
    const double rows = a.N * 1e-3 * a.kt;
    return 1000.0 + rows * (a.T <= 16 ? 53.0 : a.T <= 32 ? 142.0 : 285.0);
}

cudaError_t launch_linear_w4(const void* x, long long ld_x, int T, const moe_w4& w, const float* bias, void* y, int y_dtype, long long ld_y,
                             bool add, moe_dev_status* st, cudaStream_t s) {
    LinearArgs a;
    a.st = st;
    a.tiles = static_cast<const uint8_t*>(w.tiles);
    a.row_scale = w.row_scale;
    a.x = static_cast<const __nv_bfloat16*>(x);
    a.ld_x = ld_x;
    a.ld_y = ld_y;
    a.T = T;
    a.N = w.N;
    a.K = w.K;
    a.kt = (w.K + kW4Tile - 1) / kW4Tile;
    a.bias = bias;
    a.y = y;
    a.y_bf16 = y_dtype == MOE_DTYPE_BF16;
    a.add = add;
    a.wide = (reinterpret_cast<uintptr_t>(x) & 15u) == 0 && ld_x % 8 == 0;
    if (T > 8) {
        const LinearTile t = linear_w4_tile(a);
        if (T > 64 || t.clocks < few_clocks(a)) return launch_linear_w4_tc(a, t, s);
    }
    if (T <= 8) return launch_few<1>(a, s);
    return T <= 16 ? launch_few<2>(a, s) : launch_few<4>(a, s);
}

cudaError_t launch_w4_pack(const void* w, int dtype, long long ld, int N, int K, void* tiles, float* row_scale, moe_dev_status* st, cudaStream_t s) {
    const dim3 grid((N + kW4Tile - 1) / kW4Tile * (kW4Tile / kWarps));
    if (dtype == MOE_DTYPE_BF16)
        return launch_pdl(w4_pack_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, s, static_cast<const __nv_bfloat16*>(w), ld, N, K, static_cast<uint8_t*>(tiles), row_scale, st);
    return launch_pdl(w4_pack_kernel<float>, grid, dim3(kThreads), 0, s, static_cast<const float*>(w), ld, N, K, static_cast<uint8_t*>(tiles), row_scale, st);
}

}  // namespace moe
