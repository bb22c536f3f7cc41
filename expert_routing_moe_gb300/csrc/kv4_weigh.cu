// kv4_weigh.cu -- the attention weight that cached tokens draw (moe_kv4_weigh):
//     score[j] += sum over rows i and heads h of exp(scale * q_i . k_j - lse[i][h])
//
// A CTA takes a page of a sequence; its warps share the key heads and the
// groups of eight query rows.  Scores come from m16n8k16 products with the cached keys as the
// 16-row operand, as in the attention over few rows; a lane adds up the
// probabilities of its eight tokens over all rows that it sees, so that only one
// sum a token is left to add across lanes and warps, in a fixed order.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kv4_weigh.cuh"
#include "launch.h"
#include "tmap.h"

namespace moe {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Eight query rows as fragments: row g of them, numbers (D/4) t + 4 ks + 0..3, scaled by a power of two that puts the
// row's largest magnitude into [2^10, 2^11).
template <int D>
struct Queries {
    uint32_t f[D / 16][2];
    float up, z;                 // the scores' factor and the row's log-sum-exp, in powers of two; of row g
};
template <int D>
__device__ __forceinline__ void load_rows(Queries<D>& w, const WeighArgs& a, const WeighSeq& s, int h, int r0, int lane, float k_scale) {
    const int g = lane >> 2, t = lane & 3, r = r0 + g;
    const bool live = r < s.n * a.group;
    uint32_t raw[D / 8];
#pragma unroll
    for (int i = 0; i < D / 8; ++i) raw[i] = 0u;
    float lse = -INFINITY;
    if (live) {
        const long long row = s.q0 + r / a.group;
        const int head = h * a.group + r % a.group;
        const __nv_bfloat16* p = a.q + row * a.ld_q + static_cast<long long>(head) * D + (D / 4) * t;
        lse = a.lse[row * a.n_q + head];
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
    int e = static_cast<int>(__float_as_uint(top) >> 23) - 127;
    e = (top > 0.f && e < 128) ? max(-100, min(100, 10 - e)) : 0;
    const float up = __int_as_float((e + 127) << 23);
    // a row that sees nothing, or is none: 2^-inf of whatever the products are
    const bool none = !live || lse == -INFINITY;
    w.up = none ? 0.f : a.scale * kLog2e * k_scale * __int_as_float((127 - e) << 23);
    w.z = none ? INFINITY : lse * kLog2e;
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
        w.f[i / 2][i & 1] = none ? 0u : pack_f16(__uint_as_float(raw[i] << 16) * up, __uint_as_float(raw[i] & 0xffff0000u) * up);
}

template <int D>
__global__ void __launch_bounds__(kThreads) kv4_weigh_kernel(const WeighArgs a) {
    using L = Kv4Layout<D>;
    constexpr int W = D / 32;
    __shared__ float s_sum[kWarps][kPage];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    pdl_wait();
    pdl_trigger();
    for (int s = blockIdx.y; s < a.c.S; s += gridDim.y) {
        const WeighSeq q = weigh_seq(a, s);
        if (!q.fit && blockIdx.x == 0 && threadIdx.x == 0) report(a.st, MOE_DEV_BAD_INDEX, s);
        if (q.n == 0 || q.len == 0 || (q.n - q.i0) * a.group >= a.many) continue;
        const int lo = weigh_first(a, q);
        for (int page = lo / kPage + blockIdx.x; page < pages_of(q.len); page += gridDim.x) {
            const int id = a.c.page_table[static_cast<long long>(s) * a.c.max_pages + page];
            const bool ok = id >= 0 && id < a.c.n_pages;
            if (!ok) {
                if (threadIdx.x == 0) report(a.st, MOE_DEV_BAD_INDEX, id);
                continue;
            }
            const int key0 = page * kPage;
            int ia, ib;
            weigh_rows(a, q, key0, kPage, ia, ib);
            const int r_begin = ia * a.group, r_end = ib * a.group;
            const int tiles = (r_end - r_begin + 7) / 8;
            float sum[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) sum[i] = 0.f;
            for (int item = warp; item < tiles * a.c.n_kv; item += kWarps) {
                const int h = item / tiles, r0 = r_begin + item % tiles * 8;
                const uint8_t* base = static_cast<const uint8_t*>(a.c.pages) + (static_cast<long long>(id) * a.c.n_kv + h) * L::bytes;
                Queries<D> w;
                load_rows<D>(w, a, q, h, r0, lane, a.c.k_scale != nullptr ? a.c.k_scale[h] : 1.f);
                float up[2], z[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    up[c] = __shfl_sync(kFull, w.up, (2 * t + c) * 4);
                    z[c] = __shfl_sync(kFull, w.z, (2 * t + c) * 4);
                }
                float acc[4][4];
#pragma unroll
                for (int m = 0; m < 4; ++m)
#pragma unroll
                    for (int c = 0; c < 4; ++c) acc[m][c] = 0.f;
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    uint32_t c0[W], c1[W];
                    memcpy(c0, __builtin_assume_aligned(base + (16 * m + g) * (D / 2) + t * (D / 8), D / 8), D / 8);
                    memcpy(c1, __builtin_assume_aligned(base + (16 * m + 8 + g) * (D / 2) + t * (D / 8), D / 8), D / 8);
                    // scales of tokens 16 m + g, 16 m + 8 + g: R bytes each, side by side
                    uint32_t s0[L::R], s1[L::R];
                    const uint8_t* sp = base + L::kScales + ((t * 8 + g) * 8 + 2 * m) * L::R;
                    if constexpr (L::R == 2) {
                        const uint32_t two = *reinterpret_cast<const uint32_t*>(sp);
                        const uint32_t x = e4m3x2_to_f16(two & 0xffffu), y = e4m3x2_to_f16(two >> 16);
                        s0[0] = __byte_perm(x, 0, 0x1010); s0[1] = __byte_perm(x, 0, 0x3232);
                        s1[0] = __byte_perm(y, 0, 0x1010); s1[1] = __byte_perm(y, 0, 0x3232);
                    } else {
                        const uint32_t x = e4m3x2_to_f16(*reinterpret_cast<const uint16_t*>(sp));
                        s0[0] = __byte_perm(x, 0, 0x1010);
                        s1[0] = __byte_perm(x, 0, 0x3232);
                    }
#pragma unroll
                    for (int k2 = 0; k2 < W; ++k2) {
                        uint32_t x[4], y[4];
                        e2m1x8_to_f16(c0[k2], x[0], x[1], x[2], x[3]);
                        e2m1x8_to_f16(c1[k2], y[0], y[1], y[2], y[3]);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int k = 2 * k2 + e, r = k / 4;
                            const uint32_t af[4] = {hmul2_u(x[2 * e], s0[r]), hmul2_u(y[2 * e], s1[r]), hmul2_u(x[2 * e + 1], s0[r]),
                                                    hmul2_u(y[2 * e + 1], s1[r])};
                            mma_f16(acc[m], af, w.f[k][0], w.f[k][1]);
                        }
                    }
                }
                // places of the tile's rows: token 8 i + g is seen from its own place on, as far as the window goes
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int r = r0 + 2 * t + c;
                    const int p = q.len - q.n + r / a.group;
                    const bool live = r < r_end;
                    const int last = live ? min(p, q.len - 1) : -1, first = a.window > 0 ? p - a.window + 1 : 0;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int key = key0 + 8 * i + g;
                        const float x = ex2(fmaf(acc[i >> 1][2 * (i & 1) + c], up[c], -z[c]));
                        sum[i] += key <= last && key >= first ? x : 0.f;
                    }
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                sum[i] += __shfl_xor_sync(kFull, sum[i], 1);
                sum[i] += __shfl_xor_sync(kFull, sum[i], 2);
                if (t == 0) s_sum[warp][8 * i + g] = sum[i];
            }
            __syncthreads();
            if (threadIdx.x < kPage && key0 + static_cast<int>(threadIdx.x) < q.len) {
                float v = 0.f;
#pragma unroll
                for (int i = 0; i < kWarps; ++i) v += s_sum[i][threadIdx.x];
                weigh_add(a, q, s, key0 + threadIdx.x, v);
            }
            __syncthreads();
        }
    }
}

template <int D>
cudaError_t launch(const WeighArgs& a, cudaStream_t s) {
    const int pages = a.c.max_pages < 1024 ? a.c.max_pages : 1024, seqs = a.c.S;
    return launch_pdl(kv4_weigh_kernel<D>, dim3(pages, seqs), dim3(kThreads), 0, s, a);
}

}  // namespace

size_t kv4_weigh_workspace(int S, int T, int n_q, int n_kv, int D, int max_pages) {
    (void)D;
    const int group = n_q / n_kv;
    return static_cast<long long>(T) * group >= kWeighMany && weigh_tc_fits(group) ? kv4_weigh_tc_workspace(S, max_pages) : 0;
}

cudaError_t launch_kv4_weigh(const void* q, long long ld_q, int T, int n_q, const moe_kv4_cache& c, const int32_t* q_start, int max_new,
                             const float* lse, float scale, int window, int last, float* score, long long ld_score, bool fresh, void* ws,
                             moe_dev_status* st, cudaStream_t s) {
    if (c.max_pages < 1) return cudaSuccess;
    const int group = n_q / c.n_kv;
    long long most = max_new < T ? max_new : T;        // rows of a sequence that count
    if (last > 0 && last < most) most = last;
    const bool prompts = most * group >= kWeighMany && weigh_tc_fits(group);
    const WeighArgs a = {static_cast<const __nv_bfloat16*>(q), ld_q, T, n_q, group, c, q_start, lse, scale, window, last, score, ld_score, fresh,
                         prompts ? kWeighMany : 0x7fffffff, st};
    if (prompts) {
        const cudaError_t e = launch_kv4_weigh_tc(a, ws, s);
        if (e != cudaSuccess) return e;
    }
    return c.head_dim == 64 ? launch<64>(a, s) : launch<128>(a, s);
}

}  // namespace moe
