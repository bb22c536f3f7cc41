// qk_rope.cu -- norms of q and k for each head, rotary positions, and the
// append of k and v to the 4-bit cache, in one pass over the projection's
// rows; and the reverse, cached tokens as values.
//
// Per number of a query or key head: y = x * inv * w with inv = 1/sqrt(mean
// x^2 + eps) of its head, then the rotation of its pair.  The pass has to
// read the rows once and write q once (the cache takes 4.5 bits a number), so
// device memory bounds it for prompts and the chain of loads (row, position,
// table) for single tokens.
//
// D/8 threads hold one head's row, eight numbers each: the four pairs
// 4j..4j+3, i.e. two runs of four numbers (pairs i, i + rot/2) or one run of
// eight (pairs of neighbours).  Both members of a pair are then in one
// thread, and a block of 16 numbers that shares a scale is in two or four
// neighbouring threads.  A thread keeps its position's four (cos, sin) in registers for
// all heads of its token that it takes: the table is read once per thread
// and not once per head.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kv4.cuh"
#include "launch.h"

namespace moe {

namespace {

constexpr int kRopeThreads = 128;
constexpr float kSixth = 0x1.555556p-3f;   // 1/6, nearest fp32

template <typename XT>
struct Row8;   // eight numbers as loaded, in two runs of four
template <>
struct Row8<__nv_bfloat16> {
    uint2 a, b;
    __device__ void load(const __nv_bfloat16* p, int i, int k) {
        a = *reinterpret_cast<const uint2*>(p + i);
        b = *reinterpret_cast<const uint2*>(p + k);
    }
    __device__ void get(float (&x)[8]) const {
        const uint32_t u[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = __uint_as_float(u[j] << 16);
            x[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
        }
    }
};
template <>
struct Row8<float> {
    float4 a, b;
    __device__ void load(const float* p, int i, int k) {
        a = *reinterpret_cast<const float4*>(p + i);
        b = *reinterpret_cast<const float4*>(p + k);
    }
    __device__ void get(float (&x)[8]) const {
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
};

__device__ __forceinline__ void store4(float* p, const float* y) {
    *reinterpret_cast<float4*>(p) = make_float4(y[0], y[1], y[2], y[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float* y) {
    const __nv_bfloat162 l = __floats2bfloat162_rn(y[0], y[1]), h = __floats2bfloat162_rn(y[2], y[3]);
    uint2 v;
    memcpy(&v.x, &l, 4);
    memcpy(&v.y, &h, 4);
    *reinterpret_cast<uint2*>(p) = v;
}

// hi + lo += v, exactly but for lo's own rounding (Knuth's two-sum).
__device__ __forceinline__ void two_add(float& hi, float& lo, float v) {
    const float s = __fadd_rn(hi, v);
    const float t = __fsub_rn(s, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, t)), __fsub_rn(v, t)));
    hi = s;
}

// Sum of the squares of a head's row over its G threads.  `exact` (keys that
// are cached) carries it in two words: a key's code then depends on the sum's
// nearest fp32 and not on the order of its terms.
template <int G>
__device__ __forceinline__ float row_squares(const float (&x)[8], bool exact) {
    float hi = 0.f, lo = 0.f;
    if (!exact) {
#pragma unroll
        for (int j = 0; j < 8; ++j) hi = fmaf(x[j], x[j], hi);
#pragma unroll
        for (int off = G / 2; off >= 1; off >>= 1) hi += __shfl_xor_sync(kFull, hi, off);
        return hi;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float p = __fmul_rn(x[j], x[j]);
        lo = __fadd_rn(lo, __fmaf_rn(x[j], x[j], -p));
        two_add(hi, lo, p);
    }
#pragma unroll
    for (int off = G / 2; off >= 1; off >>= 1) {
        const float h = __shfl_xor_sync(kFull, hi, off), l = __shfl_xor_sync(kFull, lo, off);
        lo = __fadd_rn(lo, l);
        two_add(hi, lo, h);
    }
    return __fadd_rn(hi, lo);
}

// The scale byte of a block with largest magnitude `top`, and 1 / scale (0 for scale 0).
__device__ __forceinline__ uint32_t block_scale(float top, float& r) {
    const uint32_t b = f32_to_e4m3(fminf(__fmul_rn(top, kSixth), 448.f));
    const float s = e4m3_to_f32(b);
    r = s > 0.f ? __frcp_rn(s) : 0.f;
    return b;
}

__device__ __forceinline__ float finite_or_zero(float z, bool& bad) {
    if (isfinite(z)) return z;
    bad = true;
    return 0.f;
}

struct RopeArgs {
    const void* qkv;
    long long ld;
    int T, n_q, n_kv;
    const float* q_w;
    const float* k_w;
    float eps;
    const float2* table;
    const int32_t* positions;
    const uint8_t* axis;
    int n_pos, rot, axes, pairs;
    void* q_out;
    long long ld_q;
    void* k_out;
    long long ld_k;
    moe_kv4_cache c;
    const int32_t* q_start;
    int rows;   // heads that a CTA takes of its token
    moe_dev_status* st;
};

// One CTA: `rows` heads of one token (blockIdx.x), from blockIdx.y * rows on.
// MAXR rows a thread group are loaded before the first is used.
template <typename XT, int D, int MAXR>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(const RopeArgs a) {
    constexpr int G = D / 8;                    // threads of a row
    constexpr int NG = kRopeThreads / G;        // rows at a time
    using L = Kv4Layout<D>;
    pdl_wait();
    pdl_trigger();
    const int t = blockIdx.x;
    const int grp = threadIdx.x / G, j = threadIdx.x % G;
    const int n_rows = a.n_q + 2 * a.n_kv;
    const int h0 = blockIdx.y * a.rows;
    const int h1 = min(h0 + a.rows, a.c.pages != nullptr ? n_rows : a.n_q + a.n_kv);
    const XT* x_row = static_cast<const XT*>(a.qkv) + static_cast<long long>(t) * a.ld;

    // the thread's two runs of four numbers in a rotated head
    int ia, ib;
    bool turn = false;
    if (a.pairs || a.rot == 0) {
        ia = 8 * j;
        ib = ia + 4;
        turn = ia < a.rot;
    } else if (4 * j < a.rot / 2) {
        ia = 4 * j;
        ib = ia + a.rot / 2;
        turn = true;
    } else {                                    // numbers that pass through, in the same two halves
        ia = a.rot + 4 * j - a.rot / 2;
        ib = ia + (D - a.rot) / 2;
    }

    Row8<XT> raw[MAXR];
    auto load_rows = [&](int first) {
#pragma unroll
        for (int r = 0; r < MAXR; ++r) {
            const int h = first + r * NG + grp;
            if (h >= h1) break;
            const bool val = h >= a.n_q + a.n_kv;
            raw[r].load(x_row + static_cast<long long>(h) * D, val ? 8 * j : ia, val ? 8 * j + 4 : ib);
        }
    };
    load_rows(h0);

    // the token's place in the cache, and its page
    int seq = -1, place = -1, first_new = 0;
    const bool with_cache = a.c.pages != nullptr;
    if (with_cache) {
        seq = find_seq(a.q_start, a.c.S, t);
        if (seq >= 0) {
            const int q0 = a.q_start[seq];
            const int n = a.q_start[seq + 1] - q0;
            first_new = a.c.seq_len[seq] - n;
            place = first_new + (t - q0);
        }
    }
    int page = -1;
    if (place >= 0) {
        const int col = place / kPage;
        page = col < a.c.max_pages ? a.c.page_table[static_cast<long long>(seq) * a.c.max_pages + col] : -1;
        if (page < 0 || page >= a.c.n_pages) {
            if (threadIdx.x == 0) report(a.st, MOE_DEV_BAD_INDEX, page);
            page = -1;
        }
    }
    uint8_t* page_base = nullptr;
    if (page >= 0) page_base = static_cast<uint8_t*>(a.c.pages) + static_cast<long long>(page) * a.c.n_kv * L::bytes;

    // (cos, sin) of the thread's four pairs
    float2 cs[4];
    if (turn) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int f = 4 * j + i;
            int p = place;
            if (a.positions != nullptr) {
                const int ax = a.axis != nullptr ? a.axis[f] : 0;
                if (ax < a.axes) p = a.positions[static_cast<long long>(ax) * a.T + t];
                else p = -1;
            } else if (p < 0) {
                p = 0;                          // a row of a padded batch: not appended
            }
            if (p < 0 || p >= a.n_pos) {
                report(a.st, MOE_DEV_BAD_INDEX, p);
                p = 0;
            }
            cs[i] = a.table[static_cast<long long>(p) * (a.rot / 2) + f];
        }
    }

    for (int first = h0; first < h1; first += MAXR * NG) {
        if (first != h0) load_rows(first);
#pragma unroll
        for (int r = 0; r < MAXR; ++r) {
            const int h = first + r * NG + grp;
            // whole warps leave together: the shuffles below want every lane
            if (first + r * NG + (static_cast<int>(threadIdx.x) & ~31) / G >= h1) break;
            const bool live = h < h1;
            const bool is_k = live && h >= a.n_q && h < a.n_q + a.n_kv, is_v = live && h >= a.n_q + a.n_kv;
            float y[8];
            if (live) raw[r].get(y);
            else {
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] = 0.f;
            }
            const float* w = h < a.n_q ? a.q_w : a.k_w;
            // keys that are cached take the two-word sum; a warp's rows may be of both kinds
            const bool any_k = __any_sync(kFull, is_k && with_cache);
            const float ss = row_squares<G>(y, any_k);
            if (live && !is_v) {
                if (w != nullptr) {
                    const float inv = __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(ss, 1.0f / D), a.eps)));
                    const float4 wa = *reinterpret_cast<const float4*>(w + ia), wb = *reinterpret_cast<const float4*>(w + ib);
                    const float wv[8] = {wa.x, wa.y, wa.z, wa.w, wb.x, wb.y, wb.z, wb.w};
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = __fmul_rn(__fmul_rn(y[i], inv), wv[i]);
                }
                if (turn) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int pa = a.pairs ? 2 * i : i, pb = a.pairs ? 2 * i + 1 : i + 4;
                        const float u = y[pa], v = y[pb];
                        y[pa] = __fsub_rn(__fmul_rn(u, cs[i].x), __fmul_rn(v, cs[i].y));
                        y[pb] = __fadd_rn(__fmul_rn(v, cs[i].x), __fmul_rn(u, cs[i].y));
                    }
                }
                XT* out = nullptr;
                if (h < a.n_q) out = static_cast<XT*>(a.q_out) + static_cast<long long>(t) * a.ld_q + static_cast<long long>(h) * D;
                else if (a.k_out != nullptr)
                    out = static_cast<XT*>(a.k_out) + static_cast<long long>(t) * a.ld_k + static_cast<long long>(h - a.n_q) * D;
                if (out != nullptr) {
                    store4(out + ia, y);
                    store4(out + ib, y + 4);
                }
            }
            if (!__any_sync(kFull, (is_k || is_v) && page_base != nullptr)) continue;
            // quantise: keys alone, values with the other token of their pair
            const int kv = h - a.n_q - (is_v ? a.n_kv : 0);
            bool bad = false;
            float inv_h = 1.f;
            if (is_k || is_v) {
                const float* hs = is_k ? a.c.k_scale : a.c.v_scale;
                if (hs != nullptr) inv_h = __frcp_rn(hs[kv]);
            }
            float top_a = 0.f, top_b = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                y[i] = finite_or_zero(__fmul_rn(y[i], inv_h), bad);
                float& top = i < 4 ? top_a : top_b;
                top = fmaxf(top, fabsf(y[i]));
            }
            // a block of 16: the runs of four threads (halves), or both runs of two threads
            const bool whole = a.pairs || a.rot == 0 || is_v;
            float ta = whole ? fmaxf(top_a, top_b) : top_a, tb = whole ? ta : top_b;
            ta = fmaxf(ta, __shfl_xor_sync(kFull, ta, 1));
            tb = fmaxf(tb, __shfl_xor_sync(kFull, tb, 1));
            {
                const float oa = __shfl_xor_sync(kFull, ta, 2), ob = __shfl_xor_sync(kFull, tb, 2);
                if (!whole) {
                    ta = fmaxf(ta, oa);
                    tb = fmaxf(tb, ob);
                }
            }
            float ra, rb;
            const uint32_t sa = block_scale(ta, ra), sb = block_scale(tb, rb);
            if (is_k && page_base != nullptr) {
                uint8_t* base = page_base + static_cast<long long>(kv) * L::bytes;
                const int tok = place % kPage;
                const uint32_t c0 = f32_to_e2m1x2(__fmul_rn(y[0], ra), __fmul_rn(y[1], ra)) |
                                    (f32_to_e2m1x2(__fmul_rn(y[2], ra), __fmul_rn(y[3], ra)) << 8);
                const uint32_t c1 = f32_to_e2m1x2(__fmul_rn(y[4], rb), __fmul_rn(y[5], rb)) |
                                    (f32_to_e2m1x2(__fmul_rn(y[6], rb), __fmul_rn(y[7], rb)) << 8);
                *reinterpret_cast<uint16_t*>(base + L::k_code(tok, ia)) = static_cast<uint16_t>(c0);
                *reinterpret_cast<uint16_t*>(base + L::k_code(tok, ib)) = static_cast<uint16_t>(c1);
                if (whole) {
                    if ((j & 1) == 0) base[L::k_scale(tok, ia / 16)] = static_cast<uint8_t>(sa);
                } else if ((j & 3) == 0) {
                    base[L::k_scale(tok, ia / 16)] = static_cast<uint8_t>(sa);
                    base[L::k_scale(tok, ib / 16)] = static_cast<uint8_t>(sb);
                }
            }
            if (bad && page_base != nullptr && (is_k || is_v)) report(a.st, MOE_DEV_NONFINITE, t);
            if (!__any_sync(kFull, is_v)) continue;
            // Codes of two neighbouring tokens share a byte.  The even token's row also writes
            // the odd one's if that is new too; an odd token whose partner is
            // older puts its half beside the codes that are there.
            const int n_new_end = with_cache && seq >= 0 ? a.c.seq_len[seq] : 0;
            const bool odd = place & 1;
            const bool partner = is_v && page_base != nullptr && !odd && place + 1 < n_new_end && t + 1 < a.T;
            const bool skip = odd && place - 1 >= first_new && place - 1 >= 0;
            float z[8];
            bool bad2 = false;
            float top2 = 0.f;
#pragma unroll
            for (int i = 0; i < 8; ++i) z[i] = 0.f;
            if (partner) {
                Row8<XT> o;
                o.load(x_row + a.ld + static_cast<long long>(h) * D, 8 * j, 8 * j + 4);
                o.get(z);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    z[i] = finite_or_zero(__fmul_rn(z[i], inv_h), bad2);
                    top2 = fmaxf(top2, fabsf(z[i]));
                }
            }
            top2 = fmaxf(top2, __shfl_xor_sync(kFull, top2, 1));
            if (is_v && page_base != nullptr && !skip) {
                float rz;
                const uint32_t sz = block_scale(top2, rz);
                uint8_t* base = page_base + static_cast<long long>(kv) * L::bytes;
                const int tok = place % kPage, pj = tok / 2;
                uint2* codes = reinterpret_cast<uint2*>(base + L::v_code(pj, 8 * j));
                uint32_t c[2] = {0u, 0u};
                if (odd) {
                    const uint2 old = *codes;
                    c[0] = old.x & 0x0f0f0f0fu;
                    c[1] = old.y & 0x0f0f0f0fu;
#pragma unroll
                    for (int i = 0; i < 8; ++i) c[i / 4] |= f32_to_e2m1x2(0.f, __fmul_rn(y[i], ra)) << (8 * (i % 4));
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        c[i / 4] |= f32_to_e2m1x2(__fmul_rn(y[i], ra), __fmul_rn(z[i], rz)) << (8 * (i % 4));
                }
                *codes = make_uint2(c[0], c[1]);
                if ((j & 1) == 0) {
                    uint8_t* s = base + L::v_scale(pj, j / 2);
                    if (partner) *reinterpret_cast<uint16_t*>(s) = static_cast<uint16_t>(sa | (sz << 8));
                    else s[odd] = static_cast<uint8_t>(sa);
                }
                if (bad2) report(a.st, MOE_DEV_NONFINITE, t + 1);
            }
        }
    }
}

// One CTA: one row of moe_kv4_read; D/8 threads hold eight numbers of a key
// or value head.
template <int D>
__global__ void __launch_bounds__(kRopeThreads) kv4_read_kernel(const moe_kv4_cache c, const int32_t* q_start,
                                                                __nv_bfloat16* k_out, __nv_bfloat16* v_out,
                                                                moe_dev_status* st) {
    constexpr int G = D / 8;
    using L = Kv4Layout<D>;
    pdl_wait();
    pdl_trigger();
    const int t = blockIdx.x;
    const int j = threadIdx.x % G;
    const int seq = find_seq(q_start, c.S, t);
    int place = -1, page = -1;
    if (seq >= 0) place = c.seq_len[seq] - q_start[seq + 1] + t;
    if (place >= 0) {
        const int col = place / kPage;
        page = col < c.max_pages ? c.page_table[static_cast<long long>(seq) * c.max_pages + col] : -1;
        if (page < 0 || page >= c.n_pages) {
            if (threadIdx.x == 0) report(st, MOE_DEV_BAD_INDEX, page);
            page = -1;
        }
    }
    const int tok = place >= 0 ? place % kPage : 0;
    for (int r = blockIdx.y * (kRopeThreads / G) + threadIdx.x / G; r < 2 * c.n_kv; r += gridDim.y * (kRopeThreads / G)) {
        const bool is_v = r >= c.n_kv;
        const int kv = is_v ? r - c.n_kv : r;
        __nv_bfloat16* out = is_v ? v_out : k_out;
        if (out == nullptr) continue;
        float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (page >= 0) {
            const uint8_t* base = static_cast<const uint8_t*>(c.pages) + (static_cast<long long>(page) * c.n_kv + kv) * L::bytes;
            const float* hs = is_v ? c.v_scale : c.k_scale;
            const float h = hs != nullptr ? hs[kv] : 1.f;
            uint32_t f[4], w, sb;
            if (is_v) {
                const uint2 two = *reinterpret_cast<const uint2*>(base + L::v_code(tok / 2, 8 * j));
                const int sh = 4 * (tok & 1);
                const uint32_t lo = (two.x >> sh) & 0x0f0f0f0fu, hi = (two.y >> sh) & 0x0f0f0f0fu;
                // bytes of single codes -> eight codes in a word
                auto squeeze = [](uint32_t u) {
                    u |= u >> 4;
                    return (u & 0xffu) | ((u >> 8) & 0xff00u);
                };
                w = squeeze(lo) | (squeeze(hi) << 16);
                sb = base[L::v_scale(tok / 2, j / 2) + (tok & 1)];
            } else {
                w = *reinterpret_cast<const uint32_t*>(base + L::k_code(tok, 8 * j));
                sb = base[L::k_scale(tok, j / 2)];
            }
            e2m1x8_to_f16(w, f[0], f[1], f[2], f[3]);
            const float s = e4m3_to_f32(sb);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                __half2 p;
                memcpy(&p, &f[i], 4);
                const float2 v = __half22float2(p);
                y[2 * i] = __fmul_rn(__fmul_rn(v.x, s), h);
                y[2 * i + 1] = __fmul_rn(__fmul_rn(v.y, s), h);
            }
        }
        __nv_bfloat16* o = out + (static_cast<long long>(t) * c.n_kv + kv) * D + 8 * j;
        store4(o, y);
        store4(o + 4, y + 4);
    }
}

}  // namespace

template <typename XT, int D>
static cudaError_t launch_rope_t(RopeArgs& a, cudaStream_t s) {
    constexpr int NG = kRopeThreads / (D / 8);
    const int heads = a.c.pages != nullptr ? a.n_q + 2 * a.n_kv : a.n_q + a.n_kv;
    // Few tokens: a head for each thread group, so that the heads' loads and
    // reductions run side by side on many SMs.  Many tokens: a CTA takes up
    // to six heads a group, and the table and position are read once for them.
    const bool few = static_cast<long long>(a.T) * heads < 32768;
    constexpr int kMany = sizeof(XT) == 2 ? 6 : 3;
    a.rows = few ? NG : heads;
    const dim3 grid(a.T, (heads + a.rows - 1) / a.rows);
    if (few) return launch_pdl(qk_norm_rope_kernel<XT, D, 1>, grid, dim3(kRopeThreads), 0, s, a);
    return launch_pdl(qk_norm_rope_kernel<XT, D, kMany>, grid, dim3(kRopeThreads), 0, s, a);
}

cudaError_t launch_qk_norm_rope(const void* qkv, int dtype, long long ld, int T, int n_q, int n_kv, int D,
                                const float* q_w, const float* k_w, float eps, const moe_rope_params* rope,
                                void* q_out, long long ld_q, void* k_out, long long ld_k,
                                const moe_kv4_cache* cache, const int32_t* q_start, moe_dev_status* st,
                                cudaStream_t s) {
    RopeArgs a = {};
    a.qkv = qkv; a.ld = ld; a.T = T; a.n_q = n_q; a.n_kv = n_kv;
    a.q_w = q_w; a.k_w = k_w; a.eps = eps;
    if (rope != nullptr) {
        a.table = reinterpret_cast<const float2*>(rope->table);
        a.positions = rope->positions; a.axis = rope->axis;
        a.n_pos = rope->n_pos; a.rot = rope->rot; a.axes = rope->axes; a.pairs = rope->pairs;
    }
    a.q_out = q_out; a.ld_q = ld_q; a.k_out = k_out; a.ld_k = ld_k;
    if (cache != nullptr) { a.c = *cache; a.q_start = q_start; }
    a.st = st;
    if (dtype == MOE_DTYPE_BF16) return D == 128 ? launch_rope_t<__nv_bfloat16, 128>(a, s) : launch_rope_t<__nv_bfloat16, 64>(a, s);
    return D == 128 ? launch_rope_t<float, 128>(a, s) : launch_rope_t<float, 64>(a, s);
}

cudaError_t launch_kv4_read(const moe_kv4_cache& c, const int32_t* q_start, int T, void* k_out, void* v_out,
                            moe_dev_status* st, cudaStream_t s) {
    const int ng = kRopeThreads / (c.head_dim / 8);
    const dim3 grid(T, (2 * c.n_kv + ng - 1) / ng);
    auto* k = static_cast<__nv_bfloat16*>(k_out);
    auto* v = static_cast<__nv_bfloat16*>(v_out);
    if (c.head_dim == 128) return launch_pdl(kv4_read_kernel<128>, grid, dim3(kRopeThreads), 0, s, c, q_start, k, v, st);
    return launch_pdl(kv4_read_kernel<64>, grid, dim3(kRopeThreads), 0, s, c, q_start, k, v, st);
}

}  // namespace moe
