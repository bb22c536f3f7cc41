// qk_rope.cu -- norms of q and k for each head, rotary positions, and the
// append of k and v to the 4-bit cache, in one pass over the projection's
// rows; and the reverse, cached tokens as values.
//
// Per number of a query or key head: y = x * inv * w with inv = 1/sqrt(mean
// x^2 + eps) of its head, then the rotation of its pair.  The pass has to
// read the rows once and write q once (the cache takes 4.5 bits a number).  For
// single tokens the chain of loads (row, position, table) bounds it.  For 8192
// tokens of 32 + 4 heads without a cache it moves 151 MB in 30.2 us (5.0 TB/s, 0.75
// of a copy's rate); with the cache, whose codes cost a third of the
// instructions, 156 MB in 40.5 us (3.9 TB/s; 42.1 with three axes).
//
// D/16 threads hold one head's row, sixteen numbers each: the eight pairs
// 8j..8j+7, i.e. two runs of eight numbers (pairs i, i + rot/2) or one run of
// sixteen (pairs of neighbours).  Both members of a pair are then in one
// thread, loads are 16 bytes, and a block of 16 numbers that shares a scale is in one thread or
// two neighbours.  What bounds the pass for many tokens is instructions, not
// yet memory: so a thread multiplies its position's (cos, sin) by the norm's
// weights once for all heads of its token that it takes, and pairs of fp32
// operations go in one instruction.  Cached keys take a path of their own whose every
// rounding is fixed: their codes must not depend on how sums are ordered.
#include <cuda_bf16.h>

#include "common.cuh"
#include "kv4.cuh"
#include "launch.h"

namespace moe {

namespace {

constexpr int kReadThreads = 128;
constexpr int kReadTokens = 4;
constexpr float kSixth = 0x1.555556p-3f;   // 1/6, nearest fp32

// Sixteen numbers as loaded, in two runs of eight.
template <typename XT>
struct Row16;
template <>
struct Row16<__nv_bfloat16> {
    uint4 a, b;
    __device__ void load(const __nv_bfloat16* p, int i, int k) {
        a = *reinterpret_cast<const uint4*>(p + i);
        b = *reinterpret_cast<const uint4*>(p + k);
    }
    __device__ void get(float (&x)[16]) const {
        const uint32_t u[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            x[2 * j] = __uint_as_float(u[j] << 16);
            x[2 * j + 1] = __uint_as_float(u[j] & 0xffff0000u);
        }
    }
};
template <>
struct Row16<float> {
    float4 v[4];
    __device__ void load(const float* p, int i, int k) {
        v[0] = *reinterpret_cast<const float4*>(p + i);
        v[1] = *reinterpret_cast<const float4*>(p + i + 4);
        v[2] = *reinterpret_cast<const float4*>(p + k);
        v[3] = *reinterpret_cast<const float4*>(p + k + 4);
    }
    __device__ void get(float (&x)[16]) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[4 * j] = v[j].x; x[4 * j + 1] = v[j].y; x[4 * j + 2] = v[j].z; x[4 * j + 3] = v[j].w;
        }
    }
};

__device__ __forceinline__ void store8(float* p, const float* y) {
    reinterpret_cast<float4*>(p)[0] = make_float4(y[0], y[1], y[2], y[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(y[4], y[5], y[6], y[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float* y) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
        memcpy(&u[i], &h, 4);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}

// hi + lo += v, exactly but for lo's own rounding (Knuth's two-sum).
__device__ __forceinline__ void two_add(float& hi, float& lo, float v) {
    const float s = __fadd_rn(hi, v);
    const float t = __fsub_rn(s, hi);
    lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, t)), __fsub_rn(v, t)));
    hi = s;
}

// Sum of the squares of a cached key's row over its G threads, carried in two
// words: the key's codes then depend on the sum's nearest fp32 and not on the
// order of its terms.
template <int G>
__device__ __forceinline__ float exact_squares(const float (&x)[16]) {
    float hi = 0.f, lo = 0.f;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
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

// x *= f, and the largest magnitude of each half.  NaN and infinities, whose
// bits are the largest, count as zero and set `bad`.
__device__ __forceinline__ void scale_and_top(float (&x)[16], float f, float& ta, float& tb, bool& bad) {
    uint32_t top[2] = {0u, 0u};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        x[i] = __fmul_rn(x[i], f);
        top[i / 8] = max(top[i / 8], __float_as_uint(x[i]) & 0x7fffffffu);
    }
    if (max(top[0], top[1]) >= 0x7f800000u) {
        bad = true;
        top[0] = top[1] = 0u;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            if ((__float_as_uint(x[i]) & 0x7fffffffu) >= 0x7f800000u) x[i] = 0.f;
            top[i / 8] = max(top[i / 8], __float_as_uint(x[i]) & 0x7fffffffu);
        }
    }
    ta = __uint_as_float(top[0]);
    tb = __uint_as_float(top[1]);
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
// R rows of a thread group are loaded before the first is used.
template <typename XT, int D, bool PAIRS, int R, int TH>
__global__ void __launch_bounds__(TH) qk_norm_rope_kernel(const RopeArgs a) {
    constexpr int G = D / 16;                   // threads of a row
    constexpr int NG = TH / G;                  // rows at a time
    using L = Kv4Layout<D>;
    pdl_wait();
    pdl_trigger();
    const int t = blockIdx.x;
    const int grp = threadIdx.x / G, j = threadIdx.x % G;
    const bool with_cache = a.c.pages != nullptr;
    const int n_qk = a.n_q + a.n_kv;
    const int h0 = blockIdx.y * a.rows, h1 = min(h0 + a.rows, with_cache ? n_qk + a.n_kv : n_qk);
    const XT* x_row = static_cast<const XT*>(a.qkv) + static_cast<long long>(t) * a.ld;

    // the thread's two runs of eight numbers in a rotated head
    int ia, ib;
    bool turn = false;
    if (PAIRS) {
        ia = 16 * j;
        ib = ia + 8;
        turn = ia < a.rot;
    } else if (8 * j < a.rot / 2) {
        ia = 8 * j;
        ib = ia + a.rot / 2;
        turn = true;
    } else {                                    // numbers that pass through, in the same two halves
        ia = a.rot + 8 * j - a.rot / 2;
        ib = ia + (D - a.rot) / 2;
    }
    // numbers u[i], v[i] of pair i among the sixteen
    auto split = [&](const float (&x)[16], float (&u)[8], float (&v)[8]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            u[i] = PAIRS ? x[2 * i] : x[i];
            v[i] = PAIRS ? x[2 * i + 1] : x[8 + i];
        }
    };
    auto join = [&](const float (&u)[8], const float (&v)[8], float (&x)[16]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            x[PAIRS ? 2 * i : i] = u[i];
            x[PAIRS ? 2 * i + 1 : 8 + i] = v[i];
        }
    };

    // first rows on their way
    Row16<XT> raw[R];
    auto load_rows = [&](int first, int end) {
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int h = first + r * NG + grp;
            if (h < end) raw[r].load(x_row + static_cast<long long>(h) * D, ia, ib);
        }
    };
    const int q_end = min(h1, with_cache ? a.n_q : n_qk);   // rows of the plain path
    load_rows(h0, q_end);

    // the token's place in the cache, and its page
    int seq = -1, place = -1, first_new = 0, len = 0;
    if (with_cache) {
        seq = find_seq(a.q_start, a.c.S, t);
        if (seq >= 0) {
            const int q0 = a.q_start[seq];
            len = a.c.seq_len[seq];
            first_new = len - (a.q_start[seq + 1] - q0);
            place = first_new + (t - q0);
        }
    }
    int page = -1;
    if (place >= 0 && h1 > a.n_q) {
        const int col = place / kPage;
        if (col < a.c.max_pages) page = a.c.page_table[static_cast<long long>(seq) * a.c.max_pages + col];
    }

    // The other token of the values' bytes, if it is new too: codes of places 2 j and 2 j + 1 share them.
    const bool odd = place & 1;
    const bool other = place >= 0 && (odd ? place - 1 >= first_new && t > 0 : place + 1 < len && t + 1 < a.T);
    const int step = odd ? -1 : 1;

    // (cos, sin) of the thread's eight pairs
    float cs[8], sn[8];
    bool off = false, other_off = false;        // a position of this or the other token is outside the table
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        cs[i] = 1.f;
        sn[i] = 0.f;
    }
    if (turn) {
        const int half = a.rot / 2;
        auto position = [&](int ax, int d) {    // of token t + d
            if (a.positions != nullptr) return ax < a.axes ? a.positions[static_cast<long long>(ax) * a.T + t + d] : -1;
            return max(place + d, 0);           // negative: a row of a padded batch, not appended
        };
        auto inside = [&](int p) { return p >= 0 && p < a.n_pos; };
        auto row_of = [&](int ax) {
            if (other && h1 > n_qk && !inside(position(ax, step))) other_off = true;
            const int p = position(ax, 0);
            if (inside(p)) return p;
            report(a.st, MOE_DEV_BAD_INDEX, p);
            off = true;
            return 0;
        };
        if (a.axis == nullptr) {
            const float4* src = reinterpret_cast<const float4*>(a.table + static_cast<long long>(row_of(0)) * half + 8 * j);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 v = src[i];
                cs[2 * i] = v.x; sn[2 * i] = v.y; cs[2 * i + 1] = v.z; sn[2 * i + 1] = v.w;
            }
        } else {
            const uint2 axes = *reinterpret_cast<const uint2*>(a.axis + 8 * j);
            int last_ax = -1, p = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int ax = ((i < 4 ? axes.x : axes.y) >> (8 * (i % 4))) & 0xff;
                if (ax != last_ax) p = row_of(ax);
                last_ax = ax;
                const float2 v = a.table[static_cast<long long>(p) * half + 8 * j + i];
                cs[i] = v.x;
                sn[i] = v.y;
            }
        }
    }

    // nothing is written of a token with a position outside the table (a warp holds all pairs of its rows)
    if (__any_sync(kFull, off)) return;
    other_off = __any_sync(kFull, other_off);

    // ---- rows of the plain path: queries, and keys that are not cached ----
    // y_u = inv (u (w_u cos) - v (w_v sin)),  y_v = inv (v (w_v cos) + u (w_u sin)): the products in
    // brackets are the same for all heads
    auto plain = [&](int begin, int end, const float* w, XT* out, long long ld_out, int h_out) {
        float2 uc[4], vs[4], vc[4], us[4];
        {
            float x[16], wu[8], wv[8];
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = 1.f;
            if (w != nullptr) {
                Row16<float> ww;
                ww.load(w, ia, ib);
                ww.get(x);
            }
            split(x, wu, wv);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uc[i] = make_float2(wu[2 * i] * cs[2 * i], wu[2 * i + 1] * cs[2 * i + 1]);
                us[i] = make_float2(wu[2 * i] * sn[2 * i], wu[2 * i + 1] * sn[2 * i + 1]);
                vc[i] = make_float2(wv[2 * i] * cs[2 * i], wv[2 * i + 1] * cs[2 * i + 1]);
                vs[i] = make_float2(-wv[2 * i] * sn[2 * i], -wv[2 * i + 1] * sn[2 * i + 1]);
            }
        }
        for (int first = begin; first < end; first += R * NG) {
            if (first != h0) load_rows(first, end);
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int h = first + r * NG + grp;
                // whole warps leave together: the shuffles below want every lane
                if (first + r * NG + (static_cast<int>(threadIdx.x) & ~31) / G >= end) break;
                float x[16], u[8], v[8];
                raw[r].get(x);
                split(x, u, v);
                float inv = 1.f;
                if (w != nullptr) {
                    float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 p = make_float2(x[2 * i], x[2 * i + 1]);
                        s2 = fma2(p, p, s2);
                    }
                    float ss = s2.x + s2.y;
#pragma unroll
                    for (int off = G / 2; off >= 1; off >>= 1) ss += __shfl_xor_sync(kFull, ss, off);
                    // 1 / sqrt, refined once from the approximate one (rows of zeros with eps = 0 give inf * 0 = NaN, as the formula)
                    const float mean = fmaf(ss, 1.0f / D, a.eps);
                    inv = rsqrtf(mean);
                    const float e = fmaf(-mean * inv, inv, 1.f);
                    if (isfinite(e)) inv = fmaf(0.5f * inv, e, inv);
                }
                const float2 i2 = make_float2(inv, inv);
                float yu[8], yv[8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float2 u2 = make_float2(u[2 * i], u[2 * i + 1]), v2 = make_float2(v[2 * i], v[2 * i + 1]);
                    float2 p = mul2(u2, uc[i]), q = mul2(v2, vc[i]);
                    if (turn) {                 // numbers that pass through keep an infinity to themselves
                        p = fma2(v2, vs[i], p);
                        q = fma2(u2, us[i], q);
                    }
                    if (w != nullptr) {
                        p = mul2(p, i2);
                        q = mul2(q, i2);
                    }
                    yu[2 * i] = p.x; yu[2 * i + 1] = p.y;
                    yv[2 * i] = q.x; yv[2 * i + 1] = q.y;
                }
                join(yu, yv, x);
                if (h < end && out != nullptr) {
                    XT* o = out + static_cast<long long>(t) * ld_out + static_cast<long long>(h - h_out) * D;
                    store8(o + ia, x);
                    store8(o + ib, x + 8);
                }
            }
        }
    };
    if (h0 < min(h1, a.n_q)) plain(h0, min(h1, a.n_q), a.q_w, static_cast<XT*>(a.q_out), a.ld_q, 0);
    if (!with_cache) {
        const int begin = max(h0, a.n_q);
        if (begin < h1) plain(begin, h1, a.k_w, static_cast<XT*>(a.k_out), a.ld_k, a.n_q);
        return;
    }
    if (h1 <= a.n_q) return;

    // ---- keys and values into the cache ----
    if (place >= 0 && (page < 0 || page >= a.c.n_pages)) {
        if (threadIdx.x == 0) report(a.st, MOE_DEV_BAD_INDEX, page);
        page = -1;
    }
    uint8_t* page_base = page >= 0 ? static_cast<uint8_t*>(a.c.pages) + static_cast<long long>(page) * a.c.n_kv * L::bytes : nullptr;
    const int tok = place >= 0 ? place % kPage : 0;
    for (int first = max(h0, a.n_q); first < h1; first += NG) {
        const int h = first + grp;
        const bool is_k = h < h1 && h < n_qk, is_v = h < h1 && h >= n_qk;
        const int kv = is_v ? h - n_qk : h - a.n_q;
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = 0.f;
        if (h < h1) {
            Row16<XT> row;
            row.load(x_row + static_cast<long long>(h) * D, is_v ? 16 * j : ia, is_v ? 16 * j + 8 : ib);
            row.get(x);
        }
        if (__any_sync(kFull, is_k)) {
            float u[8], v[8];
            if (a.k_w != nullptr) {
                const float ss = exact_squares<G>(x);
                const float inv = __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(ss, 1.0f / D), a.eps)));
                if (is_k) {
                    Row16<float> ww;
                    float w[16];
                    ww.load(a.k_w, ia, ib);
                    ww.get(w);
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] = __fmul_rn(__fmul_rn(x[i], inv), w[i]);
                }
            }
            if (is_k) {
                if (turn) {
                    split(x, u, v);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float p = __fsub_rn(__fmul_rn(u[i], cs[i]), __fmul_rn(v[i], sn[i]));
                        v[i] = __fadd_rn(__fmul_rn(v[i], cs[i]), __fmul_rn(u[i], sn[i]));
                        u[i] = p;
                    }
                    join(u, v, x);
                }
                if (a.k_out != nullptr) {
                    XT* o = static_cast<XT*>(a.k_out) + static_cast<long long>(t) * a.ld_k + static_cast<long long>(kv) * D;
                    store8(o + ia, x);
                    store8(o + ib, x + 8);
                }
            }
        }
        if (page_base == nullptr) continue;
        // quantise: keys alone, values with the other token of their pair
        bool bad = false;
        float inv_h = 1.f;
        if (is_k || is_v) {
            const float* hs = is_k ? a.c.k_scale : a.c.v_scale;
            if (hs != nullptr) inv_h = __frcp_rn(hs[kv]);
        }
        float ta, tb;
        scale_and_top(x, inv_h, ta, tb, bad);
        // a block of 16: the thread's own, or the runs of two threads
        const float oa = __shfl_xor_sync(kFull, ta, 1), ob = __shfl_xor_sync(kFull, tb, 1);
        if (PAIRS || is_v) {
            ta = tb = fmaxf(ta, tb);
        } else {
            ta = fmaxf(ta, oa);
            tb = fmaxf(tb, ob);
        }
        float ra, rb;
        const uint32_t sa = block_scale(ta, ra), sb = block_scale(tb, rb);
        if (bad) report(a.st, MOE_DEV_NONFINITE, t);
        uint8_t* base = page_base + static_cast<long long>(kv) * L::bytes;
        if (is_k) {
            uint32_t c[2];
#pragma unroll
            for (int z = 0; z < 2; ++z) {
                const float r = z ? rb : ra;
                c[z] = 0u;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    c[z] |= f32_to_e2m1x2(__fmul_rn(x[8 * z + 2 * i], r), __fmul_rn(x[8 * z + 2 * i + 1], r)) << (8 * i);
            }
            *reinterpret_cast<uint32_t*>(base + L::k_code(tok, ia)) = c[0];
            *reinterpret_cast<uint32_t*>(base + L::k_code(tok, ib)) = c[1];
            if (PAIRS) {
                base[L::k_scale(tok, j)] = static_cast<uint8_t>(sa);
            } else if ((j & 1) == 0) {
                base[L::k_scale(tok, ia / 16)] = static_cast<uint8_t>(sa);
                base[L::k_scale(tok, ib / 16)] = static_cast<uint8_t>(sb);
            }
        }
        if (!is_v) continue;
        // Codes of two neighbouring tokens share a byte.  The even token's row also writes
        // the odd one's if that is new too; a token whose partner is older, or is
        // not written, puts its half beside the codes that are there.
        const bool partner = other && !other_off;
        if (odd && partner) continue;
        float z[16];
        float rz = 0.f;
        uint32_t sz = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) z[i] = 0.f;
        if (partner) {
            bool bad2 = false;
            Row16<XT> o;
            o.load(x_row + a.ld + static_cast<long long>(h) * D, 16 * j, 16 * j + 8);
            o.get(z);
            float za, zb;
            scale_and_top(z, inv_h, za, zb, bad2);
            sz = block_scale(fmaxf(za, zb), rz);
            if (bad2) report(a.st, MOE_DEV_NONFINITE, t + 1);
        }
        const int pj = tok / 2;
        uint32_t c[4] = {0u, 0u, 0u, 0u};
        uint32_t* codes0 = reinterpret_cast<uint32_t*>(base + L::v_code(pj, 16 * j));
        uint32_t* codes1 = reinterpret_cast<uint32_t*>(base + L::v_code(pj, 16 * j + 8));
        if (odd) {
#pragma unroll
            for (int i = 0; i < 4; ++i) c[i] = (i < 2 ? codes0[i] : codes1[i - 2]) & 0x0f0f0f0fu;
#pragma unroll
            for (int i = 0; i < 16; ++i) c[i / 4] |= f32_to_e2m1x2(0.f, __fmul_rn(x[i], ra)) << (8 * (i % 4));
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) c[i / 4] |= f32_to_e2m1x2(__fmul_rn(x[i], ra), __fmul_rn(z[i], rz)) << (8 * (i % 4));
            if (other && !partner) {
#pragma unroll
                for (int i = 0; i < 4; ++i) c[i] |= (i < 2 ? codes0[i] : codes1[i - 2]) & 0xf0f0f0f0u;
            }
        }
        *reinterpret_cast<uint2*>(codes0) = make_uint2(c[0], c[1]);
        *reinterpret_cast<uint2*>(codes1) = make_uint2(c[2], c[3]);
        uint8_t* s = base + L::v_scale(pj, j);
        if (partner) *reinterpret_cast<uint16_t*>(s) = static_cast<uint16_t>(sa | (sz << 8));
        else s[odd] = static_cast<uint8_t>(sa);
    }
}

// One CTA: `tokens` rows of moe_kv4_read; D/8 threads hold eight numbers of a
// key or value head.
template <int D>
__global__ void __launch_bounds__(kReadThreads) kv4_read_kernel(const moe_kv4_cache c, const int32_t* q_start, int T,
                                                                int tokens, __nv_bfloat16* k_out, __nv_bfloat16* v_out,
                                                                moe_dev_status* st) {
    constexpr int G = D / 8;
    using L = Kv4Layout<D>;
    __shared__ int s_page[kReadTokens], s_tok[kReadTokens];
    pdl_wait();
    pdl_trigger();
    const int j = threadIdx.x % G;
    const int t0 = blockIdx.x * tokens, n_t = min(tokens, T - t0);
    // the chain sequence -> length -> page of every token at once
    if (static_cast<int>(threadIdx.x) < n_t) {
        const int t = t0 + threadIdx.x;
        const int seq = find_seq(q_start, c.S, t);
        int place = -1, page = -1;
        if (seq >= 0) place = c.seq_len[seq] - q_start[seq + 1] + t;
        if (place >= 0) {
            const int col = place / kPage;
            page = col < c.max_pages ? c.page_table[static_cast<long long>(seq) * c.max_pages + col] : -1;
            if (page < 0 || page >= c.n_pages) {
                report(st, MOE_DEV_BAD_INDEX, page);
                page = -1;
            }
        }
        s_page[threadIdx.x] = page;
        s_tok[threadIdx.x] = place >= 0 ? place % kPage : 0;
    }
    __syncthreads();
    const int heads = 2 * c.n_kv;
    for (int x = blockIdx.y * (kReadThreads / G) + threadIdx.x / G; x < n_t * heads; x += gridDim.y * (kReadThreads / G)) {
        const int i = x / heads, r = x - i * heads, t = t0 + i;
        const int page = s_page[i], tok = s_tok[i];
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
        store8(o, y);
    }
}

}  // namespace

template <typename XT, int D, bool PAIRS>
static cudaError_t launch_rope_t(RopeArgs& a, cudaStream_t s) {
    const int heads = a.c.pages != nullptr ? a.n_q + 2 * a.n_kv : a.n_q + a.n_kv;
    // Few tokens: a head for each thread group, so that the heads' loads and
    // reductions run side by side on many SMs.  Many tokens: one warp takes all
    // heads of a token, four rows a thread group in flight, and what the token
    // needs besides its rows is read and multiplied once (8192 tokens of 40
    // heads, no cache: one warp 29 us, two 33, four 45; two rows in flight 32, eight 32).
    // us of few/many for 256, 512, 1024, 2048 tokens of 32 + 4 + 4 heads: 4.4/4.3 5.8/4.4 9.2/5.0 16.1/6.6, and
    // with the cache (read back in the same time) 8.5/10.5 11.0/10.9 16.0/11.5 25.5/14.2.
    const bool few = static_cast<long long>(a.T) * heads < (a.c.pages != nullptr ? 20480 : 9216);
    constexpr int kFew = 128, kMany = 32;
    constexpr int R = sizeof(XT) == 2 ? 4 : 2;
    a.rows = few ? kFew / (D / 16) : heads;
    const dim3 grid(a.T, (heads + a.rows - 1) / a.rows);
    if (few) return launch_pdl(qk_norm_rope_kernel<XT, D, PAIRS, 1, kFew>, grid, dim3(kFew), 0, s, a);
    return launch_pdl(qk_norm_rope_kernel<XT, D, PAIRS, R, kMany>, grid, dim3(kMany), 0, s, a);
}
template <typename XT, int D>
static cudaError_t launch_rope_p(RopeArgs& a, cudaStream_t s) {
    return a.pairs || a.rot == 0 ? launch_rope_t<XT, D, true>(a, s) : launch_rope_t<XT, D, false>(a, s);
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
    if (dtype == MOE_DTYPE_BF16) return D == 128 ? launch_rope_p<__nv_bfloat16, 128>(a, s) : launch_rope_p<__nv_bfloat16, 64>(a, s);
    return D == 128 ? launch_rope_p<float, 128>(a, s) : launch_rope_p<float, 64>(a, s);
}

cudaError_t launch_kv4_read(const moe_kv4_cache& c, const int32_t* q_start, int T, void* k_out, void* v_out,
                            moe_dev_status* st, cudaStream_t s) {
    const int ng = kReadThreads / (c.head_dim / 8);
    // Few tokens: a CTA each (and one for every eight heads).  Many: four tokens a CTA, whose
    // look-ups then run side by side.  us of few/many, 4 key heads: 1024 tokens 3.0/4.4, 2048 4.1/4.8, 4096 6.2/5.6,
    // 8192 10.4/9.3, 16384 18.7/14.4.
    const bool many = T >= 4096;
    const int tokens = many ? kReadTokens : 1;
    const dim3 grid((T + tokens - 1) / tokens, many ? 1 : (2 * c.n_kv + ng - 1) / ng);
    auto* k = static_cast<__nv_bfloat16*>(k_out);
    auto* v = static_cast<__nv_bfloat16*>(v_out);
    if (c.head_dim == 128) return launch_pdl(kv4_read_kernel<128>, grid, dim3(kReadThreads), 0, s, c, q_start, T, tokens, k, v, st);
    return launch_pdl(kv4_read_kernel<64>, grid, dim3(kReadThreads), 0, s, c, q_start, T, tokens, k, v, st);
}

}  // namespace moe
