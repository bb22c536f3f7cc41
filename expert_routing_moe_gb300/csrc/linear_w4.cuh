// linear_w4.cuh -- what the two kernels of the products with weights in 4 bits
// share: their arguments, the tokens' numbers and the outputs.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "w4.cuh"

namespace moe {

struct LinearArgs {
    const uint8_t* tiles;
    const float* row_scale;
    const __nv_bfloat16* x;
    long long ld_x, ld_y;
    int T, N, K, kt;                // kt: tiles of 128 columns
    const float* bias;
    void* y;
    bool y_bf16, add, wide;         // wide: x's rows start at 16-byte boundaries
    moe_dev_status* st;
};

// Eight numbers of token t's row from column k on; what lies outside is zero.
__device__ __forceinline__ uint4 load_x8(const LinearArgs& a, int t, int k) {
    if (t >= a.T || k >= a.K) return make_uint4(0u, 0u, 0u, 0u);
    const __nv_bfloat16* p = a.x + t * a.ld_x + k;
    if (a.wide && k + 8 <= a.K) return *reinterpret_cast<const uint4*>(p);
    // the one or two 16-byte words that hold the eight numbers (each holds one of the row at least), shifted into place
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    const uint4* words = reinterpret_cast<const uint4*>(at & ~static_cast<uintptr_t>(15));
    const int off = static_cast<int>(at & 15), left = min(8, a.K - k);
    const uint4 lo = words[0], hi = off + 2 * left > 16 ? words[1] : make_uint4(0u, 0u, 0u, 0u);
    const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int q = off >> 2;
        // (selected, so that the words stay in registers)
        uint32_t x = w[i], y = w[i + 1];
        if (q == 1) { x = w[i + 1]; y = w[i + 2]; }
        if (q == 2) { x = w[i + 2]; y = w[i + 3]; }
        if (q == 3) { x = w[i + 3]; y = w[i + 4 < 8 ? i + 4 : 7]; }
        x = __funnelshift_r(x, y, (off & 2) * 8);
        const int n = left - 2 * i;       // numbers of the pair that are the row's
        v[i] = n >= 2 ? x : n == 1 ? x & 0xffffu : 0u;
    }
    return make_uint4(v[0], v[1], v[2], v[3]);
}

__device__ __forceinline__ void put_y(const LinearArgs& a, int t, int n, float v) {
    const long long at = t * a.ld_y + n;
    if (a.y_bf16) static_cast<__nv_bfloat16*>(a.y)[at] = __float2bfloat16_rn(v);
    else static_cast<float*>(a.y)[at] = a.add ? static_cast<float*>(a.y)[at] + v : v;
}

// How the kernel for many tokens cuts a call: tokens of a tile, CTAs that share one, and the clocks that it should take (for rows of
// x at 16-byte boundaries).
struct LinearTile {
    int tok, split;
    double clocks;
};
LinearTile linear_w4_tile(const LinearArgs& a);
cudaError_t launch_linear_w4_tc(const LinearArgs& a, const LinearTile& t, cudaStream_t s);

}  // namespace moe
