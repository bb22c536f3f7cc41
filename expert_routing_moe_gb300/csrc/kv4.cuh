// kv4.cuh -- the 4-bit cache's page layout (moe_kv4_cache in moe_gb300.h) and
// the conversions between its codes and fp16/fp32, shared by the kernels that
// write, read and attend over it.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "common.cuh"

namespace moe {

constexpr int kPage = MOE_KV4_PAGE;

// Byte offsets within one head's part of a page.
template <int D>
struct Kv4Layout {
    static constexpr int kCodes = 0;
    static constexpr int kScales = kPage * D / 2;
    static constexpr int vCodes = kScales + kPage * D / 16;
    static constexpr int vScales = vCodes + kPage * D / 2;
    static constexpr int bytes = vScales + kPage * D / 16;
    static constexpr int U = D / 8;      // value numbers of one 8-row group: a lane's run
    static constexpr int R = D / 64;     // key scales of a lane's run

    __device__ static int k_code(int tok, int i) { return tok * (D / 2) + i / 2; }
    __device__ static int k_scale(int tok, int b) {
        return kScales + (((b / R) * 8 + tok % 8) * 8 + tok / 8) * R + b % R;
    }
    __device__ static int v_code(int j, int e) { return vCodes + (((j / 4) * 8 + e / U) * 4 + j % 4) * U + e % U; }
    __device__ static int v_scale(int j, int b) { return vScales + ((b * 4 + j % 4) * 8 + j / 4) * 2; }
};

// Four bytes of codes as four f16x2: byte k -> (low code, high code).
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
        : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
        : "r"(w));
}

// Two e4m3 scales (low, high byte) as f16x2; every e4m3 number is exact in fp16.
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t two) {
    uint32_t r;
    asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(two));
    return r;
}

// e2m1 codes of (lo, hi), nearest, ties to even, at most 6: hi in the upper half.
__device__ __forceinline__ uint32_t f32_to_e2m1x2(float lo, float hi) {
    uint16_t r;
    asm("{\n\t.reg .b8 b, z;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %2, %1;\n\tmov.b16 %0, {b, 0};\n\t}"
        : "=h"(r)
        : "f"(lo), "f"(hi));
    return r;
}

// e4m3 of x >= 0, nearest, at most 448.
__device__ __forceinline__ uint32_t f32_to_e4m3(float x) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
    return r & 0xffu;
}
__device__ __forceinline__ float e4m3_to_f32(uint32_t b) {
    const uint32_t h = e4m3x2_to_f16(b);
    __half x;
    const uint16_t lo = static_cast<uint16_t>(h & 0xffffu);
    memcpy(&x, &lo, 2);
    return __half2float(x);
}

__device__ __forceinline__ uint32_t hmul2_u(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, c, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y), "f"(z.x), "f"(z.y));
    return r;
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "add.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
    return r;
}
__device__ __forceinline__ float2 mul2(float2 x, float2 y) {
    float2 r;
    asm("{\n\t.reg .b64 a, b, d;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
        "mul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(x.x), "f"(x.y), "f"(y.x), "f"(y.y));
    return r;
}

// The sequence of row t: the s with q_start[s] <= t < q_start[s+1], or -1.
// A decode batch has one row for each sequence, so s = t is tried first.
__device__ __forceinline__ int find_seq(const int32_t* q_start, int S, int t) {
    if (t < S && q_start[t] <= t && t < q_start[t + 1]) return t;
    int lo = 0, hi = S;   // q_start[lo] <= t < q_start[hi], if any
    if (S < 1 || t < q_start[0] || t >= q_start[S]) return -1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (q_start[mid] <= t) lo = mid; else hi = mid;
    }
    return lo;
}

}  // namespace moe
