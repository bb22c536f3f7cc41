// w4.cuh -- weights in 4 bits (moe_w4 in moe_gb300.h): the layout of a tile and
// the conversion of its codes to bf16, shared by the kernels that pack them
// and those that multiply by them.
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace moe {

constexpr int kW4Tile = 128;                       // rows and columns of a tile
constexpr int kW4Codes = kW4Tile * kW4Tile / 2;    // bytes of its codes
constexpr int kW4Bytes = kW4Codes + kW4Tile * 8;   // and of all of it
// What the operands are too small by: a code's bits stand for its value times 2^-126, the scales are taken times
// 2^119, and the sums are multiplied by this at the end (a power of two, so exact).
constexpr float kW4Up = 128.f;

// Byte of the 16-byte run with columns 32 c .. 32 c + 31 of row r.  The run's place among its eight rows is
// turned by 2c, so that neither eight rows of one column nor two rows of four columns share a bank.
__host__ __device__ __forceinline__ int w4_run(int r, int c) { return (r >> 3) * 512 + c * 128 + (((r & 7) ^ (2 * c)) * 16); }
__host__ __device__ __forceinline__ int w4_scale(int r, int b) { return kW4Codes + r * 8 + b; }

// A code's four bits (sign, magnitude) in a half of a word, for the codes j = 0 .. 3 of the half.  Shifted left by 0, 3
// and 6 the first three have sign and magnitude where a bf16 has its sign, the two low bits of its exponent
// and its first bit behind; the fourth takes what is left.
__host__ __device__ __forceinline__ uint32_t w4_half_bits(uint32_t code, int j) {
    const uint32_t s = code >> 3, m = code & 7u;
    switch (j) {
        case 0: return s << 15 | m << 6;
        case 1: return s << 12 | m << 3;
        case 2: return s << 9 | m;
        default: return s << 14 | (m >> 2) << 13 | (m & 3u) << 10;
    }
}

// Eight codes as four bf16x2, (0, 1), (2, 3), (4, 5), (6, 7): each the code's value times 2^-126, exactly (0.5 is a
// subnormal bf16).
__device__ __forceinline__ void w4_values(uint32_t w, uint32_t (&f)[4]) {
    constexpr uint32_t kSignMag = 0x81c081c0u;
    f[0] = w & kSignMag;
    f[1] = (w << 3) & kSignMag;
    f[2] = (w << 6) & kSignMag;
    f[3] = ((w << 1) & 0x80008000u) | ((w >> 5) & 0x01000100u) | ((w >> 4) & 0x00c000c0u);
}

__device__ __forceinline__ uint32_t bmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Two e4m3 scales (low, high byte), each as a pair of bf16 equal to it times 2^119.
__device__ __forceinline__ void w4_scales(uint32_t two, uint32_t& lo, uint32_t& hi) {
    uint32_t b;
    float x, y;
    asm("{\n\t.reg .b16 s, p, q;\n\t.reg .b32 h;\n\tcvt.u16.u32 s, %2;\n\tcvt.rn.f16x2.e4m3x2 h, s;\n\t"
        "mov.b32 {p, q}, h;\n\tcvt.f32.f16 %0, p;\n\tcvt.f32.f16 %1, q;\n\t}"
        : "=f"(x), "=f"(y)
        : "r"(two));
    x *= 0x1p119f;
    y *= 0x1p119f;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(b) : "f"(y), "f"(x));   // exact: four significant bits
    lo = __byte_perm(b, 0, 0x1010);
    hi = __byte_perm(b, 0, 0x3232);
}

}  // namespace moe
