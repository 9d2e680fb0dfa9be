// Numbers in 8 bits (e4m3: 4 exponent bits, 3 of the significand, largest 448, no
// infinities) and their scales.
#pragma once

#include "biv_common.cuh"

namespace biv {
namespace {

constexpr float kE4M3Max = 448.0f;
constexpr float kLeastScale = 7.888609052210118e-31f;      // 2^-100: its inverse is in fp32's range

// Two numbers, rounded to nearest even; what passes 448 is held as 448, a NaN as NaN.
BIV_DEV uint32_t pack_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
BIV_DEV uint32_t pack_e4m3x4(float a, float b, float c, float d) { return pack_e4m3x2(a, b) | pack_e4m3x2(c, d) << 16; }

// Numbers 0, 1 (lo) or 2, 3 (hi) of four as fp16, which holds every e4m3 number.
BIV_DEV uint32_t e4m3_lo(uint32_t x) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(x));
    return r;
}
BIV_DEV uint32_t e4m3_hi(uint32_t x) {
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(x));
    return r;
}

// The larger of |x| in each half of packed bf16 numbers; a NaN counts as nothing.
BIV_DEV uint32_t max_abs_bf16x2(uint32_t m, uint32_t x) {
    uint32_t r;
    asm("{\n\t.reg .b32 a;\n\tabs.bf16x2 a, %2;\n\tmax.bf16x2 %0, %1, a;\n\t}" : "=r"(r) : "r"(m), "r"(x));
    return r;
}
BIV_DEV float max_of_halves(uint32_t m) { return fmaxf(bf16lo(m), bf16hi(m)); }

// The scale of values up to amax: amax / 448, and no less than 2^-100 (a block of zeros).
// An infinity counts as the largest bf16 number.
BIV_DEV float scale_of(float amax) {
    return fmaxf(__fdiv_rn(fminf(amax, 3.3895313892515355e38f), kE4M3Max), kLeastScale);
}

// Eight bf16 numbers over s (inv: its inverse) as e4m3.  x inv alone falls beside a tie of the
// quotient too often (one value in 10^3, where x and the largest of its block are small multiples
// of one another); one correction by its remainder (Markstein's) makes it the quotient.  An infinity leaves it as a NaN.
BIV_DEV float over(float x, float s, float inv) {
    const float q = x * inv;
    return fmaf(fmaf(-q, s, x), inv, q);
}
BIV_DEV uint2 e4m3x8(const uint4& x, float s, float inv) {
    return make_uint2(pack_e4m3x4(over(bf16lo(x.x), s, inv), over(bf16hi(x.x), s, inv), over(bf16lo(x.y), s, inv), over(bf16hi(x.y), s, inv)),
                      pack_e4m3x4(over(bf16lo(x.z), s, inv), over(bf16hi(x.z), s, inv), over(bf16lo(x.w), s, inv), over(bf16hi(x.w), s, inv)));
}
BIV_DEV uint32_t max_abs8(const uint4& x) {
    return max_abs_bf16x2(max_abs_bf16x2(max_abs_bf16x2(max_abs_bf16x2(0u, x.x), x.y), x.z), x.w);
}

}  // namespace
}  // namespace biv
