// Bias, activation and residual of a GEMM's epilogue.
#pragma once

#include "biv_common.cuh"

namespace biv {

// Bias, activation and residual of an epilogue.
struct BiasActArgs {
    const __nv_bfloat16* bias;        // [N] or null
    const __nv_bfloat16* residual;    // [M, N] or null; may be C itself
    int act;                          // BIV_ACT_*
};

namespace {

// 1 + erf(x / sqrt 2) = erfc(-x / sqrt 2), without branches (the epilogue of the last tile
// is not hidden behind any product, and erff takes both of its branches in nearly every
// warp): for x <= 0 and z = |x| / sqrt 2, erfc z = e^(-z^2) t P(t) with t = 1 / (1 + 0.44 z)
// and P of degree 7, fitted here to a least largest RELATIVE error over 0 <= z <= 10
// (1.8e-7), so that GELU's negative tail keeps its digits: what is left is the roundings,
// those of the exponent z^2 above all, below (24 + 4 z^2) 2^-24 of the value together.
BIV_DEV float one_plus_erf_half(float x) {
    const float t = __fdividef(1.0f, fmaf(0.44f * 0.70710678118654752f, fabsf(x), 1.0f));
    float p = fmaf(0.0712231752f, t, -0.277946787f);
    p = fmaf(p, t, 0.296685352f);
    p = fmaf(p, t, -0.0201787074f);
    p = fmaf(p, t, 0.215811205f);
    p = fmaf(p, t, 0.217313856f);
    p = fmaf(p, t, 0.248871132f);
    p = fmaf(p, t, 0.248220955f);
    const float e = p * t * ex2_approx(-0.72134752f * x * x);
    return x < 0.0f ? e : 2.0f - e;
}

// x / (1 + e^-y), a few ulp (silu with y = x).  e^-y = infinity gives 0.
BIV_DEV float times_sigmoid(float x, float y) { return __fdividef(x, 1.0f + ex2_approx(-1.4426950408889634f * y)); }

// act(x) in fp32, without branches: the epilogue of a CTA's last tile is not hidden
// behind any product.  Relative errors stay below (24 + 4 |y|) 2^-24, y being the
// exponential's argument (x^2 / 2 for the erf form; |x|; 2 |u| for the tanh form), and what
// lies below 2^-126 |x| may be lost: far below a bf16 C's half step of 2^-8, and some units
// of an fp32 C.  x/2 (1 + tanh u) = x / (1 + e^-2u) loses nothing to cancellation.
BIV_DEV float activate(float x, int act) {
    switch (act) {
        case BIV_ACT_RELU: return x > 0.0f || x != x ? x : 0.0f;
        case BIV_ACT_GELU: return 0.5f * x * one_plus_erf_half(x);
        case BIV_ACT_GELU_TANH: return times_sigmoid(x, 1.5957691216057308f * fmaf(0.044715f * x * x, x, x));
        case BIV_ACT_SILU: return times_sigmoid(x, x);
        default: return x;
    }
}

// Sixteen bytes of a row that this kernel may overwrite later (a residual that
// is C itself): an ordinary load, never through the read-only path.
BIV_DEV uint4 ld_global_16(const void* p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

// Sixteen columns of one row: C = act(acc + bias) + residual, one rounding.
// 1023 x 14336 x 4096 with bias and GELU: 78 us, the plain product 71 (the last tile's
// epilogue is not covered by MMAs); operands after the accumulators and the C library's
// erff: 80.
struct BiasActRow {
    uint4 bs[2], rs[2];
    bool in[2];
    long long at;

    // The operands from memory (requested before the accumulators are waited for).
    BIV_DEV BiasActRow(bool live, int row, int col, int N, const BiasActArgs& ba) {
        at = static_cast<long long>(row) * N + col;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            in[h] = live && col + 8 * h < N;
            bs[h] = rs[h] = make_uint4(0, 0, 0, 0);
            if (in[h] && ba.bias) bs[h] = __ldg(reinterpret_cast<const uint4*>(ba.bias + col + 8 * h));
            if (in[h] && ba.residual) rs[h] = ld_global_16(ba.residual + at + 8 * h);
        }
    }
    static BIV_DEV float operand(const uint4& y, int e) {
        const uint32_t w = e < 2 ? y.x : e < 4 ? y.y : e < 6 ? y.z : y.w;
        return (e & 1) ? bf16hi(w) : bf16lo(w);
    }
    // All sixteen columns, v(e) the accumulator of column e; an activation's steps run side by side for all
    // of them: 1023 x 14336 x 4096 in e4m3 with (relu, gelu, gelu_tanh, silu) 61.5, 84.1, 67.2, 66.7 us, 63.9, 91.1, 71.6, 73.5
    // for eight and eight (59.8 without an activation).
    template <typename V>
    BIV_DEV void values(V&& v, const BiasActArgs& ba, float (&x)[2][8]) const {
        auto all = [&](auto f) {                   // f(value, half, column of it), all of them side by side
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int e = 0; e < 8; ++e) x[h][e] = f(x[h][e], h, e);
        };
        all([&](float, int h, int e) { return v(8 * h + e); });
        if (ba.bias) all([&](float y, int h, int e) { return y + operand(bs[h], e); });
        switch (ba.act) {
            case BIV_ACT_NONE: break;
            case BIV_ACT_RELU: all([](float y, int, int) { return activate(y, BIV_ACT_RELU); }); break;
            case BIV_ACT_GELU: all([](float y, int, int) { return activate(y, BIV_ACT_GELU); }); break;
            case BIV_ACT_GELU_TANH: all([](float y, int, int) { return activate(y, BIV_ACT_GELU_TANH); }); break;
            default: all([](float y, int, int) { return activate(y, BIV_ACT_SILU); }); break;
        }
        if (ba.residual) all([&](float y, int h, int e) { return y + operand(rs[h], e); });
    }
    static BIV_DEV uint4 pack8(const float (&x)[8]) {
        return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    }
    template <bool F32, typename V>
    BIV_DEV void store(V&& v, void* C, const BiasActArgs& ba) const {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (!in[h]) continue;
            // column after column: the last tile of a small product waits for it (8 x 6144 x 4096 in bf16 12.5 us, with the
            // steps of eight columns side by side 12.75)
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                x[e] = v(8 * h + e);
                if (ba.bias) x[e] += operand(bs[h], e);
            }
            if (ba.act != BIV_ACT_NONE) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = activate(x[e], ba.act);
            }
            if (ba.residual) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] += operand(rs[h], e);
            }
            if constexpr (F32) {
                float4* dst = reinterpret_cast<float4*>(static_cast<float*>(C) + at + 8 * h);
                dst[0] = make_float4(x[0], x[1], x[2], x[3]);
                dst[1] = make_float4(x[4], x[5], x[6], x[7]);
            } else {
                *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(C) + at + 8 * h) = pack8(x);
            }
        }
    }
};

}  // namespace
}  // namespace biv
