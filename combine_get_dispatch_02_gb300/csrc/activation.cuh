// Activations of the expert products' epilogue, their slopes, and SwiGLU's gate, in
// fp32.
//   gelu       v Phi(v), Phi by the normal distribution's tail: for v < 0, 1 + erf would cancel
//   gelu_tanh  v (1 + tanh a) / 2 = v / (1 + exp(-2 a)), a = sqrt(2 / pi) (v + 0.044715 v^3)
// Of the epilogue's results 8 bits are kept, and the instructions bound products of few
// channels and the backward pass: all are written in the instructions that take two numbers
// at a time and take the fast exponential, which is off by 1.2 |v| ulp (2^-16 of an activation
// at most before it vanishes).  32768 rows x 2048 x 1024, GELU / SiLU: 102 /
// 100 us, with erfcf and expf 180 / 111 (without activation 94).  The slopes are 1.13 at
// most and bias gradients add them up unrounded, so they are kept to fp32's last bits, which they can be because where
// they matter their exponential's argument is small.  Off by 4e-8 in the root of the mean square over z of N(0, 1) and
// 1.8e-7 at most (the formulas in fp32 3e-8 and 2.4e-7); 262144 rows x 2048, tanh GELU 463 us, with erfcf and expf 669.
#pragma once

#include "ep_internal.cuh"
#include "umma.cuh"

namespace ep {

#ifdef __CUDACC__
// g / (1 + exp(-g)), by exp(-|g|), which does not overflow; the fast division is good to 2 ulp for a denominator in
// [1, 2].
__device__ __forceinline__ float silu(float g) {
    const float e = expf(-fabsf(g));
    return __fdividef(g < 0.0f ? g * e : g, 1.0f + e);
}

constexpr float kGeluC = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t both(float v) { return umma::pair2(__float_as_uint(v), __float_as_uint(v)); }
__device__ __forceinline__ uint64_t two(float a, float b) { return umma::pair2(__float_as_uint(a), __float_as_uint(b)); }
__device__ __forceinline__ float fast_exp2(float v) {
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v));
    return e;
}
__device__ __forceinline__ uint64_t exp2_2(uint64_t v) { return two(fast_exp2(umma::lo2(v)), fast_exp2(umma::hi2(v))); }
__device__ __forceinline__ uint64_t rcp2(uint64_t v) {
    float a, b;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(a) : "f"(umma::lo2(v)));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(b) : "f"(umma::hi2(v)));
    return two(a, b);
}
// Within lo .. hi; a NaN stays one.
__device__ __forceinline__ float within(float v, float lo, float hi) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(v), "f"(lo));
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(r), "f"(hi));
    return r;
}

// |v|, hi at most; a NaN stays one.
__device__ __forceinline__ float size_to(float v, float hi) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(v)), "f"(hi));
    return r;
}
__device__ __forceinline__ float relu(float v) {
    float r;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(v));
    return r;
}

// ReLU's slope, 0 at 0; a NaN stays one.
__device__ __forceinline__ float step(float v) { return v > 0.0f ? 1.0f : v <= 0.0f ? 0.0f : v; }

constexpr float kLog2e = 1.4426950408889634f;

// The activations of a pair.
template <Act ACT>
__device__ __forceinline__ uint64_t activate2(uint64_t v) {
    using namespace umma;
    const float a = lo2(v), b = hi2(v);
    if constexpr (ACT == Act::kRelu) return two(relu(a), relu(b));
    if constexpr (ACT == Act::kGelu) {
        // relu(v) - |v| Phi(-|v|); Phi(-w) exp(w^2 / 2) as t times a polynomial in t = 1 / (1 + 0.31 w), fitted for
        // the least relative error over 0 .. 14.5 (5e-6), behind which it vanishes
        const uint64_t w = two(size_to(a, 20.0f), size_to(b, 20.0f)), t = rcp2(fma2(w, both(0.31f), both(1.0f)));
        const uint64_t e = exp2_2(mul2(mul2(w, w), both(-0.5f * kLog2e)));
        uint64_t q = fma2(t, both(0.07392937650144059f), both(-0.18045104996980305f));
        q = fma2(t, q, both(-0.015743919288480356f));
        q = fma2(t, q, both(-0.13343019678263507f));
        q = fma2(t, q, both(-0.1204411788976998f));
        q = fma2(t, q, both(-0.1238607102091547f));
        return fma2(mul2(mul2(t, q), e), w, two(relu(a), relu(b)));
    }
    if constexpr (ACT == Act::kGeluTanh || ACT == Act::kSilu) {
        // v / (1 + exp(-u)): for u < 0 v exp(u) / (1 + exp(u)), the exponential times 2^24, so that it does not vanish
        // before its product with v does
        const uint64_t u = ACT == Act::kSilu ? v : mul2(v, fma2(mul2(v, v), both(kGeluC * kGeluA), both(kGeluC)));
        const uint64_t e = exp2_2(fma2(two(size_to(lo2(u), 110.0f), size_to(hi2(u), 110.0f)), both(-kLog2e), both(24.0f)));
        const uint64_t r = rcp2(fma2(e, both(0x1p-24f), both(1.0f))), low = mul2(mul2(v, e), both(0x1p-24f));
        return mul2(two(a < 0.0f ? lo2(low) : a, b < 0.0f ? hi2(low) : b), r);
    }
    return v;
}

// The slopes at a and b, in the instructions that take two numbers at a time.  Values so far out that a slope
// is 0 or 1 to 2^-70 are taken for the limit, so that no factor overflows (dy of 1e38 beside z of -1e38 apart).
template <Act ACT>
__device__ __forceinline__ uint64_t slope2(float a, float b) {
    using namespace umma;
    if constexpr (ACT == Act::kRelu) return two(step(a), step(b));
    if constexpr (ACT == Act::kGelu) {
        // Phi(v) + v phi(v): 1 - x for v >= 0 and x below, x = Phi(-w) - w phi(w), w = |v|; Phi(-w) exp(w^2 / 2) as t times
        // a polynomial in t = 1 / (1 + 0.45 w), fitted for the least absolute error of Phi (4e-9 with fp32's coefficients)
        const uint64_t v = two(a, b), w = two(fabsf(a), fabsf(b)), t = rcp2(fma2(w, both(0.45f), both(1.0f)));
        const uint64_t e = exp2_2(mul2(mul2(v, v), both(-0.5f * kLog2e)));  // exp(-v^2 / 2)
        uint64_t q = fma2(t, both(-0.037853848189115524f), both(0.21744683384895325f));
        q = fma2(t, q, both(-0.4740411639213562f));
        q = fma2(t, q, both(0.3936392664909363f));
        q = fma2(t, q, both(0.01813637837767601f));
        q = fma2(t, q, both(0.20540092885494232f));
        q = fma2(t, q, both(0.17727160453796387f));
        const uint64_t x = mul2(e, fma2(t, q, mul2(w, both(-0.3989422804014327f)))), up = fma2(x, both(-1.0f), both(1.0f));
        return two(a < 0.0f ? lo2(x) : lo2(up), b < 0.0f ? hi2(x) : hi2(up));
    }
    if constexpr (ACT == Act::kGeluTanh) {
        const uint64_t v = two(within(a, -9.5f, 15.0f), within(b, -9.5f, 15.0f)), v2 = mul2(v, v);
        const uint64_t e = exp2_2(mul2(v, fma2(v2, both(-kGeluC * kGeluA * kLog2e), both(-kGeluC * kLog2e))));
        const uint64_t s = rcp2(add2(e, both(1.0f))), sc = mul2(mul2(e, s), s);
        return fma2(mul2(v, sc), fma2(v2, both(3.0f * kGeluC * kGeluA), both(kGeluC)), s);
    }
    if constexpr (ACT == Act::kSilu) {
        const uint64_t v = two(within(a, -85.0f, 3e38f), within(b, -85.0f, 3e38f)), e = exp2_2(mul2(v, both(-kLog2e)));
        const uint64_t s = rcp2(add2(e, both(1.0f)));
        return mul2(s, fma2(v, mul2(e, s), both(1.0f)));
    }
    return both(1.0f);
}
#endif

}  // namespace ep
