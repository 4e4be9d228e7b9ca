// Activations of the expert products' epilogue, their slopes, and SwiGLU's gate, in
// fp32.  All go through e = exp(-|v|), which does not overflow: 1 / (1 + exp(-v)) is
// 1 / (1 + e) or e / (1 + e), and the fast division is good to 2 ulp for a
// denominator in [1, 2].
//   gelu       v Phi(v), Phi(v) = erfc(-v / sqrt 2) / 2 (1 + erf cancels below v = -3)
//   gelu_tanh  v (1 + tanh a) / 2 = v / (1 + exp(-2 a)), a = sqrt(2 / pi) (v + 0.044715 v^3)
// The slopes, of which 8 bits are kept, take the fast exponential, which is off by 1.2
// |v| ulp (2^-16 of it at most before it vanishes), and gelu's the rational approximation
// 7.1.26 of Abramowitz and Stegun's Handbook of Mathematical Functions, erf to 1.5e-7,
// whose exponential is the density's.  With expf and erfcf the instructions bound the
// backward pass (262144 rows x 2048: 669 us).
#pragma once

#include "ep_internal.cuh"
#include "umma.cuh"

namespace ep {

#ifdef __CUDACC__
// 1 / (1 + exp(-v)) and its complement, neither with cancellation.
struct Logistic {
    float s, c;
};
__device__ __forceinline__ Logistic logistic(float v) {
    const float e = expf(-fabsf(v)), big = __fdividef(1.0f, 1.0f + e), small = e * big;
    return v < 0.0f ? Logistic{small, big} : Logistic{big, small};
}

// g / (1 + exp(-g)).
__device__ __forceinline__ float silu(float g) {
    const float e = expf(-fabsf(g));
    return __fdividef(g < 0.0f ? g * e : g, 1.0f + e);
}

constexpr float kGeluC = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;

__device__ __forceinline__ float normal_cdf(float v) { return 0.5f * erfcf(-0.70710678118654752f * v); }

template <Act ACT>
__device__ __forceinline__ float activate(float v) {
    if constexpr (ACT == Act::kRelu) return v < 0.0f ? 0.0f : v;  // a NaN stays one
    if constexpr (ACT == Act::kGelu) return v * normal_cdf(v);
    if constexpr (ACT == Act::kGeluTanh) return v * logistic(kGeluC * (v + kGeluA * v * v * v)).s;
    if constexpr (ACT == Act::kSilu) return silu(v);
    return v;
}

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

constexpr float kLog2e = 1.4426950408889634f;

// The slopes at a and b, in the instructions that take two numbers at a time.  Values so far out that a slope
// is 0 or 1 to 2^-70 are taken for the limit, so that no factor overflows (dy of 1e38 beside z of -1e38 apart).
template <Act ACT>
__device__ __forceinline__ uint64_t slope2(float a, float b) {
    using namespace umma;
    if constexpr (ACT == Act::kRelu) return two(a > 0.0f ? 1.0f : 0.0f, b > 0.0f ? 1.0f : 0.0f);
    if constexpr (ACT == Act::kGelu) {
        const uint64_t v = two(a, b), t = rcp2(fma2(two(fabsf(a), fabsf(b)), both(0.3275911f * 0.70710678118654752f), both(1.0f)));
        const uint64_t e = exp2_2(mul2(mul2(v, v), both(-0.5f * kLog2e)));  // exp(-v^2 / 2)
        uint64_t q = fma2(t, both(0.5f * 1.061405429f), both(0.5f * -1.453152027f));
        q = fma2(t, q, both(0.5f * 1.421413741f));
        q = fma2(t, q, both(0.5f * -0.284496736f));
        q = mul2(t, fma2(t, q, both(0.5f * 0.254829592f)));
        const uint64_t half = fma2(mul2(q, e), both(-1.0f), both(0.5f));     // Phi(|v|) - 1 / 2
        return fma2(v, mul2(e, both(0.3989422804014327f)), add2(two(copysignf(lo2(half), a), copysignf(hi2(half), b)), both(0.5f)));
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
