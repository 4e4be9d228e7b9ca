// Activations of the expert products' epilogue, their slopes, and SwiGLU's gate, in
// fp32.  All go through e = exp(-|v|), which does not overflow: 1 / (1 + exp(-v)) is
// 1 / (1 + e) or e / (1 + e), and the fast division is good to 2 ulp for a
// denominator in [1, 2].
//   gelu       v Phi(v), Phi(v) = erfc(-v / sqrt 2) / 2 (1 + erf cancels below v = -3)
//   gelu_tanh  v (1 + tanh a) / 2 = v / (1 + exp(-2 a)), a = sqrt(2 / pi) (v + 0.044715 v^3)
#pragma once

#include "ep_internal.cuh"

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

template <Act ACT>
__device__ __forceinline__ float slope(float v) {
    if constexpr (ACT == Act::kRelu) return v > 0.0f ? 1.0f : 0.0f;
    if constexpr (ACT == Act::kGelu) return normal_cdf(v) + v * expf(-0.5f * v * v) * 0.3989422804014327f;
    if constexpr (ACT == Act::kGeluTanh) {
        const Logistic l = logistic(kGeluC * (v + kGeluA * v * v * v));
        // far out s c is 0 and the polynomial beside it may be infinite
        const float b = l.s * l.c, d = b > 0.0f ? v * b * (kGeluC * (1.0f + 3.0f * kGeluA * v * v)) : 0.0f;
        return l.s + d;
    }
    if constexpr (ACT == Act::kSilu) {
        const Logistic l = logistic(v);
        return l.s * fmaf(v, l.c, 1.0f);
    }
    return 1.0f;
}
#endif

}  // namespace ep
