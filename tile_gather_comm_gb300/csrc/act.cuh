// act.cuh -- the linear operator's activations and their derivatives in fp32, and
// the conversions between its 16-bit types and fp32.
#pragma once

#include <cstdint>
#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/tgc.h"

namespace tgc {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

constexpr float kGeluC = 0.7978845608028654f;   // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;
constexpr float kSqrtHalf = 0.7071067811865476f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

// 1 / (1 + exp(-v)).  __expf and __fdividef are good to about 2^-21 here, far below the
// 2^-9 or 2^-11 of the 16-bit result.
__device__ __forceinline__ float sigmoid_f32(float v) { return __fdividef(1.0f, 1.0f + __expf(-v)); }

// The normal distribution function Phi(z) and g = exp(-z^2 / 2), which gelu and its derivative
// both need.  Phi by Abramowitz and Stegun 7.1.26: erfc(x) = (a1 t + ... + a5 t^5) exp(-x^2),
// t = 1 / (1 + p x), x >= 0, off by at most 1.5e-7 (so Phi by 0.75e-7): a tenth of what rounding
// the result to 16 bits does, for one exponential that the derivative shares.  erff instead took
// the backward's elementwise pass from memory-bound to 168 us for 8192 x 14336 (floor 104 us).
__device__ __forceinline__ float normal_cdf(float z, float *g) {
    const float x = fabsf(z) * kSqrtHalf, e = __expf(-0.5f * z * z);
    const float t = __fdividef(1.0f, fmaf(0.3275911f, x, 1.0f));
    float q = fmaf(1.061405429f, t, -1.453152027f);
    q = fmaf(q, t, 1.421413741f);
    q = fmaf(q, t, -0.284496736f);
    q = fmaf(q, t, 0.254829592f);
    const float tail = 0.5f * q * t * e;  // Phi(-|z|)
    *g = e;
    return z < 0.0f ? tail : 1.0f - tail;
}

template <int ACT>
__device__ __forceinline__ float act_of(float z) {
    if constexpr (ACT == TGC_ACT_RELU) return z < 0.0f ? 0.0f : z;  // NaN stays NaN
    if constexpr (ACT == TGC_ACT_GELU) {
        float g;
        return z * normal_cdf(z, &g);
    }
    // 0.5 (1 + tanh(u)) = 1 / (1 + exp(-2u))
    if constexpr (ACT == TGC_ACT_GELU_TANH) return z * sigmoid_f32(2.0f * kGeluC * z * fmaf(kGeluA * z, z, 1.0f));
    if constexpr (ACT == TGC_ACT_SILU) return z * sigmoid_f32(z);
    return z;
}

template <int ACT>
__device__ __forceinline__ float act_grad_of(float z) {
    if constexpr (ACT == TGC_ACT_RELU) return z > 0.0f ? 1.0f : 0.0f;
    if constexpr (ACT == TGC_ACT_GELU) {
        float g;
        const float phi = normal_cdf(z, &g);
        return fmaf(z * kInvSqrt2Pi, g, phi);
    }
    if constexpr (ACT == TGC_ACT_GELU_TANH) {
        const float s = sigmoid_f32(2.0f * kGeluC * z * fmaf(kGeluA * z, z, 1.0f));
        return s + z * s * (1.0f - s) * 2.0f * kGeluC * fmaf(3.0f * kGeluA * z, z, 1.0f);
    }
    if constexpr (ACT == TGC_ACT_SILU) {
        const float s = sigmoid_f32(z);
        return s * fmaf(z, 1.0f - s, 1.0f);
    }
    return 1.0f;
}

// f(integral constant of the activation): one branch for many elements.
template <typename F>
__device__ __forceinline__ void with_act(int act, F &&f) {
    switch (act) {
        case TGC_ACT_RELU: f(std::integral_constant<int, TGC_ACT_RELU>{}); break;
        case TGC_ACT_GELU: f(std::integral_constant<int, TGC_ACT_GELU>{}); break;
        case TGC_ACT_GELU_TANH: f(std::integral_constant<int, TGC_ACT_GELU_TANH>{}); break;
        case TGC_ACT_SILU: f(std::integral_constant<int, TGC_ACT_SILU>{}); break;
        default: f(std::integral_constant<int, TGC_ACT_NONE>{}); break;
    }
}

}  // namespace tgc
