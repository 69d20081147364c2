// act.cuh -- the linear operator's activations and their derivatives in fp32, and
// the conversions between its 16-bit types and fp32.
#pragma once

#include <cstdint>
#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/tgc.h"
#include "pairs.cuh"

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

// The activations work on pairs (packed fp32): beside the products the epilogue's arithmetic is not
// free -- 13 single instructions an element more took 13 % off the tensor pipe of a 4096 x 4096 x
// 14336 product, whose other limits they do not touch.
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;
constexpr float kTanhK1 = 1.5957691216057308f;    // 2 sqrt(2 / pi)
constexpr float kTanhK2 = 0.07135481627260025f;   // 2 sqrt(2 / pi) 0.044715

// 2^x and 1 / x by the hardware's approximations (about 2^-22): far below the 2^-9 or 2^-11 that
// rounding the result to 16 bits costs.
__device__ __forceinline__ F2 exp2_f2(F2 a) {
    float2 f = split(a);
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(f.x));
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(f.y));
    return f2(f.x, f.y);
}
__device__ __forceinline__ F2 rcp_f2(F2 a) {
    float2 f = split(a);
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(f.x));
    asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(f.y));
    return f2(f.x, f.y);
}

// 1 / (1 + exp(-v))
__device__ __forceinline__ F2 sigmoid_f2(F2 v) {
    return rcp_f2(add(exp2_f2(mul(v, every<F2>(-kLog2e))), every<F2>(1.0f)));
}

// The normal distribution function Phi(z) and e = exp(-z^2 / 2), which gelu and its derivative
// both need.  Phi by Abramowitz and Stegun 7.1.26: erfc(x) = (a1 t + ... + a5 t^5) exp(-x^2),
// t = 1 / (1 + p x), x >= 0, off by at most 1.5e-7, so Phi by 0.75e-7; with fp32's roundings by 2.5e-7 (near
// 0).  One exponential, which the derivative shares.  The bound is absolute, as that of 0.5 (1 + erf) in
// fp32: below z = -3 Phi falls faster than its error.  gelu(-4) = -1.3e-4 is off by half a unit of f16's
// last place, and of bf16's 2^-8 gelu(-5) = -1.4e-6 is off by 0.4, gelu(-7) = -9e-12 by 1.7 and gelu(-10) =
// -8e-23 by 5.  erff instead took the backward's elementwise pass from memory-bound to 168 us for 8192 x
// 14336 (floor 104 us).
__device__ __forceinline__ F2 normal_cdf(F2 z, F2 *e) {
    const F2 x = F2{z.v & 0x7fffffff7fffffffull};
    *e = exp2_f2(mul(mul(z, z), every<F2>(-0.5f * kLog2e)));
    const F2 t = rcp_f2(fma(x, every<F2>(0.3275911f * 0.7071067811865476f), every<F2>(1.0f)));
    F2 q = fma(t, every<F2>(0.5f * 1.061405429f), every<F2>(0.5f * -1.453152027f));
    q = fma(q, t, every<F2>(0.5f * 1.421413741f));
    q = fma(q, t, every<F2>(0.5f * -0.284496736f));
    q = fma(q, t, every<F2>(0.5f * 0.254829592f));
    const F2 tail = mul(mul(q, t), *e);  // Phi(-|z|)
    const float2 zs = split(z), lo = split(tail), hi = split(fma(tail, every<F2>(-1.0f), every<F2>(1.0f)));
    return f2(zs.x < 0.0f ? lo.x : hi.x, zs.y < 0.0f ? lo.y : hi.y);
}

// 0.5 (1 + tanh(u)) = 1 / (1 + exp(-2u)), u = sqrt(2 / pi) (z + 0.044715 z^3)
__device__ __forceinline__ F2 tanh_gate(F2 z, F2 zz) {
    return sigmoid_f2(mul(z, fma(zz, every<F2>(kTanhK2), every<F2>(kTanhK1))));
}

template <int ACT>
__device__ __forceinline__ F2 act_of(F2 z) {
    if constexpr (ACT == TGC_ACT_RELU) {
        const float2 f = split(z);
        return f2(f.x < 0.0f ? 0.0f : f.x, f.y < 0.0f ? 0.0f : f.y);  // NaN stays NaN
    }
    if constexpr (ACT == TGC_ACT_GELU) {
        F2 e;
        return mul(z, normal_cdf(z, &e));
    }
    if constexpr (ACT == TGC_ACT_GELU_TANH) return mul(z, tanh_gate(z, mul(z, z)));
    if constexpr (ACT == TGC_ACT_SILU) return mul(z, sigmoid_f2(z));
    return z;
}

template <int ACT>
__device__ __forceinline__ F2 act_grad_of(F2 z) {
    const F2 one = every<F2>(1.0f), minus = every<F2>(-1.0f);
    if constexpr (ACT == TGC_ACT_RELU) {
        const float2 f = split(z);
        return f2(f.x > 0.0f ? 1.0f : 0.0f, f.y > 0.0f ? 1.0f : 0.0f);
    }
    if constexpr (ACT == TGC_ACT_GELU) {
        F2 e;
        const F2 phi = normal_cdf(z, &e);
        return fma(mul(z, every<F2>(kInvSqrt2Pi)), e, phi);
    }
    if constexpr (ACT == TGC_ACT_GELU_TANH) {
        // z^2 is cut off where fp32 ends (|z| > 1.8e19): s is 0 or 1 long before, and the term that the
        // slope enters has to be zero there, not zero times infinity.
        const float2 sq = split(mul(z, z));
        const F2 zz = f2(fminf(sq.x, 1e30f), fminf(sq.y, 1e30f)), s = tanh_gate(z, zz);
        const F2 slope = fma(zz, every<F2>(3.0f * kTanhK2), every<F2>(kTanhK1));
        return fma(mul(mul(z, s), fma(s, minus, one)), slope, s);
    }
    if constexpr (ACT == TGC_ACT_SILU) {
        const F2 s = sigmoid_f2(z);
        return fma(mul(z, s), fma(s, minus, one), s);
    }
    return one;
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
