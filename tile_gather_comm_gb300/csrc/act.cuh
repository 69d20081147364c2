// act.cuh -- the linear operator's activations and their derivatives in fp32, and
// the conversions between its 16-bit types and fp32.
#pragma once

#include <cstdint>
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

__device__ __forceinline__ float act_f32(float z, int act) {
    switch (act) {
        case TGC_ACT_RELU: return z < 0.0f ? 0.0f : z;  // NaN stays NaN
        case TGC_ACT_GELU: return 0.5f * z * (1.0f + erff(z * kSqrtHalf));
        // 0.5 (1 + tanh(u)) = 1 / (1 + exp(-2u))
        case TGC_ACT_GELU_TANH: return z * sigmoid_f32(2.0f * kGeluC * (z + kGeluA * z * z * z));
        case TGC_ACT_SILU: return z * sigmoid_f32(z);
        default: return z;
    }
}

__device__ __forceinline__ float act_grad_f32(float z, int act) {
    switch (act) {
        case TGC_ACT_RELU: return z > 0.0f ? 1.0f : 0.0f;
        case TGC_ACT_GELU:
            return 0.5f * (1.0f + erff(z * kSqrtHalf)) + z * kInvSqrt2Pi * __expf(-0.5f * z * z);
        case TGC_ACT_GELU_TANH: {
            const float s = sigmoid_f32(2.0f * kGeluC * (z + kGeluA * z * z * z));
            return s + z * s * (1.0f - s) * 2.0f * kGeluC * (1.0f + 3.0f * kGeluA * z * z);
        }
        case TGC_ACT_SILU: {
            const float s = sigmoid_f32(z);
            return s * (1.0f + z * (1.0f - s));
        }
        default: return 1.0f;
    }
}

}  // namespace tgc
