// layers_math.cuh - activations and their derivatives, in fp32, and the
// conversions between storage types and fp32.
#pragma once

#include <cuda_bf16.h>

#include "dyra_layers.h"

namespace dyra {

__device__ __forceinline__ float load_f(float v) { return v; }
__device__ __forceinline__ float load_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T store_f(float v);
template <>
__device__ __forceinline__ float store_f<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ __nv_bfloat16 store_f<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

constexpr float kSqrtHalf = 0.70710678118654752f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kTanhC = 0.79788456080286536f;  // sqrt(2 / pi)
constexpr float kTanhA = 0.044715f;

// The logistic function. exp(-z) may overflow to infinity (z < -88): 1 / inf
// = 0 is then the value.
__device__ __forceinline__ float sigmoid_f(float z) { return 1.f / (1.f + expf(-z)); }

// Phi(z) = erfc(-z / sqrt 2) / 2 keeps its relative accuracy for z << 0, where
// 1 + erf cancels; the gelu of a large negative z is then exact to rounding.
template <int ACT>
__device__ __forceinline__ float act_f(float z) {
  if (ACT == DYRA_ACT_RELU) return z < 0.f ? 0.f : z;  // NaN passes
  if (ACT == DYRA_ACT_GELU) return 0.5f * z * erfcf(-z * kSqrtHalf);
  if (ACT == DYRA_ACT_GELU_TANH)  // (1 + tanh u) / 2 = sigmoid(2 u)
    return z * sigmoid_f(2.f * kTanhC * fmaf(kTanhA * z * z, z, z));
  if (ACT == DYRA_ACT_SILU) return z * sigmoid_f(z);
  return z;
}

template <int ACT>
__device__ __forceinline__ float act_grad_f(float z) {
  if (ACT == DYRA_ACT_RELU) return z > 0.f ? 1.f : 0.f;
  if (ACT == DYRA_ACT_GELU)
    return fmaf(z * kInvSqrt2Pi, expf(-0.5f * z * z), 0.5f * erfcf(-z * kSqrtHalf));
  if (ACT == DYRA_ACT_GELU_TANH) {
    const float p = sigmoid_f(2.f * kTanhC * fmaf(kTanhA * z * z, z, z));
    const float du = 2.f * kTanhC * fmaf(3.f * kTanhA * z, z, 1.f);  // d(2u)/dz
    return fmaf(z * p * (1.f - p), du, p);
  }
  if (ACT == DYRA_ACT_SILU) {
    const float p = sigmoid_f(z);
    return p * fmaf(z, 1.f - p, 1.f);
  }
  return 1.f;
}

// Calls f with a tag for the run-time activation, so that loops over values
// hold one activation's code.
template <int V>
struct ActTag {
  static constexpr int value = V;
};
template <class F>
__device__ __forceinline__ void with_act(int act, const F& f) {
  switch (act) {
    case DYRA_ACT_RELU: f(ActTag<DYRA_ACT_RELU>()); break;
    case DYRA_ACT_GELU: f(ActTag<DYRA_ACT_GELU>()); break;
    case DYRA_ACT_GELU_TANH: f(ActTag<DYRA_ACT_GELU_TANH>()); break;
    case DYRA_ACT_SILU: f(ActTag<DYRA_ACT_SILU>()); break;
    default: f(ActTag<DYRA_ACT_NONE>()); break;
  }
}
// The same on the host, around launches.
template <class F>
inline void with_act_host(int act, const F& f) {
  switch (act) {
    case DYRA_ACT_RELU: f(ActTag<DYRA_ACT_RELU>()); break;
    case DYRA_ACT_GELU: f(ActTag<DYRA_ACT_GELU>()); break;
    case DYRA_ACT_GELU_TANH: f(ActTag<DYRA_ACT_GELU_TANH>()); break;
    case DYRA_ACT_SILU: f(ActTag<DYRA_ACT_SILU>()); break;
    default: f(ActTag<DYRA_ACT_NONE>()); break;
  }
}

}  // namespace dyra
