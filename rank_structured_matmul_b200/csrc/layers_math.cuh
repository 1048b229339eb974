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

// Two accuracies of each function. FAST serves the bf16 layers, whose results
// are rounded to 2^-9 of themselves at best: __expf and __fdividef (a few units
// in the last place of fp32) and Phi by the rational approximation of Abramowitz
// and Stegun, Handbook of Mathematical Functions, 7.1.26 (|error| <= 1.5e-7). A
// 256 x 256 tile's epilogue runs 256 of these per thread: with erfcf the ViT-L
// fc1 forward was bound by them (165 us, against 102 us for twice the product
// without an activation).

// The logistic function. exp(-z) may overflow to infinity (z < -88): the
// quotient is then 0, its value.
template <bool FAST>
__device__ __forceinline__ float sigmoid_f(float z) {
  return FAST ? __fdividef(1.f, 1.f + __expf(-z)) : 1.f / (1.f + expf(-z));
}

// Phi(z), and e = exp(-z^2 / 2) on the way. erfc keeps its relative accuracy for
// z << 0, where 1 + erf cancels. 7.1.26: erfc(x) = t (a1 + .. + a5 t^4) exp(-x^2)
// with t = 1 / (1 + p x), x >= 0.
template <bool FAST>
__device__ __forceinline__ float phi_f(float z, float& e) {
  if (!FAST) {
    e = expf(-0.5f * z * z);
    return 0.5f * erfcf(-z * kSqrtHalf);
  }
  const float x = fabsf(z) * kSqrtHalf;
  e = __expf(-0.5f * z * z);
  const float t = __fdividef(1.f, fmaf(0.3275911f, x, 1.f));
  float q = fmaf(1.061405429f, t, -1.453152027f);
  q = fmaf(q, t, 1.421413741f);
  q = fmaf(q, t, -0.284496736f);
  q = fmaf(q, t, 0.254829592f);
  const float tail = 0.5f * q * t * e;  // Phi(-|z|)
  return z < 0.f ? tail : 1.f - tail;
}

template <int ACT, bool FAST = false>
__device__ __forceinline__ float act_f(float z) {
  if (ACT == DYRA_ACT_RELU) return z < 0.f ? 0.f : z;  // NaN passes
  if (ACT == DYRA_ACT_GELU) {
    float e;
    return z * phi_f<FAST>(z, e);
  }
  if (ACT == DYRA_ACT_GELU_TANH)  // (1 + tanh u) / 2 = sigmoid(2 u)
    return z * sigmoid_f<FAST>(2.f * kTanhC * fmaf(kTanhA * z * z, z, z));
  if (ACT == DYRA_ACT_SILU) return z * sigmoid_f<FAST>(z);
  return z;
}

template <int ACT, bool FAST = false>
__device__ __forceinline__ float act_grad_f(float z) {
  if (ACT == DYRA_ACT_RELU) return z > 0.f ? 1.f : 0.f;
  if (ACT == DYRA_ACT_GELU) {
    float e;
    const float phi = phi_f<FAST>(z, e);
    return fmaf(z * kInvSqrt2Pi, e, phi);
  }
  if (ACT == DYRA_ACT_GELU_TANH) {
    const float p = sigmoid_f<FAST>(2.f * kTanhC * fmaf(kTanhA * z * z, z, z));
    const float du = 2.f * kTanhC * fmaf(3.f * kTanhA * z, z, 1.f);  // d(2u)/dz
    return fmaf(z * p * (1.f - p), du, p);
  }
  if (ACT == DYRA_ACT_SILU) {
    const float p = sigmoid_f<FAST>(z);
    return p * fmaf(z, 1.f - p, 1.f);
  }
  return 1.f;
}

// Whether a storage type takes the fast functions.
template <typename T>
constexpr bool kFastMath = sizeof(T) == 2;

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
