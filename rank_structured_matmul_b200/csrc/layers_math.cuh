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
constexpr float kLog2e = 1.4426950408889634f;

// Two accuracies of each function. FAST serves the bf16 layers, whose results
// are rounded to 2^-8 of themselves at best: the hardware's approximate 2^x and
// reciprocal (about 2^-22), and for the normal distribution
//   Phi(-x) = exp(-x^2 / 2) q(x),  q(x) = erfcx(x / sqrt 2) / 2, x >= 0,
// with q a polynomial of degree 8, the minimax fit of q on [0, 6] under the
// weight exp(-x^2 / 2) (by linear programming over 4000 points): Phi is off by at
// most 2.8e-6. An epilogue thread runs 128 of these per 256 x 256 tile. On the
// ViT-L fc1 forward (40 us without an activation) the GELU with erfcf took 125 us
// more, with a rational formula of two special-function steps 15, in this form 7.

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The logistic function. exp(-z) may overflow to infinity (z < -88): the
// quotient is then 0, its value.
template <bool FAST>
__device__ __forceinline__ float sigmoid_f(float z) {
  return FAST ? rcp_approx(1.f + exp2_approx(-kLog2e * z)) : 1.f / (1.f + expf(-z));
}

// x = min(|z|, 16), e = exp(-x^2 / 2); returns Phi(-x). At 16 the polynomial is still
// finite and e is below the smallest normal number, which the instruction flushes to
// zero: z e is zero for the largest finite z too. (The polynomial is no fit beyond 6,
// where e < 2e-8 makes its error nothing.)
constexpr float kPhiMax = 16.f;
__device__ __forceinline__ float phi_poly(int k) {
  constexpr float c[9] = {1.85581324e-5f,  -3.78031295e-4f, 3.25897020e-3f,
                          -1.60708737e-2f, 5.25960136e-2f,  -1.27570483e-1f,
                          2.48509570e-1f,  -3.98784939e-1f, 4.99997257e-1f};
  return c[k];
}
__device__ __forceinline__ float phi_tail_fast(float z, float& x) {
  x = fminf(fabsf(z), kPhiMax);
  const float e = exp2_approx(-0.5f * kLog2e * x * x);
  float q = phi_poly(0);
#pragma unroll
  for (int k = 1; k < 9; ++k) q = fmaf(q, x, phi_poly(k));
  return q * e;
}

template <int ACT, bool FAST = false>
__device__ __forceinline__ float act_f(float z) {
  const float relu = z < 0.f ? 0.f : z;  // NaN passes
  if (ACT == DYRA_ACT_RELU) return relu;
  if (ACT == DYRA_ACT_GELU) {
    if (!FAST) return z * (0.5f * erfcf(-z * kSqrtHalf));  // erfc: exact for z << 0
    float x;
    const float tail = phi_tail_fast(z, x);
    return fmaf(-x, tail, relu);  // z Phi(z) = max(z, 0) - |z| Phi(-|z|)
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
    static_assert(!FAST || ACT != DYRA_ACT_GELU, "act_grad8");
    const float e = expf(-0.5f * z * z), phi = 0.5f * erfcf(-z * kSqrtHalf);
    return fmaf(z * kInvSqrt2Pi, e, phi);
  }
  if (ACT == DYRA_ACT_GELU_TANH) {
    const float p = sigmoid_f<FAST>(2.f * kTanhC * fmaf(kTanhA * z * z, z, z));
    // d(2u)/dz, kept finite: p (1 - p) is zero long before 1e4
    const float c = fminf(fabsf(z), 1e4f);
    const float du = 2.f * kTanhC * fmaf(3.f * kTanhA * c, c, 1.f);
    return fmaf(z * p * (1.f - p), du, p);
  }
  if (ACT == DYRA_ACT_SILU) {
    const float p = sigmoid_f<FAST>(z);
    return p * fmaf(z, 1.f - p, 1.f);
  }
  return 1.f;
}

// Two fp32 operations in one instruction, on the halves of 64-bit registers.
typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 halves(f32x2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Phi(-|z|) of two values (phi_tail_fast): x = min(|z|, kPhiMax) and e = exp(-x^2 / 2)
// too.
__device__ __forceinline__ f32x2 phi_tail2(float z0, float z1, f32x2& x, f32x2& e) {
  x = pair(fminf(fabsf(z0), kPhiMax), fminf(fabsf(z1), kPhiMax));
  const float2 h = halves(mul2(mul2(x, pair(-0.5f * kLog2e, -0.5f * kLog2e)), x));
  e = pair(exp2_approx(h.x), exp2_approx(h.y));
  f32x2 q = pair(phi_poly(0), phi_poly(0));
#pragma unroll
  for (int k = 1; k < 9; ++k) q = fma2(q, x, pair(phi_poly(k), phi_poly(k)));
  return mul2(q, e);
}

// act_f<ACT, true> of eight values; the GELU's polynomial two values at a time,
// which nearly halves its instructions.
template <int ACT>
__device__ __forceinline__ void act8(float (&v)[8]) {
  if constexpr (ACT == DYRA_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      f32x2 x, e;
      const f32x2 tail = phi_tail2(v[i], v[i + 1], x, e);
      const f32x2 minus = mul2(x, pair(-1.f, -1.f));
      const float2 y = halves(fma2(minus, tail, pair(v[i] < 0.f ? 0.f : v[i],
                                                     v[i + 1] < 0.f ? 0.f : v[i + 1])));
      v[i] = y.x;
      v[i + 1] = y.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = act_f<ACT, true>(v[i]);
  }
}

// The slopes of eight values, fast, in the same way.
template <int ACT>
__device__ __forceinline__ void act_grad8(float (&v)[8]) {
  if constexpr (ACT == DYRA_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      f32x2 x, e;
      const float2 tail = halves(phi_tail2(v[i], v[i + 1], x, e));
      const f32x2 phi = pair(v[i] < 0.f ? tail.x : 1.f - tail.x,
                             v[i + 1] < 0.f ? tail.y : 1.f - tail.y);
      const float2 y = halves(fma2(mul2(pair(v[i], v[i + 1]), pair(kInvSqrt2Pi, kInvSqrt2Pi)), e,
                                   phi));
      v[i] = y.x;
      v[i + 1] = y.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = act_grad_f<ACT, true>(v[i]);
  }
}

// Whether a storage type takes the fast functions.
template <typename T>
constexpr bool kFastMath = sizeof(T) == 2;

// A constant as an argument. with_act calls f with a tag for the run-time activation, so that loops over values
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
