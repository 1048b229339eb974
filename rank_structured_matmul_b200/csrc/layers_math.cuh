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
// are rounded to 2^-8 of themselves: the hardware's approximate 2^x and
// reciprocal (about 2^-22), and for the normal distribution
//   Phi(-x) = 2^P(x), x >= 0,
// with P a polynomial of degree 10. log2 Phi(-x) is nearly a parabola, so the
// tail keeps its relative accuracy where a polynomial of that degree times
// exp(-x^2 / 2) loses it. P is fitted by linear programming over 3000 points of
// [0, 13.05] so that the largest of |error of Phi| / 4e-7 and |error of Phi| /
// (2^-12 Phi) is least. Evaluated in fp32, Phi(-x) is off by at most 3.4e-7 and by
// at most 2.1e-4 of itself (a nineteenth of half a bf16 step), until it falls below
// 2^-126 at x = 12.95, where the instruction flushes it to zero. An epilogue
// thread runs 128 of these per 256 x 256 tile, of one special-function step each;
// a slope takes a second one for exp(-x^2 / 2) (backward of 6432 x 1024 -> 4096:
// 139.3 us; 137.7 with an exp(-x^2 / 2) times a polynomial that was off by a fifth of
// itself at x = 5).

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

// x = min(|z|, 13.5); returns Phi(-x). At 13.5 it is zero (P < -136), so that z far
// out gives z or 0 up to the largest finite values, and so is exp(-x^2 / 2).
constexpr float kPhiMax = 13.5f;
constexpr int kPhiDegree = 10;
__device__ __forceinline__ float phi_poly(int k) {
  constexpr float c[kPhiDegree + 1] = {
      -3.65319136e-10f, 1.98518766e-08f,  -3.99899079e-07f, 2.70403029e-06f,
      2.84406215e-05f,  -7.75194087e-04f, 8.07588827e-03f,  -5.33244498e-02f,
      -4.58895057e-01f, -1.15114748e+00f, -9.99999106e-01f};
  return c[k];
}
__device__ __forceinline__ float phi_tail_fast(float z, float& x) {
  x = fminf(fabsf(z), kPhiMax);
  float q = phi_poly(0);
#pragma unroll
  for (int k = 1; k <= kPhiDegree; ++k) q = fmaf(q, x, phi_poly(k));
  return exp2_approx(q);
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

// Phi(-|z|) of two values (phi_tail_fast), and x = min(|z|, kPhiMax).
__device__ __forceinline__ f32x2 phi_tail2(float z0, float z1, f32x2& x) {
  x = pair(fminf(fabsf(z0), kPhiMax), fminf(fabsf(z1), kPhiMax));
  f32x2 q = pair(phi_poly(0), phi_poly(0));
#pragma unroll
  for (int k = 1; k <= kPhiDegree; ++k) q = fma2(q, x, pair(phi_poly(k), phi_poly(k)));
  const float2 h = halves(q);
  return pair(exp2_approx(h.x), exp2_approx(h.y));
}

// act_f<ACT, true> of eight values; the GELU's polynomial two values at a time,
// which nearly halves its instructions.
template <int ACT>
__device__ __forceinline__ void act8(float (&v)[8]) {
  if constexpr (ACT == DYRA_ACT_GELU) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      f32x2 x;
      const f32x2 tail = phi_tail2(v[i], v[i + 1], x);
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
      f32x2 x;
      const float2 tail = halves(phi_tail2(v[i], v[i + 1], x));
      const float2 h = halves(mul2(mul2(x, pair(-0.5f * kLog2e, -0.5f * kLog2e)), x));
      const f32x2 e = pair(exp2_approx(h.x), exp2_approx(h.y));
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
