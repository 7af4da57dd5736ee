// The activations of a linear layer's output and their derivatives, in fp32.
//
//   relu         max(u, 0)
//   gelu         u Phi(u), Phi the normal distribution
//   gelu_tanh    u s(2 sqrt(2 / pi) (u + 0.044715 u^3))      s(v) = 1 / (1 + exp(-v))
//   quick_gelu   u s(1.702 u)
//   silu         u s(u)
//
// An epilogue of a product over K terms has about K / 2 issue slots an element (a tensor core takes 128 x 256 x 64 in
// 512 cycles, four schedulers issue for 32 elements each), so Phi has to be had for a dozen instructions:
//   Phi(-z) = exp(-z^2 / 2) t P(t),  t = 1 / (1 + 0.36 z),  z >= 0,
// with P of degree 6 fitted to erfcx(z / sqrt 2) / 2 over [0, 14] for the smallest largest relative error (reweighted least
// squares): 9e-7, in the tail too.  Its exponential serves the density in the derivative.
#pragma once
#include <type_traits>

#include "common.cuh"

namespace dera {

enum : int { kActNone = 0, kActRelu = 1, kActGelu = 2, kActGeluTanh = 3, kActQuickGelu = 4, kActSilu = 5, kActs = 6 };

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The smaller (larger) of two; NaN if x is.
__device__ __forceinline__ float min_nan(float x, float y) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float max_nan(float x, float y) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}

// Past it every activation here is u or 0 and every slope 1 or 0 to fp32: arguments are cut to it where an infinite one
// would be multiplied by zero.
constexpr float kActFar = 64.f;

// Phi(-z) for z >= 0; *e = exp(-z^2 / 2).
__device__ __forceinline__ float normal_tail(float z, float* e) {
  const float t = rcp_approx(fmaf(0.36f, z, 1.f));
  float p = 0.0470557399f;
  p = fmaf(p, t, -0.17976281f);
  p = fmaf(p, t, 0.180951446f);
  p = fmaf(p, t, 0.0265510548f);
  p = fmaf(p, t, 0.139718652f);
  p = fmaf(p, t, 0.141772568f);
  p = fmaf(p, t, 0.143713042f);
  *e = ex2_approx(-0.5f * kLog2e * (z * z));
  return p * t * *e;
}

__device__ __forceinline__ float sigmoid(float v) { return rcp_approx(1.f + ex2_approx(-kLog2e * v)); }

constexpr float kTanhB = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kTanhC = 0.044715f;

template <int ACT>
__device__ __forceinline__ float act_of(float u) {
  if (ACT == kActRelu) return u < 0.f ? 0.f : u;   // NaN stays
  if (ACT == kActGelu) {
    float e;
    const float z = min_nan(fabsf(u), kActFar);
    return fmaf(-z, normal_tail(z, &e), fmaxf(u, 0.f));   // u - u Phi(-u) for u > 0, u Phi(u) below
  }
  if (ACT == kActGeluTanh) return u * sigmoid(kTanhB * u * fmaf(kTanhC * u, u, 1.f));
  if (ACT == kActQuickGelu) return u * sigmoid(1.702f * u);
  if (ACT == kActSilu) return u * sigmoid(u);
  return u;
}

template <int ACT>
__device__ __forceinline__ float act_slope(float u) {
  if (ACT == kActNone) return 1.f;
  if (ACT == kActRelu) return u > 0.f ? 1.f : 0.f;
  const float v = max_nan(min_nan(u, kActFar), -kActFar);
  if (ACT == kActGelu) {
    float e;
    const float q = normal_tail(fabsf(v), &e);
    return fmaf(v * 0.3989422804014327f, e, v < 0.f ? q : 1.f - q);   // Phi + u exp(-u^2 / 2) / sqrt(2 pi)
  }
  if (ACT == kActGeluTanh) {
    const float s = sigmoid(kTanhB * v * fmaf(kTanhC * v, v, 1.f));
    return fmaf(kTanhB * v * fmaf(3.f * kTanhC * v, v, 1.f), s * (1.f - s), s);
  }
  if (ACT == kActQuickGelu) {
    const float s = sigmoid(1.702f * v);
    return fmaf(1.702f * v, s * (1.f - s), s);
  }
  const float s = sigmoid(v);
  return fmaf(v, s * (1.f - s), s);
}

// f.template operator()<ACT>() for the activation `act` (kActNone too): a switch outside of a loop over elements.
template <class F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  switch (act) {
    case kActRelu: f(std::integral_constant<int, kActRelu>()); break;
    case kActGelu: f(std::integral_constant<int, kActGelu>()); break;
    case kActGeluTanh: f(std::integral_constant<int, kActGeluTanh>()); break;
    case kActQuickGelu: f(std::integral_constant<int, kActQuickGelu>()); break;
    case kActSilu: f(std::integral_constant<int, kActSilu>()); break;
    default: f(std::integral_constant<int, kActNone>()); break;
  }
}

}  // namespace dera
