// The activations of a linear layer's output and their derivatives, in fp32.
//
//   relu         max(u, 0)
//   gelu         u Phi(u), Phi the normal distribution
//   gelu_tanh    u s(2 sqrt(2 / pi) (u + 0.044715 u^3))      s(v) = 1 / (1 + exp(-v))
//   quick_gelu   u s(1.702 u)
//   silu         u s(u)
//
// An epilogue of a product over K terms has K / 32 issue slots an element (a tensor core takes 128 x 256 x 64 in
// 512 cycles, in which four schedulers issue for 32 elements each), so Phi has to be had for ten instructions:
//   Phi(-z) = exp(-z^2 / 2) t P(t),  t = 1 / (1 + 0.36 z),  z >= 0,
// with P of degree 6 fitted to erfcx(z / sqrt 2) / 2 over [0, 14] for the smallest largest relative error (reweighted least
// squares): 9e-7.  The exponential's argument is rounded to fp32, which makes up to 6.5e-6 of it at z = 13.  The exponential serves the
// density in the derivative.
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

// Everything is on pairs: packed fp32 arithmetic takes half the issue slots.  Exponentials and reciprocals have 16 lanes a clock
// and SM: two for each of the 128 x 256 elements of a tile's half take 4096 cycles, half of its products' time at K = 1024.
__device__ __forceinline__ float2 pair_of(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 fmul2(float2 x, float2 y) { return __fmul2_rn(x, y); }
__device__ __forceinline__ float2 rcp2(float2 x) { return make_float2(rcp_approx(x.x), rcp_approx(x.y)); }
__device__ __forceinline__ float2 exp2_2(float2 x) { return make_float2(ex2_approx(x.x), ex2_approx(x.y)); }

// Phi(-|u|); *e = exp(-u^2 / 2), z = |u|, cut to kActFar and never NaN: the elements of a pair share a reciprocal, and one that is
// NaN becomes it through e alone.
__device__ __forceinline__ float2 normal_tail(float2 u, float2* z_, float2* e) {
  const float2 z = make_float2(fminf(fabsf(u.x), kActFar), fminf(fabsf(u.y), kActFar));
  *z_ = z;
  // both reciprocals from one, of the product (the arguments lie between 1 and 25)
  const float2 d = ffma2(pair_of(0.36f), z, pair_of(1.f));
  const float2 t = fmul2(pair_of(rcp_approx(d.x * d.y)), make_float2(d.y, d.x));
  float2 p = ffma2(pair_of(0.0470557399f), t, pair_of(-0.17976281f));
  p = ffma2(p, t, pair_of(0.180951446f));
  p = ffma2(p, t, pair_of(0.0265510548f));
  p = ffma2(p, t, pair_of(0.139718652f));
  p = ffma2(p, t, pair_of(0.141772568f));
  p = ffma2(p, t, pair_of(0.143713042f));
  *e = exp2_2(fmul2(fmul2(u, u), pair_of(-0.5f * kLog2e)));
  return fmul2(fmul2(p, t), *e);
}

// s(c v)
__device__ __forceinline__ float2 sigmoid(float2 v, float c) {
  return rcp2(fadd2(exp2_2(fmul2(v, pair_of(-kLog2e * c))), pair_of(1.f)));
}

constexpr float kTanhB = 1.5957691216057308f;   // 2 sqrt(2 / pi)
constexpr float kTanhC = 0.044715f;

template <int ACT>
__device__ __forceinline__ float2 act_of(float2 u) {
  if (ACT == kActRelu) return make_float2(u.x < 0.f ? 0.f : u.x, u.y < 0.f ? 0.f : u.y);   // NaN stays
  if (ACT == kActGelu) {
    float2 z, e;
    const float2 q = normal_tail(u, &z, &e);
    // u - u Phi(-u) for u > 0, u Phi(u) below
    return ffma2(make_float2(-z.x, -z.y), q, make_float2(fmaxf(u.x, 0.f), fmaxf(u.y, 0.f)));
  }
  if (ACT == kActGeluTanh)
    return fmul2(u, sigmoid(fmul2(u, ffma2(fmul2(u, u), pair_of(kTanhC), pair_of(1.f))), kTanhB));
  if (ACT == kActQuickGelu) return fmul2(u, sigmoid(u, 1.702f));
  if (ACT == kActSilu) return fmul2(u, sigmoid(u, 1.f));
  return u;
}

template <int ACT>
__device__ __forceinline__ float2 act_slope(float2 u) {
  if (ACT == kActNone) return pair_of(1.f);
  if (ACT == kActRelu) return make_float2(u.x > 0.f ? 1.f : 0.f, u.y > 0.f ? 1.f : 0.f);
  if (ACT == kActGelu) {
    float2 z, e;
    const float2 q = normal_tail(u, &z, &e);
    // Phi + u exp(-u^2 / 2) / sqrt(2 pi)
    return ffma2(fmul2(make_float2(copysignf(z.x, u.x), copysignf(z.y, u.y)), pair_of(0.3989422804014327f)), e,
                 make_float2(u.x < 0.f ? q.x : 1.f - q.x, u.y < 0.f ? q.y : 1.f - q.y));
  }
  const float2 v = make_float2(max_nan(min_nan(u.x, kActFar), -kActFar), max_nan(min_nan(u.y, kActFar), -kActFar));
  // s + m s (1 - s), m = u times the slope of the sigmoid's argument
  float2 s, m;
  if (ACT == kActGeluTanh) {
    const float2 w = fmul2(v, v);
    s = sigmoid(fmul2(v, ffma2(w, pair_of(kTanhC), pair_of(1.f))), kTanhB);
    m = fmul2(fmul2(v, pair_of(kTanhB)), ffma2(w, pair_of(3.f * kTanhC), pair_of(1.f)));
  } else {
    constexpr float c = ACT == kActQuickGelu ? 1.702f : 1.f;
    s = sigmoid(v, c);
    m = fmul2(v, pair_of(c));
  }
  return ffma2(fmul2(m, s), ffma2(s, pair_of(-1.f), pair_of(1.f)), s);
}

// x[i] = act(x[i]), and x[i] *= act'(u[i]), for an even number of values
template <int ACT, int N>
__device__ __forceinline__ void act_all(float (&x)[N]) {
  #pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float2 y = act_of<ACT>(make_float2(x[i], x[i + 1]));
    x[i] = y.x;
    x[i + 1] = y.y;
  }
}
template <int ACT, int N>
__device__ __forceinline__ void slope_all(float (&x)[N], const float (&u)[N]) {
  #pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float2 y = fmul2(make_float2(x[i], x[i + 1]), act_slope<ACT>(make_float2(u[i], u[i + 1])));
    x[i] = y.x;
    x[i + 1] = y.y;
  }
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
