// ff_math.cuh -- 16-bit packing and the activations with their derivatives.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ff_params.h"

namespace agmm {
namespace ff {

template <bool kF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (kF16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

template <bool kF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if constexpr (kF16)
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  else
    return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}

template <bool kF16>
__device__ __forceinline__ uint16_t pack1(float x) {
  return (uint16_t)(pack2<kF16>(x, 0.0f) & 0xffffu);
}

template <bool kF16>
__device__ __forceinline__ float unpack1(uint16_t w) {
  return unpack2<kF16>((uint32_t)w).x;
}

template <bool kF16>
__device__ __forceinline__ void unpack8(const uint4& u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2<kF16>(w[i]);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

template <bool kF16>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack2<kF16>(x[0], x[1]), pack2<kF16>(x[2], x[3]), pack2<kF16>(x[4], x[5]), pack2<kF16>(x[6], x[7]));
}

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

// Two float32 values in one 64-bit register pair, for the packed instructions.
using Two = uint64_t;
__device__ __forceinline__ Two two(float lo, float hi) {
  Two r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ Two both(float x) { return two(x, x); }
__device__ __forceinline__ float2 halves(Two x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ Two add2(Two a, Two b) {
  Two r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Two mul2(Two a, Two b) {
  Two r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ float sum2(Two x) {
  const float2 v = halves(x);
  return v.x + v.y;
}

// 8 values of 16 bits as four pairs, and back.
template <bool kF16>
__device__ __forceinline__ void widen(const uint4& u, Two (&x)[4]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack2<kF16>(w[i]);
    x[i] = two(f.x, f.y);
  }
}
template <bool kF16>
__device__ __forceinline__ uint4 narrow(const Two (&x)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = halves(x[i]);
    w[i] = pack2<kF16>(f.x, f.y);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kTanhScale2 = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kTanhCube = 0.044715f;

// 1 / (1 + e^-z).  A z so low that e^-z is infinite gives 0.
__device__ __forceinline__ float sigmoid(float z) { return rcp_approx(1.0f + exp2_approx(-kLog2e * z)); }

// The normal distribution Phi(z), and e^(-z^2 / 2).  For z <= 0
//     Phi(z) = t 2^(P(t) - z^2 log2(e) / 2),   t = 1 / (1 + 0.35 |z|),
// with P fitted to log2(Phi e^(z^2/2) / t) at Chebyshev nodes of |z| <= 13.5, where it is off by
// 1e-6: no cancellation where Phi is small, one reciprocal and one exponential.  In float32
// Phi is off by 2^-18.5 of itself up to |z| = 8, by the exponent's rounding.  (erfcf took 193 us
// for 4096 tokens, k 2560, n 5120, where the product alone takes a third.)
__device__ __forceinline__ float normal(float z, float& gauss) {
  const float x = fabsf(z), t = rcp_approx(fmaf(0.35f, x, 1.0f)), e = x * x * (-0.5f * kLog2e);
  float p = -0.27522552f;
  p = fmaf(p, t, 1.1202697f);
  p = fmaf(p, t, -1.5381097f);
  p = fmaf(p, t, 0.60237956f);
  p = fmaf(p, t, -0.09033469f);
  p = fmaf(p, t, 0.5817873f);
  p = fmaf(p, t, 1.4394445f);
  p = fmaf(p, t, -2.840212f);
  gauss = exp2_approx(e);
  const float low = t * exp2_approx(p + e);
  return z > 0.0f ? 1.0f - low : low;
}

// The tanh form of z Phi(z), 0.5 z (1 + tanh(v)), is z sigmoid(2 v): nothing cancels.
template <int kAct>
__device__ __forceinline__ float activate(float z) {
  if constexpr (kAct == kActRelu) return z < 0.0f ? 0.0f : z;  // a NaN stays one
  if constexpr (kAct == kActSilu) return z * sigmoid(z);
  if constexpr (kAct == kActGelu) {
    float gauss;
    return z * normal(z, gauss);
  }
  if constexpr (kAct == kActGeluTanh) return z * sigmoid(kTanhScale2 * (z + kTanhCube * z * z * z));
  return z;
}

// The activation and its derivative.  The bounds on z are where the second term of the
// derivative has long been 0 in float32: beyond them its factors would be infinity and 0.
template <int kAct>
__device__ __forceinline__ void activate_with_slope(float z, float& a, float& slope) {
  a = z;
  slope = 1.0f;
  if constexpr (kAct == kActRelu) {
    a = z < 0.0f ? 0.0f : z;
    slope = z > 0.0f ? 1.0f : (z != z ? z : 0.0f);
  } else if constexpr (kAct == kActSilu) {
    const float s = sigmoid(z), b = fminf(fmaxf(z, -200.0f), 200.0f);
    a = z * s;
    slope = s * (1.0f + b * (1.0f - s));
  } else if constexpr (kAct == kActGelu) {
    float gauss;
    const float phi = normal(z, gauss), b = fminf(fmaxf(z, -20.0f), 20.0f);
    a = z * phi;
    slope = phi + b * (kInvSqrt2Pi * gauss);
  } else if constexpr (kAct == kActGeluTanh) {
    const float b = fminf(fmaxf(z, -20.0f), 20.0f);
    const float s = sigmoid(kTanhScale2 * (z + kTanhCube * z * z * z));
    a = z * s;
    slope = s + b * s * (1.0f - s) * (kTanhScale2 * (1.0f + 3.0f * kTanhCube * b * b));
  }
}

// Calls f with the activation as a compile-time constant.
template <class F>
__device__ __forceinline__ void with_activation(int act, F&& f) {
  switch (act) {
    case kActRelu: f(std::integral_constant<int, kActRelu>()); break;
    case kActSilu: f(std::integral_constant<int, kActSilu>()); break;
    case kActGelu: f(std::integral_constant<int, kActGelu>()); break;
    case kActGeluTanh: f(std::integral_constant<int, kActGeluTanh>()); break;
    default: f(std::integral_constant<int, kActNone>()); break;
  }
}

}  // namespace ff
}  // namespace agmm
