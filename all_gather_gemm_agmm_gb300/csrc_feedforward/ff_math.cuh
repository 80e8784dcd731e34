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

// A sum over rows, as float32 or rounded once.
template <bool kF16>
__device__ __forceinline__ void store_sum(void* out, int64_t col, float sum, int out_f32) {
  if (out_f32)
    static_cast<float*>(out)[col] = sum;
  else
    static_cast<uint16_t*>(out)[col] = pack1<kF16>(sum);
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kTanhScale2 = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kTanhCube = 0.044715f;

// Activations work on pairs, in packed arithmetic: the reciprocals and exponentials take turns
// of the same unit, two to a value at most, and the rest is half as many instructions.
__device__ __forceinline__ Two exp2_two(Two x) {
  const float2 v = halves(x);
  return two(exp2_approx(v.x), exp2_approx(v.y));
}
__device__ __forceinline__ Two rcp_two(Two x) {
  const float2 v = halves(x);
  return two(rcp_approx(v.x), rcp_approx(v.y));
}
// max(z, 0); a NaN stays one
__device__ __forceinline__ float positive(float z) {
  float y;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(y) : "f"(z));
  return y;
}
__device__ __forceinline__ Two positive_two(Two z) {
  const float2 v = halves(z);
  return two(positive(v.x), positive(v.y));
}
// max(z, -FLT_MAX): an fp16 product past -65504 was saved as -infinity, and times 0 it would be a NaN.
__device__ __forceinline__ float finite_below(float z) {
  float y;
  asm("max.NaN.f32 %0, %1, 0fff7fffff;" : "=f"(y) : "f"(z));
  return y;
}
__device__ __forceinline__ Two finite_below_two(Two z) {
  const float2 v = halves(z);
  return two(finite_below(v.x), finite_below(v.y));
}
__device__ __forceinline__ Two clamp_two(Two z, float most) {
  const float2 v = halves(z);
  return two(fminf(fmaxf(v.x, -most), most), fminf(fmaxf(v.y, -most), most));
}

// 1 / (1 + 2^x): of x = -z log2(e) the logistic function of z.  An infinite 2^x gives 0.
__device__ __forceinline__ Two logistic_two(Two x) { return rcp_two(add2(both(1.0f), exp2_two(x))); }

// Phi(-|z|), e^(-z^2 / 2) and x = min(|z|, 9), where Phi is the normal distribution:
//     Phi(-x) = 2^(P(x) - z^2 log2(e) / 2)
// with P fitted to log2(Phi(-x) e^(x^2/2)) at Chebyshev nodes of [0, 9], in u = 2 x / 9 - 1, where
// it is off by 2e-6: one exponential and nothing that cancels.  In float32 Phi is off by 2^-17.5
// of itself up to x = 9, by the exponent's rounding, and by 1e-19 beyond.
__device__ __forceinline__ Two normal_tail(Two z, Two& x, Two& gauss) {
  const float2 v = halves(z);
  x = two(fminf(fabsf(v.x), 9.0f), fminf(fabsf(v.y), 9.0f));
  const Two u = fma2(x, both(2.0f / 9.0f), both(-1.0f)), e = mul2(mul2(z, z), both(-0.5f * kLog2e));
  Two p = both(0.0035879954f);
  p = fma2(p, u, both(-0.0029788145f));
  p = fma2(p, u, both(-0.011076425f));
  p = fma2(p, u, both(0.019956289f));
  p = fma2(p, u, both(-0.02364965f));
  p = fma2(p, u, both(0.04836166f));
  p = fma2(p, u, both(-0.096737415f));
  p = fma2(p, u, both(0.171032f));
  p = fma2(p, u, both(-0.30213198f));
  p = fma2(p, u, both(0.56688064f));
  p = fma2(p, u, both(-1.3264755f));
  p = fma2(p, u, both(-3.559733f));
  gauss = exp2_two(e);
  return exp2_two(add2(p, e));
}

// -log2(e) times the argument 2 v of which gelu_tanh is the logistic function: 0.5 z (1 + tanh(v))
// is z / (1 + e^(-2 v)), and nothing cancels.
__device__ __forceinline__ Two tanh_exponent(Two z) {
  return mul2(mul2(z, fma2(mul2(z, z), both(kTanhCube), both(1.0f))), both(-kLog2e * kTanhScale2));
}

template <int kAct>
__device__ __forceinline__ Two activate(Two z) {
  if constexpr (kAct == kActRelu) return positive_two(z);
  if constexpr (kAct == kActSilu) return mul2(z, logistic_two(mul2(z, both(-kLog2e))));
  if constexpr (kAct == kActGelu) {
    // z Phi(z) = max(z, 0) - |z| Phi(-|z|); past 9 the second term is less than 2^-59
    Two x, gauss;
    const Two low = normal_tail(z, x, gauss);
    return fma2(mul2(x, both(-1.0f)), low, positive_two(z));
  }
  if constexpr (kAct == kActGeluTanh) return mul2(z, logistic_two(tanh_exponent(z)));
  return z;
}

// The activation and its derivative.  The bounds on z are where the second term of the
// derivative has long been 0 in float32: beyond them its factors would be infinity and 0.
template <int kAct>
__device__ __forceinline__ void activate_with_slope(Two z, Two& a, Two& slope) {
  a = z;
  slope = both(1.0f);
  if constexpr (kAct == kActRelu) {
    const float2 v = halves(z);
    a = positive_two(z);
    slope = two(v.x > 0.0f ? 1.0f : (v.x != v.x ? v.x : 0.0f), v.y > 0.0f ? 1.0f : (v.y != v.y ? v.y : 0.0f));
  } else if constexpr (kAct == kActSilu) {
    const Two s = logistic_two(mul2(z, both(-kLog2e))), rest = fma2(s, both(-1.0f), both(1.0f));
    a = mul2(finite_below_two(z), s);
    slope = mul2(s, fma2(clamp_two(z, 200.0f), rest, both(1.0f)));
  } else if constexpr (kAct == kActGelu) {
    Two x, gauss;
    const Two low = normal_tail(z, x, gauss);
    a = fma2(mul2(x, both(-1.0f)), low, positive_two(z));
    // Phi(z) = 1/2 + sign(z) (1/2 - Phi(-|z|)); the low end without that difference
    const float2 v = halves(z), l = halves(low);
    const Two phi = two(v.x > 0.0f ? 1.0f - l.x : l.x, v.y > 0.0f ? 1.0f - l.y : l.y);
    slope = fma2(clamp_two(z, 20.0f), mul2(gauss, both(kInvSqrt2Pi)), phi);
  } else if constexpr (kAct == kActGeluTanh) {
    const Two b = clamp_two(z, 20.0f), s = logistic_two(tanh_exponent(z)), rest = fma2(s, both(-1.0f), both(1.0f));
    a = mul2(finite_below_two(z), s);
    const Two dv = mul2(fma2(mul2(b, b), both(3.0f * kTanhCube), both(1.0f)), both(kTanhScale2));
    slope = fma2(mul2(b, mul2(s, rest)), dv, s);
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
