// The elementwise end of a linear and its derivative, shared by the GEMM's
// epilogue, the few-token reduction and the gradient kernel.
#pragma once

#include <type_traits>

#include "device.h"

namespace qlora {

// f(std::integral_constant<int, act>) for a launch's (uniform) activation, so
// that its choice stays outside the element loops.
template <class F>
__device__ __forceinline__ void with_act(int act, F &&f) {
  switch (act) {
    case kActRelu: f(std::integral_constant<int, kActRelu>{}); break;
    case kActGelu: f(std::integral_constant<int, kActGelu>{}); break;
    case kActGeluTanh: f(std::integral_constant<int, kActGeluTanh>{}); break;
    case kActSilu: f(std::integral_constant<int, kActSilu>{}); break;
    default: f(std::integral_constant<int, kActNone>{}); break;
  }
}

// 1 / (1 + e^-v): e^-v is infinite below -88.8 and the quotient 0.
__device__ __forceinline__ float sigmoid(float v) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504088896340736f * v));
}

constexpr float kGeluTwo = 1.59576912160573081f;     // 2 sqrt(2 / pi)
constexpr float kGeluCube = 0.044715f;

// Phi(z), within 3e-7, and e = e^(-z^2 / 2): erfc(x) =
// e^(-x^2) (a1 t + ... + a5 t^5), t = 1 / (1 + 0.3275911 x), of Abramowitz and
// Stegun, Handbook of Mathematical Functions, 7.1.26, for x = |z| / sqrt 2.  It
// shares e with the derivative and takes 15 operations where erfcf takes 60
// (the forward of 2048 x 4096 x 11008 with it 263 us, so 229).
__device__ __forceinline__ float normal_cdf(float z, float &e) {
  const float a = fabsf(z);
  const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.231641888f, a, 1.0f));
  e = __builtin_amdgcn_exp2f(-0.72134752044448170f * z * z);
  float s = __builtin_fmaf(1.061405429f, t, -1.453152027f);
  s = __builtin_fmaf(s, t, 1.421413741f);
  s = __builtin_fmaf(s, t, -0.284496736f);
  s = __builtin_fmaf(s, t, 0.254829592f);
  const float tail = 0.5f * s * t * e;
  return z < 0.0f ? tail : 1.0f - tail;
}

// act(z).  (1 + tanh v) / 2 = sigmoid(2 v) keeps the digits of the left tail,
// where 1 + tanh cancels.
template <int act>
__device__ __forceinline__ float activated(float z) {
  if (act == kActRelu) return z <= 0.0f ? 0.0f : z;          // (a NaN stays one)
  if (act == kActSilu) return z * sigmoid(z);
  if (act == kActGeluTanh) return z * sigmoid(kGeluTwo * __builtin_fmaf(kGeluCube * z * z, z, z));
  if (act == kActGelu) {
    float e;
    return z * normal_cdf(z, e);
  }
  return z;
}

// act(z) and act'(z).
template <int act>
__device__ __forceinline__ void activated(float z, float &f, float &df) {
  f = z;
  df = 1.0f;
  if (act == kActRelu) {
    f = z <= 0.0f ? 0.0f : z;
    df = z <= 0.0f ? 0.0f : 1.0f;
  }
  if (act == kActSilu) {
    const float s = sigmoid(z);
    f = z * s;
    df = __builtin_fmaf(f, 1.0f - s, s);
  }
  if (act == kActGeluTanh) {
    const float s = sigmoid(kGeluTwo * __builtin_fmaf(kGeluCube * z * z, z, z));
    f = z * s;
    // past 30, s (1 - s) is 0 and z^2 may be infinite
    const float c = fminf(fabsf(z), 30.0f);
    df = __builtin_fmaf(f * (1.0f - s),
                        kGeluTwo * __builtin_fmaf(3.0f * kGeluCube * c, c, 1.0f), s);
  }
  if (act == kActGelu) {
    float e;
    const float cdf = normal_cdf(z, e);
    f = z * cdf;
    df = __builtin_fmaf(0.39894228040143268f * z, e, cdf);   // z e / sqrt(2 pi)
  }
}

// 16 bytes as floats: 8 bf16 or 4 fp32 values.
template <bool BF16>
constexpr int kWide = BF16 ? 8 : 4;

template <bool BF16>
__device__ __forceinline__ void widen(u32x4_t u, float (&e)[kWide<BF16>]) {
  if constexpr (BF16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      e[2 * i] = bf16_lo_to_f32(u[i]);
      e[2 * i + 1] = bf16_hi_to_f32(u[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = __uint_as_float(u[i]);
  }
}

template <bool BF16>
__device__ __forceinline__ u32x4_t narrow(const float (&e)[kWide<BF16>]) {
  if constexpr (BF16)
    return u32x4_t{pack_bf16x2(e[0], e[1]), pack_bf16x2(e[2], e[3]), pack_bf16x2(e[4], e[5]),
                   pack_bf16x2(e[6], e[7])};
  else
    return u32x4_t{__float_as_uint(e[0]), __float_as_uint(e[1]), __float_as_uint(e[2]),
                   __float_as_uint(e[3])};
}

}  // namespace qlora
