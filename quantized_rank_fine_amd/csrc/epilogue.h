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

// c[N - 1] t^(N - 1) + ... + c[0].
template <int N>
__device__ __forceinline__ float polynomial(const float (&c)[N], float t) {
  float s = c[N - 1];
#pragma unroll
  for (int i = N - 2; i >= 0; --i) s = __builtin_fmaf(s, t, c[i]);
  return s;
}

// Phi(z) and e = e^(-z^2 / 2).  The left tail is a multiple of e, so that its digits
// are kept, Phi(-x) = e R(x), and R a polynomial without constant term in t = 1 / (1 +
// p x); the coefficients have the least largest error relative to R over x <= 13.5
// (past which e is 0), found by least squares reweighted until the error is even.
// An argument's rounding moves e, and erfc as well, by about z^2 2^-24 of itself.
//   bf16 results: 8 coefficients, 1.3e-7.
//   fp32 results: 9, 3.2e-8, and for |z| < 1, where Phi - 1/2 has no tail's digits to
//     lose, 1/2 + z P(z^2) within 8e-9.  Phi is within 8e-8, and within 4.3e-7 of
//     itself down to z = -2, 8.2e-7 to -4 (emulated; erfc without any error of its
//     own, of the rounded argument: 4.6e-8, 3.2e-7, 1.1e-6).
// They share e with the derivative and take 18 and 27 operations where erfcf takes 60:
// 2048 x 4096 x 11008 with GELU and z saved, fp32: 277 us, with erfcf 289 (with the
// tanh form 250; bf16 235 and 224); the gradient of 2048 x 11008 fp32: 47.9, with
// erfcf 54.0.
template <bool BF16>
__device__ __forceinline__ float normal_cdf(float z, float &e) {
  const float w = z * z, x = fabsf(z);
  e = __builtin_amdgcn_exp2f(-0.72134752044448170f * w);
  if constexpr (BF16) {
    constexpr float c[] = {0.119626395f, 0.12079836f,   0.099637516f, 0.12946913f,
                           -0.055393703f, 0.20820644f, -0.15827592f, 0.03593172f};
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3f, x, 1.0f));
    const float tail = polynomial(c, t) * t * e;
    return z < 0.0f ? tail : 1.0f - tail;
  } else {
    constexpr float c[] = {0.13962157f,  0.13985908f,  0.11985244f, 0.10543294f, -0.022937143f,
                           0.15892929f, -0.25550455f, 0.14387223f, -0.029125864f};
    constexpr float m[] = {0.3989422f, -0.06648873f, 0.009964167f, -0.0011653508f, 9.246837e-05f};
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.35f, x, 1.0f));
    const float tail = polynomial(c, t) * t * e;
    const float outer = z < 0.0f ? tail : 1.0f - tail;
    return x < 1.0f ? __builtin_fmaf(z, polynomial(m, w), 0.5f) : outer;
  }
}

// act(z) for a result in bf16 or fp32.  (1 + tanh v) / 2 = sigmoid(2 v) keeps the
// digits of the left tail, where 1 + tanh cancels.
template <int act, bool BF16>
__device__ __forceinline__ float activated(float z) {
  if (act == kActRelu) return z <= 0.0f ? 0.0f : z;          // (a NaN stays one)
  if (act == kActSilu) return z * sigmoid(z);
  if (act == kActGeluTanh) return z * sigmoid(kGeluTwo * __builtin_fmaf(kGeluCube * z * z, z, z));
  if (act == kActGelu) {
    float e;
    return z * normal_cdf<BF16>(z, e);
  }
  return z;
}

// act(z) and act'(z).
template <int act, bool BF16>
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
    const float cdf = normal_cdf<BF16>(z, e);
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
