// The activations of the products' epilogues and their slopes.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/ozk.h"

namespace ozk {

template <typename A>
struct ActConst {
  static constexpr A kRsqrt2 = (A)0.70710678118654752440;       // 2^(-1/2)
  static constexpr A kRsqrt2Pi = (A)0.39894228040143267794;     // (2 pi)^(-1/2)
  static constexpr A kTanhScale = (A)1.59576912160573071175;    // 2 (2 / pi)^(1/2)
  static constexpr A kTanhCubic = (A)0.044715;
  static constexpr A kLog2e = (A)1.44269504088896340736;
  static constexpr A kLog2eLow = (A)(1.44269504088896340736 - (double)kLog2e);
  static constexpr A kLn2 = (A)0.69314718055994530942;
};

// gelu z Phi(z) with Phi(z) = erfc(-z / sqrt 2) / 2 (no cancellation in the lower tail);
// gelu_tanh z (1 + tanh u) / 2 = z / (1 + exp(-2 u)), u = (2 / pi)^(1/2) (z + 0.044715 z^3);
// silu z / (1 + exp(-z)).  A NaN stays NaN.
__device__ __forceinline__ double activate(double z, int act) {
  typedef ActConst<double> K;
  switch (act) {
    case OZK_ACT_RELU:
      return z < 0.0 ? 0.0 : z;
    case OZK_ACT_GELU:
      return 0.5 * z * erfc(-z * K::kRsqrt2);
    case OZK_ACT_GELU_TANH:
      return z / (1.0 + exp(-K::kTanhScale * (z + K::kTanhCubic * z * z * z)));
    case OZK_ACT_SILU:
      return z / (1.0 + exp(-z));
    default:
      return z;
  }
}

// The same for the int8 layer, whose epilogue is bound by these instructions, in two forms: for
// outputs of 16 bits, and (kFull) for fp32 outputs, off by a few units of fp32 (u = 2^-24).
// 4096 x 16384 x 4096 with gelu and residual: 299 us in bf16, 358 in fp32 (347 there with the
// shorter form; without an activation 342).
//
// z / (1 + exp(-v)), v of z's sign.  For 16 bits one exp2 and one reciprocal of the hardware,
// each within 2 u; the exponent's rounding adds |v| u.  kFull: with s = exp(-|v|) <= 1 it is
// z / (1 + s), or z s / (1 + s) below zero; what the product |v| log2 e rounds off goes into s
// by its first-order term, and the reciprocal takes one Newton step.
template <bool kFull>
__device__ __forceinline__ float logistic_times(float z, float v) {
  typedef ActConst<float> K;
  if constexpr (!kFull)
    return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-v * K::kLog2e));
  const float a = __builtin_fabsf(v), hi = -K::kLog2e * a;
  const float lo = __builtin_fmaf(-K::kLog2eLow, a, __builtin_fmaf(-K::kLog2e, a, -hi));
  float s = __builtin_amdgcn_exp2f(hi);
  s = __builtin_fmaf(s, lo * K::kLn2, s);
  s = a < 128.0f ? s : 0.0f;   // there lo is large or infinite and s 0
  const float d = 1.0f + s;
  float r = __builtin_amdgcn_rcpf(d);
  r = __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r);
  return (v < 0.0f ? z * s : z) * r;
}

// z Phi(z).  The tail Phi(-|z|) = t P(t) exp(-z^2 / 2) with t = 1 / (1 + q |z|): P is fitted to
// the scaled tail with the least relative error over |z| <= 13.3 (where the tail leaves fp32), so
// that the result keeps its leading digits however small it is; above zero Phi = 1 - tail.
// 16 bits: seven terms, off by 7.5e-7 relative, and exp2's argument by up to 1e-5 at the tail's
// end: 2^-16, a thirtieth of fp16's rounding.  kFull: eight terms for |z| >= 1 (1.5e-8), what z^2 and
// its product with log2 e / 2 round off as above, one Newton step; below, where 1 - tail would
// magnify the tail's error, Phi = 1 / 2 + z M(z^2), M of six terms (7e-10).  Eight units of u at
// most in all, in a model of these steps.
template <bool kFull>
__device__ __forceinline__ float gelu_times(float z) {
  typedef ActConst<float> K;
  if constexpr (!kFull) {
    const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.36f, __builtin_fabsf(z), 1.0f));
    float p = __builtin_fmaf(0.04746443033f, t, -0.1811617911f);
    p = __builtin_fmaf(p, t, 0.1828561127f);
    p = __builtin_fmaf(p, t, 0.02523851208f);
    p = __builtin_fmaf(p, t, 0.1401986182f);
    p = __builtin_fmaf(p, t, 0.1416846828f);
    p = __builtin_fmaf(p, t, 0.1437192857f);
    const float tail = p * t * __builtin_amdgcn_exp2f(-0.5f * K::kLog2e * z * z);
    return z * (z < 0.0f ? tail : 1.0f - tail);
  }
  const float y = z * z;
  float m = __builtin_fmaf(-7.654212823e-06f, y, 1.134863851e-04f);
  m = __builtin_fmaf(m, y, -1.186329988e-03f);
  m = __builtin_fmaf(m, y, 9.973322973e-03f);
  m = __builtin_fmaf(m, y, -6.649035960e-02f);
  m = __builtin_fmaf(m, y, 3.989422917e-01f);
  const float a = __builtin_fminf(__builtin_fabsf(z), 16.0f);
  const float d = __builtin_fmaf(0.24f, a, 1.0f);
  float t = __builtin_amdgcn_rcpf(d);
  t = __builtin_fmaf(__builtin_fmaf(-d, t, 1.0f), t, t);
  float p = __builtin_fmaf(-0.05917223543f, t, 0.1761606038f);
  p = __builtin_fmaf(p, t, -0.1021098420f);
  p = __builtin_fmaf(p, t, 0.1485771835f);
  p = __builtin_fmaf(p, t, 0.04906247184f);
  p = __builtin_fmaf(p, t, 0.09672495723f);
  p = __builtin_fmaf(p, t, 0.09496610612f);
  p = __builtin_fmaf(p, t, 0.09578620642f);
  constexpr float kHalf = -0.5f * K::kLog2e, kHalfLow = -0.5f * K::kLog2eLow;
  const float sq = a * a, rest = __builtin_fmaf(a, a, -sq), hi = kHalf * sq;
  float lo = __builtin_fmaf(kHalfLow, sq, __builtin_fmaf(kHalf, sq, -hi));
  lo = __builtin_fmaf(kHalf, rest, lo);
  float e = __builtin_amdgcn_exp2f(hi);
  e = __builtin_fmaf(e, lo * K::kLn2, e);
  const float tail = p * t * e;
  const float phi = __builtin_fabsf(z) < 1.0f ? __builtin_fmaf(m, z, 0.5f)
                                              : (z < 0.0f ? tail : 1.0f - tail);
  return z * phi;
}

// Results of the last three below 2^-119 may come as zero.
template <bool kFull>
__device__ __forceinline__ float activate32(float z, int act) {
  typedef ActConst<float> K;
  switch (act) {
    case OZK_ACT_RELU:
      return z < 0.0f ? 0.0f : z;
    case OZK_ACT_GELU:
      return gelu_times<kFull>(z);
    case OZK_ACT_GELU_TANH:
      return logistic_times<kFull>(z,
                                   K::kTanhScale * __builtin_fmaf(K::kTanhCubic * z * z, z, z));
    case OZK_ACT_SILU:
      return logistic_times<kFull>(z, z);
    default:
      return z;
  }
}

// activate32 of N values: the choice of the function stands outside their loop.
template <bool kFull, int N>
__device__ __forceinline__ void activate_all(float (&z)[N], int act) {
  auto each = [&](int a) {
#pragma unroll
    for (int u = 0; u < N; ++u) z[u] = activate32<kFull>(z[u], a);
  };
  if (act == OZK_ACT_RELU) each(OZK_ACT_RELU);
  else if (act == OZK_ACT_GELU) each(OZK_ACT_GELU);
  else if (act == OZK_ACT_GELU_TANH) each(OZK_ACT_GELU_TANH);
  else if (act == OZK_ACT_SILU) each(OZK_ACT_SILU);
}

// d activate / dz.  p (1 - p) is an exact 0 where the logistic function has settled; there
// the slope is p, also where the factor beside it would overflow.
__device__ __forceinline__ double activate_slope(double z, int act) {
  typedef ActConst<double> K;
  switch (act) {
    case OZK_ACT_RELU:
      return z > 0 ? 1 : 0;
    case OZK_ACT_GELU:
      return 0.5 * erfc(-z * K::kRsqrt2) + z * (exp(-0.5 * z * z) * K::kRsqrt2Pi);
    case OZK_ACT_GELU_TANH: {
      const double p = 1 / (1 + exp(-K::kTanhScale * (z + K::kTanhCubic * z * z * z)));
      const double q = p * (1 - p);
      return q == 0 ? p : p + z * q * K::kTanhScale * (1 + 3 * K::kTanhCubic * z * z);
    }
    case OZK_ACT_SILU: {
      const double p = 1 / (1 + exp(-z));
      const double q = p * (1 - p);
      return q == 0 ? p : p + z * q;
    }
    default:
      return 1;
  }
}

}  // namespace ozk
