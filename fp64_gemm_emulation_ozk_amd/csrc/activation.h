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

// z / (1 + exp(-v)): one exp2 and one reciprocal of the hardware, each within one ulp.
__device__ __forceinline__ float logistic_times(float z, float v) {
  return z * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-v * ActConst<float>::kLog2e));
}

// The same in fp32 for the int8 layer, whose epilogue is bound by these instructions (16 of
// them for gelu; 4096 x 16384 x 4096 with gelu and residual took 403 us with the library's
// erfcf and expf, 367 with these, the rest of the kernel the same).
// gelu: with x = |z| / sqrt 2 and t = 1 / (1 + 0.3275911 x),
//   erfc(x) = (a1 t + a2 t^2 + a3 t^3 + a4 t^4 + a5 t^5) exp(-x^2) + e, |e| <= 1.5e-7
// (Abramowitz and Stegun, Handbook of Mathematical Functions, 7.1.26), so the result is off
// by at most 0.75e-7 |z| beside its roundings: about one unit of fp32 in |z|.
__device__ __forceinline__ float activate(float z, int act) {
  typedef ActConst<float> K;
  switch (act) {
    case OZK_ACT_RELU:
      return z < 0.0f ? 0.0f : z;
    case OZK_ACT_GELU: {
      const float x = __builtin_fabsf(z) * K::kRsqrt2;
      const float t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3275911f, x, 1.0f));
      float p = __builtin_fmaf(1.061405429f, t, -1.453152027f);
      p = __builtin_fmaf(p, t, 1.421413741f);
      p = __builtin_fmaf(p, t, -0.284496736f);
      p = __builtin_fmaf(p, t, 0.254829592f);
      const float half_tail = 0.5f * (p * t) * __builtin_amdgcn_exp2f(-K::kLog2e * x * x);
      return z * (z < 0.0f ? half_tail : 1.0f - half_tail);
    }
    case OZK_ACT_GELU_TANH:
      return logistic_times(z, K::kTanhScale * __builtin_fmaf(K::kTanhCubic * z * z, z, z));
    case OZK_ACT_SILU:
      return logistic_times(z, z);
    default:
      return z;
  }
}

// activate of N values: the choice of the function stands outside their loop.
template <int N>
__device__ __forceinline__ void activate_all(float (&z)[N], int act) {
  auto each = [&](int a) {
#pragma unroll
    for (int u = 0; u < N; ++u) z[u] = activate(z[u], a);
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
