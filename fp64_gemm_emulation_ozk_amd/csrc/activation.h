// The activations of the products' epilogues and their slopes.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/ozk.h"

namespace ozk {

__device__ __forceinline__ double act_exp(double v) { return exp(v); }
__device__ __forceinline__ float act_exp(float v) { return expf(v); }
__device__ __forceinline__ double act_erfc(double v) { return erfc(v); }
__device__ __forceinline__ float act_erfc(float v) { return erfcf(v); }

template <typename A>
struct ActConst {
  static constexpr A kRsqrt2 = (A)0.70710678118654752440;       // 2^(-1/2)
  static constexpr A kRsqrt2Pi = (A)0.39894228040143267794;     // (2 pi)^(-1/2)
  static constexpr A kTanhScale = (A)1.59576912160573071175;    // 2 (2 / pi)^(1/2)
  static constexpr A kTanhCubic = (A)0.044715;
};

// gelu z Phi(z) with Phi(z) = erfc(-z / sqrt 2) / 2 (no cancellation in the lower tail);
// gelu_tanh z (1 + tanh u) / 2 = z / (1 + exp(-2 u)), u = (2 / pi)^(1/2) (z + 0.044715 z^3);
// silu z / (1 + exp(-z)).  A NaN stays NaN.
template <typename A>
__device__ __forceinline__ A activate(A z, int act) {
  typedef ActConst<A> K;
  switch (act) {
    case OZK_ACT_RELU:
      return z < (A)0 ? (A)0 : z;
    case OZK_ACT_GELU:
      return (A)0.5 * z * act_erfc(-z * K::kRsqrt2);
    case OZK_ACT_GELU_TANH:
      return z / ((A)1 + act_exp(-K::kTanhScale * (z + K::kTanhCubic * z * z * z)));
    case OZK_ACT_SILU:
      return z / ((A)1 + act_exp(-z));
    default:
      return z;
  }
}

// d activate / dz.  p (1 - p) is an exact 0 where the logistic function has settled; there
// the slope is p, also where the factor beside it would overflow.
template <typename A>
__device__ __forceinline__ A activate_slope(A z, int act) {
  typedef ActConst<A> K;
  switch (act) {
    case OZK_ACT_RELU:
      return z > (A)0 ? (A)1 : (A)0;
    case OZK_ACT_GELU:
      return (A)0.5 * act_erfc(-z * K::kRsqrt2) + z * (act_exp((A)-0.5 * z * z) * K::kRsqrt2Pi);
    case OZK_ACT_GELU_TANH: {
      const A p = (A)1 / ((A)1 + act_exp(-K::kTanhScale * (z + K::kTanhCubic * z * z * z)));
      const A q = p * ((A)1 - p);
      return q == (A)0 ? p : p + z * q * K::kTanhScale * ((A)1 + 3 * K::kTanhCubic * z * z);
    }
    case OZK_ACT_SILU: {
      const A p = (A)1 / ((A)1 + act_exp(-z));
      const A q = p * ((A)1 - p);
      return q == (A)0 ? p : p + z * q;
    }
    default:
      return (A)1;
  }
}

}  // namespace ozk
