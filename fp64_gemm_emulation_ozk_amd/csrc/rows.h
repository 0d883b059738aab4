// Row-wise access shared by the kernels that work on whole rows (layer norm, int8 row
// codes): element types, 16-byte vectors at any element alignment, sums and maxima over
// the threads of a row.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ozk_internal.h"

namespace ozk {

typedef __bf16 bf16_t;
typedef _Float16 f16_t;

// 16 bytes of elements.  The vector type carries the alignment of one element: gfx950
// global loads and stores take any alignment, so rows with an odd leading dimension use
// the same instructions (an access that crosses a cache line costs a second one).
template <typename T>
struct Vec {
  static constexpr int N = 16 / (int)sizeof(T);
  typedef T type __attribute__((ext_vector_type(16 / sizeof(T)), aligned(sizeof(T))));
};

// Type of sums, statistics and products of T: 32 bits at least.
template <typename T>
struct AccOf {
  typedef float type;
};
template <>
struct AccOf<double> {
  typedef double type;
};

// DPP moves of one 32-bit value (all lanes active).
template <int kCtrl>
__device__ __forceinline__ uint32_t dpp_mov(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, kCtrl, 0xf, 0xf, true);
}

// f(v, v of the lane `step` away) for the six butterfly steps of a 64-lane wave: quad
// permutes, half-row and row mirrors (any lane of the other half will do once a half
// agrees), then the two gfx950 lane swaps.  Every lane ends with the same bits: each step
// combines the same two values in both partners.
template <typename F>
__device__ __forceinline__ float wave_all(float v, F f) {
  const auto move = [](uint32_t x, int step) -> uint32_t {
    switch (step) {
      case 0: return dpp_mov<0xb1>(x);        // lane ^ 1
      case 1: return dpp_mov<0x4e>(x);        // lane ^ 2
      case 2: return dpp_mov<0x141>(x);       // mirror of 8
      default: return dpp_mov<0x140>(x);      // mirror of 16
    }
  };
#pragma unroll
  for (int s = 0; s < 4; ++s) v = f(v, __uint_as_float(move(__float_as_uint(v), s)));
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false,
                                                  false);
  v = f(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false,
                                                  false);
  return f(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

template <typename F>
__device__ __forceinline__ double wave_all(double v, F f) {
  const auto join = [](uint32_t lo, uint32_t hi) {
    return __longlong_as_double((long long)(((uint64_t)hi << 32) | lo));
  };
  const auto lo_of = [](double d) { return (uint32_t)(uint64_t)__double_as_longlong(d); };
  const auto hi_of = [](double d) { return (uint32_t)((uint64_t)__double_as_longlong(d) >> 32); };
  v = f(v, join(dpp_mov<0xb1>(lo_of(v)), dpp_mov<0xb1>(hi_of(v))));
  v = f(v, join(dpp_mov<0x4e>(lo_of(v)), dpp_mov<0x4e>(hi_of(v))));
  v = f(v, join(dpp_mov<0x141>(lo_of(v)), dpp_mov<0x141>(hi_of(v))));
  v = f(v, join(dpp_mov<0x140>(lo_of(v)), dpp_mov<0x140>(hi_of(v))));
  {
    const auto l = __builtin_amdgcn_permlane16_swap(lo_of(v), lo_of(v), false, false);
    const auto h = __builtin_amdgcn_permlane16_swap(hi_of(v), hi_of(v), false, false);
    v = f(join(l[0], h[0]), join(l[1], h[1]));
  }
  const auto l = __builtin_amdgcn_permlane32_swap(lo_of(v), lo_of(v), false, false);
  const auto h = __builtin_amdgcn_permlane32_swap(hi_of(v), hi_of(v), false, false);
  return f(join(l[0], h[0]), join(l[1], h[1]));
}

struct SumOp {
  template <typename A>
  __device__ __forceinline__ A operator()(A a, A b) const { return a + b; }
};
struct MaxOp {
  template <typename A>
  __device__ __forceinline__ A operator()(A a, A b) const { return a > b ? a : b; }
};

// v combined over the kT threads of a row (one wave, or the whole workgroup of kT), the
// waves in order.  `slot` (kT / 64 values of LDS) is this reduction's own: a workgroup that
// reduces again uses another slot or passes a barrier in between.
template <int kT, typename A, typename F>
__device__ __forceinline__ A row_all(A v, F f, A* slot) {
  v = wave_all(v, f);
  if constexpr (kT > 64) {
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x >> 6] = v;
    __syncthreads();
    v = slot[0];
#pragma unroll
    for (int w = 1; w < kT / 64; ++w) v = f(v, slot[w]);
  }
  return v;
}

// Elements c .. c + N - 1 of a row of `cols`, zero past its end.
template <typename T, typename A>
__device__ __forceinline__ void load_vec(const T* p, int64_t c, int64_t cols,
                                         A (&a)[Vec<T>::N]) {
  constexpr int N = Vec<T>::N;
  if (c + N <= cols) {
    const typename Vec<T>::type v = *reinterpret_cast<const typename Vec<T>::type*>(p + c);
#pragma unroll
    for (int u = 0; u < N; ++u) a[u] = (A)v[u];
  } else {
#pragma unroll
    for (int u = 0; u < N; ++u) a[u] = c + u < cols ? (A)p[c + u] : (A)0;
  }
}

// The same in two steps, so that a row can be asked for before it is needed: the 16 bytes
// as they are (past the row's end: zeros), and their values.
template <typename T>
__device__ __forceinline__ typename Vec<T>::type ask_vec(const T* p, int64_t c,
                                                         int64_t cols) {
  constexpr int N = Vec<T>::N;
  if (c + N <= cols) return *reinterpret_cast<const typename Vec<T>::type*>(p + c);
  typename Vec<T>::type v;
#pragma unroll
  for (int u = 0; u < N; ++u) v[u] = c + u < cols ? p[c + u] : (T)0.0f;
  return v;
}

// The same with the row's first element past its end: what stands there then adds nothing to
// a maximum over the row, nor to sums of differences from that element, and needs no mask.
template <typename T>
__device__ __forceinline__ typename Vec<T>::type ask_vec_first(const T* p, int64_t c,
                                                               int64_t cols) {
  constexpr int N = Vec<T>::N;
  if (c + N <= cols) return *reinterpret_cast<const typename Vec<T>::type*>(p + c);
  typename Vec<T>::type v;
#pragma unroll
  for (int u = 0; u < N; ++u) v[u] = p[c + u < cols ? c + u : 0];
  return v;
}

// The same elements stored, each rounded once to T; nothing past the row's end.
template <typename T, typename A>
__device__ __forceinline__ void store_vec(T* p, int64_t c, int64_t cols,
                                          const A (&a)[Vec<T>::N]) {
  constexpr int N = Vec<T>::N;
  if (c + N <= cols) {
    typename Vec<T>::type v;
#pragma unroll
    for (int u = 0; u < N; ++u) v[u] = (T)a[u];
    *reinterpret_cast<typename Vec<T>::type*>(p + c) = v;
  } else {
#pragma unroll
    for (int u = 0; u < N; ++u)
      if (c + u < cols) p[c + u] = (T)a[u];
  }
}

}  // namespace ozk
