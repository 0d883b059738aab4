// Layer norm over rows, forward and backward, and rows of int8 codes.
//
// With mu = mean(x), rho = (mean((x - mu)^2) + eps)^(-1/2) of a row and xh = (x - mu) rho:
//   forward   y = xh gamma + beta
//   backward  g = dy gamma; dx = rho (g - mean(g) - xh mean(g xh));
//             dgamma = sum over rows of dy xh, dbeta = sum over rows of dy
//   codes     s = fp32(max |y| / 127), q = rint(y / s) for y = x or the forward's y
//
// Many rows are bound by HBM: a row is read once into registers (the mean, then the centred
// sum of squares, are taken from there), in 16-byte loads.  Few rows are bound by a launch and
// one chain of latencies (load, two reductions, store): 8 x 1024 fp32 takes 3.9 us.
// Sums and statistics are fp32 for the types of at most 32 bits and fp64 for fp64; the
// codes' statistics are fp64 for every type (fp64 arithmetic runs at the fp32 rate here), so
// that a code depends on the order of the sums only within 1e-13 of a rounding border.
#include "ozk_internal.h"
#include "rows.h"

namespace ozk {
namespace {

// Number of valid elements of the vector that starts at column c.
template <int N>
__device__ __forceinline__ int valid(int64_t c, int64_t cols) {
  const int64_t left = cols - c;
  return left >= N ? N : (left > 0 ? (int)left : 0);
}

// ------------------------------------------------------------------ forward
// The mean and rstd of a row from the first sum's `mean` and the sums s1 of d = x - mean and s2
// of d^2: the mean is off by some roundings of the sum, which d shows without them where the row
// lies far from zero (x - mean is exact there): y = d rstd + shift.  A constant row 12345.6 fp32
// had y up to 0.7 from the first mean alone.
template <typename A>
struct RowStats {
  A mean, rstd, shift;
};
__device__ __forceinline__ float fma_of(float a, float b, float c) {
  return __builtin_fmaf(a, b, c);
}
__device__ __forceinline__ double fma_of(double a, double b, double c) {
  return __builtin_fma(a, b, c);
}
template <int kT, typename A>
__device__ __forceinline__ RowStats<A> row_stats(A mean, A s1, A s2, A inv, A eps,
                                                 A (*slots)[kT / 64]) {
  s1 = wave_all(s1, SumOp());
  s2 = wave_all(s2, SumOp());
  if constexpr (kT > 64) {
    if ((threadIdx.x & 63) == 0) {
      slots[0][threadIdx.x >> 6] = s1;
      slots[1][threadIdx.x >> 6] = s2;
    }
    __syncthreads();
    s1 = slots[0][0];
    s2 = slots[1][0];
#pragma unroll
    for (int w = 1; w < kT / 64; ++w) {
      s1 += slots[0][w];
      s2 += slots[1][w];
    }
  }
  const A off = s1 * inv, var = s2 * inv - off * off;
  // (a constant row's difference may fall below zero; a NaN stays one)
  const A rstd = (A)1 / sqrt((var < 0 ? (A)0 : var) + eps);
  return {mean + off, rstd, -off * rstd};
}

// kT threads of a row hold it in kV vectors each (vector v of thread t starts at column
// (v kT + t) N).  kT = 64: four rows per workgroup; else one.  16384 x 4096 bf16: 51 us, 268 MB
// at 5.26 TB/s, 0.96 of a large copy's rate.
template <typename T, int kT, int kV>
__global__ __launch_bounds__(kT < 256 ? 256 : kT) void layernorm_kernel(
    int64_t rows, int64_t cols, const T* x, int64_t ldx,
    const T* __restrict__ gamma, const T* __restrict__ beta, typename AccOf<T>::type eps, T* y, int64_t ldy, typename AccOf<T>::type* __restrict__ mean_out,
    typename AccOf<T>::type* __restrict__ rstd_out) {
  typedef typename AccOf<T>::type A;
  constexpr int N = Vec<T>::N;
  constexpr int kRows = kT < 256 ? 256 / kT : 1;
  __shared__ A slots[3][kT / 64];
  const int t = threadIdx.x % kT;
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / kT;
  if (kRows > 1 && row >= rows) return;  // whole waves
  const T* xr = x + row * ldx;
  A a[kV][N];
  A sum = 0;
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    load_vec<T, A>(xr, (int64_t)(v * kT + t) * N, cols, a[v]);
#pragma unroll
    for (int u = 0; u < N; ++u) sum += a[v][u];
  }
  const A inv = (A)1 / (A)cols;
  const A mean = row_all<kT>(sum, SumOp(), slots[0]) * inv;
  A s1 = 0, s2 = 0;
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    const int nv = valid<N>((int64_t)(v * kT + t) * N, cols);
#pragma unroll
    for (int u = 0; u < N; ++u) {
      a[v][u] = u < nv ? a[v][u] - mean : (A)0;
      s1 += a[v][u];
      s2 = fma_of(a[v][u], a[v][u], s2);
    }
  }
  const RowStats<A> S = row_stats<kT>(mean, s1, s2, inv, eps, slots + 1);
  if (t == 0) {
    if (mean_out) mean_out[row] = S.mean;
    if (rstd_out) rstd_out[row] = S.rstd;
  }
  T* yr = y + row * ldy;
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    const int64_t c = (int64_t)(v * kT + t) * N;
    if (c >= cols) continue;
    A g[N], b[N];
    if (gamma) load_vec<T, A>(gamma, c, cols, g);
    if (beta) load_vec<T, A>(beta, c, cols, b);
#pragma unroll
    for (int u = 0; u < N; ++u) a[v][u] = fma_of(a[v][u], S.rstd, S.shift);
    if (gamma && beta) {
#pragma unroll
      for (int u = 0; u < N; ++u) a[v][u] = fma_of(a[v][u], g[u], b[u]);
    } else {
#pragma unroll
      for (int u = 0; u < N; ++u) {
        if (gamma) a[v][u] *= g[u];
        if (beta) a[v][u] += b[u];
      }
    }
    store_vec<T, A>(yr, c, cols, a[v]);
  }
}

// Rows too long for registers: three passes over the row (it stays in L2).
template <typename T>
__global__ __launch_bounds__(1024) void layernorm_long_kernel(
    int64_t cols, const T* x, int64_t ldx, const T* __restrict__ gamma,
    const T* __restrict__ beta, typename AccOf<T>::type eps, T* y, int64_t ldy,
    typename AccOf<T>::type* __restrict__ mean_out,
    typename AccOf<T>::type* __restrict__ rstd_out) {
  typedef typename AccOf<T>::type A;
  constexpr int N = Vec<T>::N, kT = 1024;
  __shared__ A slots[3][kT / 64];
  const int64_t row = blockIdx.x;
  const T* xr = x + row * ldx;
  A sum = 0, a[N];
  for (int64_t c = (int64_t)threadIdx.x * N; c < cols; c += kT * N) {
    load_vec<T, A>(xr, c, cols, a);
#pragma unroll
    for (int u = 0; u < N; ++u) sum += a[u];
  }
  const A inv = (A)1 / (A)cols;
  const A mean = row_all<kT>(sum, SumOp(), slots[0]) * inv;
  A s1 = 0, s2 = 0;
  for (int64_t c = (int64_t)threadIdx.x * N; c < cols; c += kT * N) {
    load_vec<T, A>(xr, c, cols, a);
    const int nv = valid<N>(c, cols);
#pragma unroll
    for (int u = 0; u < N; ++u)
      if (u < nv) {
        const A d = a[u] - mean;
        s1 += d;
        s2 = fma_of(d, d, s2);
      }
  }
  const RowStats<A> S = row_stats<kT>(mean, s1, s2, inv, eps, slots + 1);
  if (threadIdx.x == 0) {
    if (mean_out) mean_out[row] = S.mean;
    if (rstd_out) rstd_out[row] = S.rstd;
  }
  T* yr = y + row * ldy;
  for (int64_t c = (int64_t)threadIdx.x * N; c < cols; c += kT * N) {
    load_vec<T, A>(xr, c, cols, a);
    A g[N], b[N];
    if (gamma) load_vec<T, A>(gamma, c, cols, g);
    if (beta) load_vec<T, A>(beta, c, cols, b);
#pragma unroll
    for (int u = 0; u < N; ++u) {
      A w = fma_of(a[u] - mean, S.rstd, S.shift);
      if (gamma) w *= g[u];
      if (beta) w += b[u];
      a[u] = w;
    }
    store_vec<T, A>(yr, c, cols, a);
  }
}

// ------------------------------------------------------------------ int8 codes
// Scale and reciprocal of a row from its largest magnitude.  A row with a value that is not
// finite, or whose scale is no finite fp32, gets the scale NaN and zero codes; a row of
// zeros (or of values below the smallest fp32 scale) the scale 0 and zero codes.
struct CodeScale {
  float scale;
  double inv;
};
__device__ __forceinline__ CodeScale code_scale(double amax, bool bad) {
  const float s = (float)(amax / 127.0);
  if (bad || !(s <= 3.402823466e38f)) return {__builtin_nanf(""), 0.0};
  return {s, s > 0.0f ? 1.0 / (double)s : 0.0};
}

// rint(w inv) as a byte: adding 1.5 2^52 rounds to the nearest integer, ties to even, and
// leaves it in the low word.  A subnormal scale can be off by a third: then the quotient
// passes 127 and is cut.
__device__ __forceinline__ int code_of(double w, double inv) {
  const double p = w * inv;
  const double c = p > 127.0 ? 127.0 : (p < -127.0 ? -127.0 : p);
  return (int)(uint32_t)__double_as_longlong(c + kMagic);
}

template <int N>
__device__ __forceinline__ void store_codes(int8_t* __restrict__ p, int64_t c, int64_t cols,
                                            const int (&q)[N]) {
  if (c + N <= cols) {
    typedef int8_t V __attribute__((ext_vector_type(N), aligned(1)));
    V v;
#pragma unroll
    for (int u = 0; u < N; ++u) v[u] = (int8_t)q[u];
    *reinterpret_cast<V*>(p + c) = v;
  } else {
#pragma unroll
    for (int u = 0; u < N; ++u)
      if (c + u < cols) p[c + u] = (int8_t)q[u];
  }
}

// kNorm: y = layer norm of x, else y = x.  fp64 x: everything in fp64.
template <int kT, int kV, bool kNorm>
__device__ __forceinline__ void int8quant_row_f64(
    int64_t row, int64_t cols, const double* __restrict__ x, int64_t ldx,
    const double* __restrict__ gamma, const double* __restrict__ beta, double eps,
    int8_t* __restrict__ q, int64_t ldq, float* __restrict__ scale) {
  constexpr int N = Vec<double>::N;
  __shared__ double slots[3][kT / 64];
  const int t = threadIdx.x % kT;
  const double* xr = x + row * ldx;
  double a[kV][N];
  double sum = 0;
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    load_vec<double, double>(xr, (int64_t)(v * kT + t) * N, cols, a[v]);
    if (kNorm) {
#pragma unroll
      for (int u = 0; u < N; ++u) sum += a[v][u];
    }
  }
  if constexpr (kNorm) {
    const double mean = row_all<kT>(sum, SumOp(), slots[0]) / (double)cols;
    double sq = 0;
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      const int nv = valid<N>((int64_t)(v * kT + t) * N, cols);
#pragma unroll
      for (int u = 0; u < N; ++u) {
        a[v][u] -= mean;
        if (u < nv) sq += a[v][u] * a[v][u];
      }
    }
    const double var = row_all<kT>(sq, SumOp(), slots[1]) / (double)cols;
    const double rstd = 1.0 / sqrt(var + eps);
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      const int64_t c = (int64_t)(v * kT + t) * N;
      double g[N], b[N];
      if (gamma) load_vec<double, double>(gamma, c, cols, g);
      if (beta) load_vec<double, double>(beta, c, cols, b);
      const int nv = valid<N>(c, cols);
#pragma unroll
      for (int u = 0; u < N; ++u) {
        double w = a[v][u] * rstd;
        if (gamma) w *= g[u];
        if (beta) w += b[u];
        a[v][u] = u < nv ? w : 0.0;
      }
    }
  }
  double amax = 0;
  bool bad = false;
#pragma unroll
  for (int v = 0; v < kV; ++v)
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const double m = __builtin_fabs(a[v][u]);
      bad |= !(m <= 1.7976931348623157e308);
      amax = m > amax ? m : amax;
    }
  amax = row_all<kT>(bad ? __builtin_huge_val() : amax, MaxOp(), slots[2]);
  const CodeScale cs = code_scale(amax, !(amax <= 1.7976931348623157e308));
  if (t == 0) scale[row] = cs.scale;
  int8_t* qr = q + row * ldq;
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    const int64_t c = (int64_t)(v * kT + t) * N;
    if (c >= cols) continue;
    int codes[N];
#pragma unroll
    for (int u = 0; u < N; ++u) codes[u] = cs.inv == 0.0 ? 0 : code_of(a[v][u], cs.inv);
    store_codes<N>(qr, c, cols, codes);
  }
}

// x of at most 32 bits: the same codes and scale, most of the work in fp32.  The row's sums are
// fp64 (of x - c and its square, c the row's first value; again about the mean where c lies
// far from it).  y and y / s are formed in fp32 beside a bound e of their error; where that
// bound leaves the largest magnitude or a code's rounding open (about one value in five
// thousand), the value is formed in fp64.  A row whose magnitudes are out of the bound's
// reach (below 1e-30, above 1e37, not finite) takes fp64 throughout.
// All in fp64, 4096 x 8192 bf16 with the norm took 69.5 us, 4096 x 16384 without 61.1; so they
// take 37 and 36, the latter 201 MB at a large copy's rate.  With the norm the vector instructions
// bind, 42 a value (16 without), five of them fp64: they issue in 0.8 of the cycles in bf16, in 0.65
// in fp32 (4096 x 8192 fp32: 56 us, 3.0 TB/s).
template <typename T, int kT, int kV, bool kNorm>
__device__ __forceinline__ void int8quant_row(
    int64_t row, int64_t cols, const T* __restrict__ x, int64_t ldx,
    const T* __restrict__ gamma, const T* __restrict__ beta, double eps,
    int8_t* __restrict__ q, int64_t ldq, float* __restrict__ scale) {
  constexpr int N = Vec<T>::N, kW = kT / 64;
  __shared__ double sums[kNorm ? 3 : 1][kW];
  __shared__ uint32_t tops[kNorm ? 2 : 1][kW];
  const int t = threadIdx.x % kT;
  const T* xr = x + row * ldx;
  typename Vec<T>::type raw[kV];
  uint32_t in_row = 0;   // a bit per value that lies in the row
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    const int64_t c = (int64_t)(v * kT + t) * N;
    raw[v] = ask_vec_first<T>(xr, c, cols);
    in_row |= ((1u << valid<N>(c, cols)) - 1u) << (v * N);
  }

  double mean = 0.0, rstd = 1.0;
  bool level = true;   // y is exactly what fp32 makes of it where that is all zeros
  if constexpr (kNorm) {
    const double c0 = (double)xr[0], rows_inv = 1.0 / (double)cols;
    double s1 = 0, s2 = 0;
#pragma unroll
    for (int v = 0; v < kV; ++v)
#pragma unroll
      for (int u = 0; u < N; ++u) {
        const double d = (double)raw[v][u] - c0;
        s1 += d;
        s2 = __builtin_fma(d, d, s2);
      }
    s1 = wave_all(s1, SumOp());
    s2 = wave_all(s2, SumOp());
    if constexpr (kT > 64) {
      if ((threadIdx.x & 63) == 0) {
        sums[0][threadIdx.x >> 6] = s1;
        sums[1][threadIdx.x >> 6] = s2;
      }
      __syncthreads();
      s1 = sums[0][0];
      s2 = sums[1][0];
#pragma unroll
      for (int w = 1; w < kW; ++w) {
        s1 += sums[0][w];
        s2 += sums[1][w];
      }
    }
    level = s2 == 0.0;   // every value is c0, so is the mean
    const double off = s1 * rows_inv;
    mean = c0 + off;
    double var = s2 * rows_inv - off * off;
    // the difference keeps 2^-53 (1 + off^2 / var) of var (uniform over the row)
    if (!(off * off <= 64.0 * var)) {
      double sq = 0;
#pragma unroll 1
      for (int64_t c = t; c < cols; c += kT) {
        const double d = (double)xr[c] - mean;
        sq = __builtin_fma(d, d, sq);
      }
      var = row_all<kT>(sq, SumOp(), sums[2]) * rows_inv;
    }
    rstd = 1.0 / sqrt(var + eps);
  }
  // y of column c in fp64
  auto exact = [&](int64_t c) {
    double y = (double)xr[c];
    if (kNorm) {
      y = (y - mean) * rstd;
      if (gamma) y *= (double)gamma[c];
      if (beta) y += (double)beta[c];
    }
    return y;
  };
  // Values that stand open are marked in a word per lane and taken up one by one: their code
  // stands once, and no fp64 value lives in registers beside the row.
  static_assert(kV * N <= 32, "one bit per value");
  auto column = [&](int bit) { return (int64_t)(bit / N * kT + t) * N + bit % N; };
  const float mean_hi = (float)mean, mean_lo = (float)(mean - (double)mean_hi);
  const float rstd32 = (float)rstd;
  float y[kV][N];
  uint32_t top_y = 0, top_b = 0;   // magnitudes as bits: a NaN is above everything
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    const int64_t c = (int64_t)(v * kT + t) * N;
    typename Vec<T>::type g, b;
    if (kNorm && gamma) g = ask_vec_first<T>(gamma, c, cols);
    if (kNorm && beta) b = ask_vec_first<T>(beta, c, cols);
#pragma unroll
    for (int u = 0; u < N; ++u) {
      float w = (float)raw[v][u];
      if (kNorm) {
        w = ((w - mean_hi) - mean_lo) * rstd32;
        if (gamma) w *= (float)g[u];
        if (beta) {
          w += (float)b[u];
          const uint32_t m = __float_as_uint((float)b[u]) & 0x7fffffffu;
          top_b = m > top_b ? m : top_b;
        }
      }
      y[v][u] = w;
      const uint32_t m = __float_as_uint(w) & 0x7fffffffu;
      top_y = m > top_y ? m : top_y;
    }
  }
  // as floats the order of bits is that of the magnitudes, infinities included; a NaN is
  // passed on as one
  auto top = [](uint32_t bits) {
    return wave_all(bits > 0x7f800000u ? __builtin_huge_valf() : __uint_as_float(bits), MaxOp());
  };
  uint32_t ybits = __float_as_uint(top(top_y));
  uint32_t bbits = kNorm && beta ? __float_as_uint(top(top_b)) : 0u;
  if constexpr (kT > 64) {
    if ((threadIdx.x & 63) == 0) {
      tops[0][threadIdx.x >> 6] = ybits;
      if (kNorm) tops[1][threadIdx.x >> 6] = bbits;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kW; ++w) {
      ybits = tops[0][w] > ybits ? tops[0][w] : ybits;
      if (kNorm) bbits = tops[1][w] > bbits ? tops[1][w] : bbits;
    }
  }
  // uniform over the row, so over the wave
  ybits = __builtin_amdgcn_readfirstlane(ybits);
  const float ymax = __uint_as_float(ybits), bmax = __uint_as_float(bbits);
  // fp32 y is off by at most 8 roundings of |y - b| + |y| <= 2 |y| + |b| (x is exact)
  const float e = kNorm ? 8.0f * 5.97e-8f * (2.0f * ymax + bmax) : 0.0f;
  // A row of zeros (a padded token; a constant one after the norm without beta) is not open: 4096
  // x 16384 bf16 takes 27 us where all rows are such, 44 where none is (119 with each of their
  // values formed in fp64, 176 after the norm and now 65).
  const bool zero = ybits == 0 && level;
  const bool hard = !zero && !(ymax >= 1e-30f && ymax <= 1e37f && bmax <= 1e37f);
  double amax = (double)ymax;
  bool bad = false;
  if ((kNorm && !zero) || hard) {   // uniform
    double m64 = 0;
    uint32_t open = 0;
    const float least = ymax - 2.0f * e;
#pragma unroll
    for (int v = 0; v < kV; ++v)
#pragma unroll
      for (int u = 0; u < N; ++u)
        open |= __builtin_fabsf(y[v][u]) >= least ? 1u << (v * N + u) : 0u;
    open = (hard ? ~0u : open) & in_row;
#pragma unroll 1
    for (; open; open &= open - 1) {
      const double m = __builtin_fabs(exact(column(__builtin_ctz(open))));
      bad |= !(m <= 1.7976931348623157e308);
      m64 = m > m64 ? m : m64;
    }
    amax = row_all<kT>(bad ? __builtin_huge_val() : m64, MaxOp(), sums[0]);
  }
  const CodeScale cs = code_scale(amax, !(amax <= 1.7976931348623157e308));
  if (t == 0) scale[row] = cs.scale;
  int8_t* qr = q + row * ldq;
  if (cs.inv == 0.0) {   // uniform: all codes zero
    const int none[N] = {};
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      const int64_t c = (int64_t)(v * kT + t) * N;
      if (c < cols) store_codes<N>(qr, c, cols, none);
    }
    return;
  }
  const float inv32 = (float)cs.inv;
  // of a quotient of at most 127: y's error, and roundings of the reciprocal and the product
  const float within = hard ? -1.0f : 0.5f - (e * inv32 + 4.0f * 127.0f * 5.97e-8f);
  uint32_t open = 0;
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    int codes[N];
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const float p = y[v][u] * inv32, r = __builtin_rintf(p);
      codes[u] = (int)r;
      open |= __builtin_fabsf(p - r) <= within ? 0u : 1u << (v * N + u);
    }
    const int64_t c = (int64_t)(v * kT + t) * N;
    if (c < cols) store_codes<N>(qr, c, cols, codes);
  }
  open &= in_row;
#pragma unroll 1
  for (; open; open &= open - 1) {
    const int64_t c = column(__builtin_ctz(open));
    qr[c] = (int8_t)code_of(exact(c), cs.inv);
  }
}

template <typename T, int kT, int kV, bool kNorm>
__global__ __launch_bounds__(kT < 256 ? 256 : kT) void int8quant_kernel(
    int64_t rows, int64_t cols, const T* __restrict__ x, int64_t ldx,
    const T* __restrict__ gamma, const T* __restrict__ beta, double eps,
    int8_t* __restrict__ q, int64_t ldq, float* __restrict__ scale) {
  constexpr int kRows = kT < 256 ? 256 / kT : 1;
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / kT;
  if (kRows > 1 && row >= rows) return;   // whole waves
  if constexpr (sizeof(T) == 8)
    int8quant_row_f64<kT, kV, kNorm>(row, cols, x, ldx, gamma, beta, eps, q, ldq, scale);
  else
    int8quant_row<T, kT, kV, kNorm>(row, cols, x, ldx, gamma, beta, eps, q, ldq, scale);
}

template <typename T, bool kNorm>
__global__ __launch_bounds__(1024) void int8quant_long_kernel(
    int64_t cols, const T* __restrict__ x, int64_t ldx, const T* __restrict__ gamma,
    const T* __restrict__ beta, double eps, int8_t* __restrict__ q, int64_t ldq,
    float* __restrict__ scale) {
  constexpr int N = Vec<T>::N, kT = 1024;
  __shared__ double slots[3][kT / 64];
  const int64_t row = blockIdx.x;
  const T* xr = x + row * ldx;
  double a[N], mean = 0, rstd = 1;
  if (kNorm) {
    double sum = 0;
    for (int64_t c = (int64_t)threadIdx.x * N; c < cols; c += kT * N) {
      load_vec<T, double>(xr, c, cols, a);
#pragma unroll
      for (int u = 0; u < N; ++u) sum += a[u];
    }
    mean = row_all<kT>(sum, SumOp(), slots[0]) / (double)cols;
    double sq = 0;
    for (int64_t c = (int64_t)threadIdx.x * N; c < cols; c += kT * N) {
      load_vec<T, double>(xr, c, cols, a);
      const int nv = valid<N>(c, cols);
#pragma unroll
      for (int u = 0; u < N; ++u)
        if (u < nv) sq += (a[u] - mean) * (a[u] - mean);
    }
    rstd = 1.0 / sqrt(row_all<kT>(sq, SumOp(), slots[1]) / (double)cols + eps);
  }
  auto values = [&](int64_t c) {
    load_vec<T, double>(xr, c, cols, a);
    if (!kNorm) return;
    double g[N], b[N];
    if (gamma) load_vec<T, double>(gamma, c, cols, g);
    if (beta) load_vec<T, double>(beta, c, cols, b);
    const int nv = valid<N>(c, cols);
#pragma unroll
    for (int u = 0; u < N; ++u) {
      double w = (a[u] - mean) * rstd;
      if (gamma) w *= g[u];
      if (beta) w += b[u];
      a[u] = u < nv ? w : 0.0;
    }
  };
  double amax = 0;
  bool bad = false;
  for (int64_t c = (int64_t)threadIdx.x * N; c < cols; c += kT * N) {
    values(c);
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const double m = __builtin_fabs(a[u]);
      bad |= !(m <= 1.7976931348623157e308);
      amax = m > amax ? m : amax;
    }
  }
  amax = row_all<kT>(bad ? __builtin_huge_val() : amax, MaxOp(), slots[2]);
  const CodeScale cs = code_scale(amax, !(amax <= 1.7976931348623157e308));
  if (threadIdx.x == 0) scale[row] = cs.scale;
  for (int64_t c = (int64_t)threadIdx.x * N; c < cols; c += kT * N) {
    values(c);
    int codes[N];
#pragma unroll
    for (int u = 0; u < N; ++u) codes[u] = cs.inv == 0.0 ? 0 : code_of(a[u], cs.inv);
    store_codes<N>(q + row * ldq, c, cols, codes);
  }
}

// ------------------------------------------------------------------ backward
// Workgroup b of G walks rows b, b + G, ... (four rows at once, one a wave, where a wave
// holds a row): dx row by row, and the column sums dy xh and dy of its rows in registers,
// written to partials [G][2][cols] at the end.  A row is asked for one row ahead, before the
// reduction of the row in hand.  16384 x 4096 bf16: 78 us and 7 for the join of the sums, 403
// MB at 4.75 TB/s together (the partials are another 34 MB of traffic); 1000 x 1537 fp32: 10
// and 5 us, where two rows a workgroup and the second launch are the time.
template <typename T, int kT, int kV>
__global__ __launch_bounds__(kT < 256 ? 256 : kT) void layernorm_backward_kernel(
    int64_t rows, int64_t cols, const T* dy, int64_t lddy, const T* x, int64_t ldx,
    const T* __restrict__ gamma, const typename AccOf<T>::type* __restrict__ mean,
    const typename AccOf<T>::type* __restrict__ rstd, T* dx, int64_t lddx,
    typename AccOf<T>::type* __restrict__ part) {
  typedef typename AccOf<T>::type A;
  typedef typename Vec<T>::type V;
  constexpr int N = Vec<T>::N;
  constexpr int kRows = kT < 256 ? 256 / kT : 1;   // rows of a workgroup at once
  __shared__ A slots[2][2][kT / 64];
  __shared__ A joined[kRows > 1 ? (kRows - 1) * 2 * kV * N * 64 : 1];
  const int t = threadIdx.x % kT, sub = threadIdx.x / kT;
  const int64_t stride = (int64_t)gridDim.x * kRows;
  // gamma stays in registers where a thread of a large workgroup has them
  constexpr bool kKeep = kT * kV * N < 16384;
  A dg[kV][N], db[kV][N], w[kKeep ? kV : 1][N];
  V nx[kV], ny[kV];
  A nmu = 0, nrho = 0;
  auto ask = [&](int64_t row) {
    if (row >= rows) return;
    nmu = mean[row];
    nrho = rstd[row];
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      const int64_t c = (int64_t)(v * kT + t) * N;
      nx[v] = ask_vec<T>(x + row * ldx, c, cols);
      ny[v] = ask_vec<T>(dy + row * lddy, c, cols);
    }
  };
  ask(blockIdx.x * kRows + sub);
#pragma unroll
  for (int v = 0; v < kV; ++v) {
#pragma unroll
    for (int u = 0; u < N; ++u) {
      dg[v][u] = db[v][u] = 0;
      if (kKeep || v == 0) w[kKeep ? v : 0][u] = 1;
    }
    if (kKeep && gamma) load_vec<T, A>(gamma, (int64_t)(v * kT + t) * N, cols, w[kKeep ? v : 0]);
  }
  const A inv = (A)1 / (A)cols;
  int flip = 0;
  for (int64_t row = blockIdx.x * kRows + sub; row < rows; row += stride, flip ^= 1) {
    const A mu = nmu, rho = nrho;
    A xh[kV][N], g[kV][N];
    A s1 = 0, s2 = 0;
#pragma unroll
    for (int v = 0; v < kV; ++v) {
      const int nv = valid<N>((int64_t)(v * kT + t) * N, cols);
      if (!kKeep && gamma) load_vec<T, A>(gamma, (int64_t)(v * kT + t) * N, cols, w[0]);
#pragma unroll
      for (int u = 0; u < N; ++u) {
        xh[v][u] = u < nv ? ((A)nx[v][u] - mu) * rho : (A)0;
        const A d = (A)ny[v][u];
        dg[v][u] += d * xh[v][u];
        db[v][u] += d;
        g[v][u] = d * w[kKeep ? v : 0][u];
        s1 += g[v][u] * xh[v][u];
        s2 += g[v][u];
      }
    }
    ask(row + stride);
    // two slot sets in turn: a row's reads of one set end before the barrier of the next
    // row, which comes before the set is written again
    s1 = wave_all(s1, SumOp());
    s2 = wave_all(s2, SumOp());
    if constexpr (kT > 64) {
      if ((t & 63) == 0) {
        slots[flip][0][t >> 6] = s1;
        slots[flip][1][t >> 6] = s2;
      }
      __syncthreads();
      s1 = slots[flip][0][0];
      s2 = slots[flip][1][0];
#pragma unroll
      for (int wv = 1; wv < kT / 64; ++wv) {
        s1 += slots[flip][0][wv];
        s2 += slots[flip][1][wv];
      }
    }
    const A c1 = s1 * inv, c2 = s2 * inv;
    if (dx) {
      T* dxr = dx + row * lddx;
#pragma unroll
      for (int v = 0; v < kV; ++v) {
        const int64_t c = (int64_t)(v * kT + t) * N;
        if (c >= cols) continue;
#pragma unroll
        for (int u = 0; u < N; ++u) g[v][u] = rho * (g[v][u] - c2 - xh[v][u] * c1);
        store_vec<T, A>(dxr, c, cols, g[v]);
      }
    }
  }
  if (!part) return;   // the whole grid
  if constexpr (kRows > 1) {   // the waves' sums, in order
    A* mine = joined + (sub - 1) * (2 * kV * N * 64) + t;
    if (sub) {
#pragma unroll
      for (int v = 0; v < kV; ++v)
#pragma unroll
        for (int u = 0; u < N; ++u) {
          mine[(v * N + u) * 64] = dg[v][u];
          mine[((kV + v) * N + u) * 64] = db[v][u];
        }
    }
    __syncthreads();
    if (sub) return;
#pragma unroll
    for (int w = 0; w < kRows - 1; ++w)
#pragma unroll
      for (int v = 0; v < kV; ++v)
#pragma unroll
        for (int u = 0; u < N; ++u) {
          const A* his = joined + w * (2 * kV * N * 64) + t;
          dg[v][u] += his[(v * N + u) * 64];
          db[v][u] += his[((kV + v) * N + u) * 64];
        }
  }
  A* p = part + (int64_t)blockIdx.x * 2 * cols;
  typedef A S __attribute__((ext_vector_type(16 / sizeof(A)), aligned(sizeof(A))));
  constexpr int NS = 16 / (int)sizeof(A);   // sums of a 16-byte store
#pragma unroll
  for (int v = 0; v < kV; ++v) {
    const int64_t c = (int64_t)(v * kT + t) * N;
    if (c + N <= cols) {
#pragma unroll
      for (int u = 0; u < N; u += NS) {
        S a, b;
#pragma unroll
        for (int e = 0; e < NS; ++e) {
          a[e] = dg[v][u + e];
          b[e] = db[v][u + e];
        }
        *reinterpret_cast<S*>(p + c + u) = a;
        *reinterpret_cast<S*>(p + cols + c + u) = b;
      }
    } else {
#pragma unroll
      for (int u = 0; u < N; ++u)
        if (c + u < cols) {
          p[c + u] = dg[v][u];
          p[cols + c + u] = db[v][u];
        }
    }
  }
}

// Rows too long for registers: dx from two passes over the row.
template <typename T>
__global__ __launch_bounds__(1024) void layernorm_backward_long_kernel(
    int64_t cols, const T* dy, int64_t lddy, const T* x, int64_t ldx,
    const T* __restrict__ gamma, const typename AccOf<T>::type* __restrict__ mean,
    const typename AccOf<T>::type* __restrict__ rstd, T* dx, int64_t lddx) {
  typedef typename AccOf<T>::type A;
  constexpr int N = Vec<T>::N, kT = 1024;
  __shared__ A slots[2][kT / 64];
  const int64_t row = blockIdx.x;
  const T* xr = x + row * ldx;
  const T* dyr = dy + row * lddy;
  const A mu = mean[row], rho = rstd[row], inv = (A)1 / (A)cols;
  A a[N], d[N], w[N], s1 = 0, s2 = 0;
  auto values = [&](int64_t c) {   // a = xh, d = g
    load_vec<T, A>(xr, c, cols, a);
    load_vec<T, A>(dyr, c, cols, d);
    if (gamma) load_vec<T, A>(gamma, c, cols, w);
    const int nv = valid<N>(c, cols);
#pragma unroll
    for (int u = 0; u < N; ++u) {
      a[u] = u < nv ? (a[u] - mu) * rho : (A)0;
      if (gamma) d[u] *= w[u];
    }
  };
  for (int64_t c = (int64_t)threadIdx.x * N; c < cols; c += kT * N) {
    values(c);
#pragma unroll
    for (int u = 0; u < N; ++u) {
      s1 += d[u] * a[u];
      s2 += d[u];
    }
  }
  const A c1 = row_all<kT>(s1, SumOp(), slots[0]) * inv;
  const A c2 = row_all<kT>(s2, SumOp(), slots[1]) * inv;
  for (int64_t c = (int64_t)threadIdx.x * N; c < cols; c += kT * N) {
    values(c);
#pragma unroll
    for (int u = 0; u < N; ++u) a[u] = rho * (d[u] - c2 - a[u] * c1);
    store_vec<T, A>(dx + row * lddx, c, cols, a);
  }
}

// Column sums of the long rows: workgroup (bx, by) of G row groups takes 256 vectors of
// columns and rows by, by + G, ...
template <typename T>
__global__ __launch_bounds__(256) void layernorm_backward_cols_kernel(
    int64_t rows, int64_t cols, const T* __restrict__ dy, int64_t lddy,
    const T* __restrict__ x, int64_t ldx, const typename AccOf<T>::type* __restrict__ mean,
    const typename AccOf<T>::type* __restrict__ rstd, typename AccOf<T>::type* __restrict__ part) {
  typedef typename AccOf<T>::type A;
  constexpr int N = Vec<T>::N;
  const int64_t c = ((int64_t)blockIdx.x * 256 + threadIdx.x) * N;
  if (c >= cols) return;
  A dg[N], db[N], a[N], d[N];
#pragma unroll
  for (int u = 0; u < N; ++u) dg[u] = db[u] = 0;
  for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
    load_vec<T, A>(x + row * ldx, c, cols, a);
    load_vec<T, A>(dy + row * lddy, c, cols, d);
    const A mu = mean[row], rho = rstd[row];
#pragma unroll
    for (int u = 0; u < N; ++u) {
      dg[u] += d[u] * ((a[u] - mu) * rho);
      db[u] += d[u];
    }
  }
  A* p = part + (int64_t)blockIdx.y * 2 * cols;
#pragma unroll
  for (int u = 0; u < N; ++u)
    if (c + u < cols) {
      p[c + u] = dg[u];
      p[cols + c + u] = db[u];
    }
}

// dgamma and dbeta from the G partials of each column, added in a fixed order: slice s of
// 16 adds partials s, s + 16, ... in order, then the slices are added in order.  Workgroup:
// 16 columns (of the 2 cols values, from workgroup `first` of all on) x 16 slices.
template <typename T>
__global__ __launch_bounds__(256) void layernorm_join_kernel(
    int64_t first, int64_t cols, int groups, const typename AccOf<T>::type* __restrict__ part,
    T* __restrict__ dgamma, T* __restrict__ dbeta) {
  typedef typename AccOf<T>::type A;
  __shared__ A sums[16][17];
  const int cl = threadIdx.x & 15, slice = threadIdx.x >> 4;
  const int64_t c = (first + blockIdx.x) * 16 + cl;
  A s = 0;
  if (c < 2 * cols) {
    const A* p = part + c;
    const int64_t ld = 2 * cols;
    int g = slice;
    for (; g + 112 < groups; g += 128) {   // eight partials asked for at once
      A a[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) a[u] = p[(g + 16 * u) * ld];
#pragma unroll
      for (int u = 0; u < 8; ++u) s += a[u];
    }
    for (; g < groups; g += 16) s += p[g * ld];
  }
  sums[slice][cl] = s;
  __syncthreads();
  if (slice == 0 && c < 2 * cols) {
    for (int w = 1; w < 16; ++w) s += sums[w][cl];
    if (c < cols) {
      if (dgamma) dgamma[c] = (T)s;
    } else {
      if (dbeta) dbeta[c - cols] = (T)s;
    }
  }
}

// Threads and vectors per thread for a row of `vecs` 16-byte vectors: of the shapes that hold the
// row, the one with the fewest threads and vectors (a reduction across waves, and every idle
// lane, costs a row the same whatever it holds).  8192 rows of bf16, us:
//   vecs   64x1  64x2  64x4  256x1  256x2  256x4  1024x1  1024x2
//     64    7.6   8.5  10.5   13.4   17.2
//    128         10.9  12.4   15.4   18.5   27.1    44.0
//    256               18.2   18.7   21.1   29.4    45.7    61.4
//    512                             27.0   35.3    51.2    63.3
//   1024                                    51.0    60.9    71.4
// With 8 rows all are within a microsecond of each other (256 vectors: 6.5 with 64x4, 5.1 with
// 256x2).  512x2 and 512x4 were no better but for 1024 vectors (46.5).
#define OZK_ROW_SHAPES(GO)            \
  if (vecs <= 64) GO(64, 1);          \
  else if (vecs <= 128) GO(64, 2);    \
  else if (vecs <= 256) GO(64, 4);    \
  else if (vecs <= 512) GO(256, 2);   \
  else if (vecs <= 1024) GO(256, 4);  \
  else if (vecs <= 2048) GO(1024, 2); \
  else GO(1024, 4)
constexpr int64_t kRowVecs = 4096;   // vectors a workgroup holds
// Rows of a launch: one takes fewer than 2^32 threads, a row up to 1024 of them.
constexpr int64_t kRowsOnce = 1 << 21;
constexpr int64_t kJoinsOnce = 1 << 23;   // and workgroups of 256 threads

template <typename T>
int layernorm_t(int64_t rows, int64_t cols, const void* x, int64_t ldx, const void* gamma,
                const void* beta, double eps, void* y, int64_t ldy, void* mean, void* rstd,
                hipStream_t s) {
  typedef typename AccOf<T>::type A;
  const int64_t vecs = (cols + Vec<T>::N - 1) / Vec<T>::N;
  const T *xt = (const T*)x, *gt = (const T*)gamma, *bt = (const T*)beta;
  if (rows > kRowsOnce) {
    const int st = layernorm_t<T>(kRowsOnce, cols, x, ldx, gamma, beta, eps, y, ldy, mean, rstd, s);
    if (st != OZK_OK) return st;
    return layernorm_t<T>(rows - kRowsOnce, cols, xt + kRowsOnce * ldx, ldx, gamma, beta, eps,
                          (T*)y + kRowsOnce * ldy, ldy, mean ? (A*)mean + kRowsOnce : nullptr,
                          rstd ? (A*)rstd + kRowsOnce : nullptr, s);
  }
  if (vecs > kRowVecs) {
    hipLaunchKernelGGL((layernorm_long_kernel<T>), dim3((unsigned)rows), dim3(1024), 0, s, cols,
                       xt, ldx, gt, bt, (A)eps, (T*)y, ldy, (A*)mean, (A*)rstd);
  } else {
#define OZK_LN(NT, NV)                                                                         \
  hipLaunchKernelGGL((layernorm_kernel<T, NT, NV>),                                            \
                     dim3((unsigned)(NT < 256 ? (rows + 3) / 4 : rows)),                       \
                     dim3(NT < 256 ? 256 : NT), 0, s, rows, cols, xt, ldx, gt, bt, (A)eps,     \
                     (T*)y, ldy, (A*)mean, (A*)rstd)
    OZK_ROW_SHAPES(OZK_LN);
#undef OZK_LN
  }
  return hipGetLastError() == hipSuccess ? OZK_OK : OZK_EHIP;
}

// Threads of a row and values per thread for the codes.  The reductions and the fp64 divisions
// cost a wave the same whatever it holds, so many rows take up to 32 values per thread (4096 x
// 8192 with the norm, bf16 / fp32: 42 / 76 us with 16 / 8 values per thread); a few rows leave
// the chip empty and spread wider (1 x 8192: 6.0 us, 8.0 with 32 values a thread, 7.1 with 8).
template <typename T, bool kNorm>
int int8quant_t(int64_t rows, int64_t cols, const void* x, int64_t ldx, const void* gamma,
                const void* beta, double eps, int8_t* q, int64_t ldq, float* scale,
                hipStream_t s) {
  constexpr int N = Vec<T>::N;
  const T *xt = (const T*)x, *gt = (const T*)gamma, *bt = (const T*)beta;
  const bool wide = rows < 256;
  if (rows > kRowsOnce) {
    const int st = int8quant_t<T, kNorm>(kRowsOnce, cols, x, ldx, gamma, beta, eps, q, ldq, scale,
                                         s);
    if (st != OZK_OK) return st;
    return int8quant_t<T, kNorm>(rows - kRowsOnce, cols, xt + kRowsOnce * ldx, ldx, gamma, beta,
                                 eps, q + kRowsOnce * ldq, ldq, scale + kRowsOnce, s);
  }
#define OZK_Q(NT, VALUES)                                                                      \
  hipLaunchKernelGGL((int8quant_kernel<T, NT, VALUES / N, kNorm>),                             \
                     dim3((unsigned)(NT < 256 ? (rows + 3) / 4 : rows)),                       \
                     dim3(NT < 256 ? 256 : NT), 0, s, rows, cols, xt, ldx, gt, bt, eps, q,     \
                     ldq, scale)
  constexpr int kMost = N == 2 ? 16 : 32;   // fp64 rows: their values' registers
  if (cols > 1024 * kMost)
    hipLaunchKernelGGL((int8quant_long_kernel<T, kNorm>), dim3((unsigned)rows), dim3(1024), 0, s,
                       cols, xt, ldx, gt, bt, eps, q, ldq, scale);
  else if (cols <= 512) OZK_Q(64, 8);
  else if (cols <= 2048 && wide) OZK_Q(256, 8);
  else if (cols <= 8192 && wide) OZK_Q(512, 16);
  else if (cols <= 1024) OZK_Q(64, 16);
  else if (cols <= 2048) OZK_Q(64, 32);
  else if (cols <= 4096) OZK_Q(256, 16);
  else if (cols <= 8192) OZK_Q(256, 32);
  else if (cols <= 16384) OZK_Q(1024, 16);
  else if constexpr (kMost == 32) OZK_Q(1024, 32);
#undef OZK_Q
  return hipGetLastError() == hipSuccess ? OZK_OK : OZK_EHIP;
}

// Vectors a backward workgroup holds per row (its column sums take registers too, so a thread
// holds two at most: 8192 rows of bf16 with 512 vectors take 43 us with 256x2, 54 with 1024x1, 105
// with 256x4; with 160 vectors 34 with 256x1, 30 with 64x4, with 256 26 and 28).
constexpr int64_t kBackwardVecs = 2048;

template <typename T>
int layernorm_backward_t(int64_t rows, int64_t cols, const void* dy, int64_t lddy,
                         const void* x, int64_t ldx, const void* gamma, const void* mean,
                         const void* rstd, void* dx, int64_t lddx, void* dgamma, void* dbeta,
                         void* workspace, hipStream_t s) {
  typedef typename AccOf<T>::type A;
  const int64_t vecs = (cols + Vec<T>::N - 1) / Vec<T>::N;
  const bool in_registers = vecs <= kBackwardVecs;
  const int rows_once = in_registers ? (vecs <= 128 ? 4 : 1) : 8;
  int groups = (int)((rows + rows_once - 1) / rows_once);
  if (groups > layernorm_backward_groups(rows)) groups = layernorm_backward_groups(rows);
  // workgroups of 1024 threads take a CU each: a second round of them would only leave more
  // partials (4096 x 16384 bf16: 140 us with 512, 119 with 256; 8192^2 92 and 84)
  if (in_registers && vecs > 512 && groups > 256) groups = 256;
  A* part = dgamma || dbeta ? (A*)workspace : nullptr;
  const T *dyt = (const T*)dy, *xt = (const T*)x, *gt = (const T*)gamma;
  const A *mt = (const A*)mean, *rt = (const A*)rstd;
  if (rows == 0) {
    part = nullptr;
  } else if (!in_registers) {
    // the column sums first: dx may take the place of dy or x
    if (part)
      hipLaunchKernelGGL((layernorm_backward_cols_kernel<T>),
                         dim3((unsigned)((vecs + 255) / 256), (unsigned)groups), dim3(256), 0, s,
                         rows, cols, dyt, lddy, xt, ldx, mt, rt, part);
    for (int64_t r0 = 0; dx && r0 < rows; r0 += kRowsOnce)
      hipLaunchKernelGGL((layernorm_backward_long_kernel<T>),
                         dim3((unsigned)(rows - r0 < kRowsOnce ? rows - r0 : kRowsOnce)),
                         dim3(1024), 0, s, cols, dyt + r0 * lddy, lddy, xt + r0 * ldx, ldx, gt,
                         mt + r0, rt + r0, (T*)dx + r0 * lddx, lddx);
  } else {
#define OZK_LNB(NT, NV)                                                                       \
  hipLaunchKernelGGL((layernorm_backward_kernel<T, NT, NV>), dim3((unsigned)groups),          \
                     dim3(NT < 256 ? 256 : NT), 0, s, rows, cols, dyt, lddy, xt, ldx, gt, mt, \
                     rt, (T*)dx, lddx, part)
    if (vecs <= 64) OZK_LNB(64, 1);
    else if (vecs <= 128) OZK_LNB(64, 2);
    else if (vecs <= 256) OZK_LNB(256, 1);
    else if (vecs <= 512) OZK_LNB(256, 2);
    else if (vecs <= 1024) OZK_LNB(1024, 1);
    else OZK_LNB(1024, 2);
#undef OZK_LNB
  }
  // zeros where there are no rows
  const int64_t joins = dgamma || dbeta ? (2 * cols + 15) / 16 : 0;
  for (int64_t b = 0; b < joins; b += kJoinsOnce)
    hipLaunchKernelGGL((layernorm_join_kernel<T>),
                       dim3((unsigned)(joins - b < kJoinsOnce ? joins - b : kJoinsOnce)),
                       dim3(256), 0, s, b, cols, groups, part, (T*)dgamma, (T*)dbeta);
  return hipGetLastError() == hipSuccess ? OZK_OK : OZK_EHIP;
}

}  // namespace

// Row groups of the backward pass at most: two workgroups per CU, each leaving one partial of
// the column sums.
int layernorm_backward_groups(int64_t rows) { return (int)(rows < 512 ? rows : 512); }

int launch_layernorm(int64_t rows, int64_t cols, int type, const void* x, int64_t ldx,
                     const void* gamma, const void* beta, double eps, void* y, int64_t ldy,
                     void* mean, void* rstd, hipStream_t s) {
  switch (type) {
    case OZK_F64:
      return layernorm_t<double>(rows, cols, x, ldx, gamma, beta, eps, y, ldy, mean, rstd, s);
    case OZK_F32:
      return layernorm_t<float>(rows, cols, x, ldx, gamma, beta, eps, y, ldy, mean, rstd, s);
    case OZK_F16:
      return layernorm_t<f16_t>(rows, cols, x, ldx, gamma, beta, eps, y, ldy, mean, rstd, s);
    default:
      return layernorm_t<bf16_t>(rows, cols, x, ldx, gamma, beta, eps, y, ldy, mean, rstd, s);
  }
}

int launch_int8quant(int64_t rows, int64_t cols, int type, const void* x, int64_t ldx, int norm,
                     const void* gamma, const void* beta, double eps, int8_t* q, int64_t ldq,
                     float* scale, hipStream_t s) {
#define OZK_QT(T)                                                                             \
  return norm ? int8quant_t<T, true>(rows, cols, x, ldx, gamma, beta, eps, q, ldq, scale, s)  \
              : int8quant_t<T, false>(rows, cols, x, ldx, gamma, beta, eps, q, ldq, scale, s)
  switch (type) {
    case OZK_F64: OZK_QT(double);
    case OZK_F32: OZK_QT(float);
    case OZK_F16: OZK_QT(f16_t);
    default: OZK_QT(bf16_t);
  }
#undef OZK_QT
}

int launch_layernorm_backward(int64_t rows, int64_t cols, int type, const void* dy, int64_t lddy,
                              const void* x, int64_t ldx, const void* gamma, const void* mean,
                              const void* rstd, void* dx, int64_t lddx, void* dgamma, void* dbeta,
                              void* workspace, hipStream_t s) {
#define OZK_BT(T)                                                                            \
  return layernorm_backward_t<T>(rows, cols, dy, lddy, x, ldx, gamma, mean, rstd, dx, lddx,  \
                                 dgamma, dbeta, workspace, s)
  switch (type) {
    case OZK_F64: OZK_BT(double);
    case OZK_F32: OZK_BT(float);
    case OZK_F16: OZK_BT(f16_t);
    default: OZK_BT(bf16_t);
  }
#undef OZK_BT
}

}  // namespace ozk
