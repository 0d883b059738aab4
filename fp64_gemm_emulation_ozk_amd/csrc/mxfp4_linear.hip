// Linear layer and gated feed-forward block on microscaled 4-bit operands:
//   C = act(X W^T + 1 b^T) + R,   and, W = [Wg; Wu],   C = act(X Wg^T + 1 bg^T) * (X Wu^T + 1 bu^T)
// X m x k and W n (2n) x k as MX FP4 lines.  A v_mfma_scale_f32_16x16x128_f8f6f4 takes 32 codes
// and their scale from every lane, so a lane's 16 bytes of a line are one block; sums are fp32,
// and what follows them is fp32, rounded once to the output's type.
#include "activation.h"
#include "ozk_internal.h"
#include "rows.h"
#include "tile_walk.h"

namespace ozk {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v4f_words __attribute__((ext_vector_type(4), aligned(4)));
typedef int v8i __attribute__((ext_vector_type(8)));

// One block's worth of a step for every lane: half kH of the lane's 32 bytes of the step, scale
// byte kH of its two.  Lane (row lane % 16, quarter lane / 16) gives 32 codes of its line; lane l of
// the sum holds line l % 16 of x and lines 4 (l / 16) .. + 3 of w.
template <int kH>
__device__ __forceinline__ v4f mfma_mx(const v4i& w, int sw, const v4i& x, int sx, const v4f& c) {
  const v8i w8 = {w[0], w[1], w[2], w[3], 0, 0, 0, 0};
  const v8i x8 = {x[0], x[1], x[2], x[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w8, x8, c, 4, 4, kH, sw, kH, sx);
}

// Lines of codes with their scales.
struct Lines {
  const uint8_t* codes;
  int64_t ld;
  const uint8_t* scales;
  int64_t lds;
};

template <typename O>
struct MxEpilogue {
  int64_t m, n;        // of C
  const O* bias;       // n, gated: 2 n
  const O* residual;   // may be c: an output is read by the lane that writes it, before
  int64_t ldr;
  O* c;
  int64_t ldc;
  int act;
};

// One output from its sum (gated: the sums of both projections).
template <bool kGated, typename O>
__device__ __forceinline__ void put1(const MxEpilogue<O>& E, int64_t row, int64_t col, float z,
                                     float up) {
  if (E.bias) z += (float)E.bias[col];
  z = activate32<sizeof(O) == 4>(z, E.act);
  if constexpr (kGated) {
    if (E.bias) up += (float)E.bias[E.n + col];
    z *= up;
  } else {
    if (E.residual) z += (float)E.residual[row * E.ldr + col];
  }
  E.c[row * E.ldc + col] = (O)z;
}

// Four consecutive outputs of one row.
template <bool kGated, typename O>
__device__ __forceinline__ void put4(const MxEpilogue<O>& E, int64_t row, int64_t col,
                                     const v4f& acc, const v4f& up) {
  typedef O V __attribute__((ext_vector_type(4), aligned(sizeof(O))));
  if (row >= E.m || col >= E.n) return;
  if (col + 4 <= E.n) {
    V b, bu, r, o;
    if (E.bias) {
      b = *reinterpret_cast<const V*>(E.bias + col);
      if constexpr (kGated) bu = *reinterpret_cast<const V*>(E.bias + E.n + col);
    }
    if constexpr (!kGated)
      if (E.residual) r = *reinterpret_cast<const V*>(E.residual + row * E.ldr + col);
    float z[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) z[u] = E.bias ? acc[u] + (float)b[u] : acc[u];
    activate_all<sizeof(O) == 4>(z, E.act);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if constexpr (kGated) z[u] *= E.bias ? up[u] + (float)bu[u] : up[u];
      else if (E.residual) z[u] += (float)r[u];
      o[u] = (O)z[u];
    }
    *reinterpret_cast<V*>(E.c + row * E.ldc + col) = o;
    return;
  }
#pragma unroll 1
  for (int u = 0; u < 3; ++u) {
    if (col + u >= E.n) break;
    put1<kGated>(E, row, col + u, u == 0 ? acc[0] : (u == 1 ? acc[1] : acc[2]),
                 u == 0 ? up[0] : (u == 1 ? up[1] : up[2]));
  }
}

// Any rows and columns: workgroup = 16 kMT rows x 16 kNT columns of C (gated: of both
// projections), its eight waves taking the K steps of 256 codes in turn.  Operands go from global
// memory to the matrix core's registers directly: a lane's 32 bytes of a step are two blocks.
template <typename O, bool kGated, int kMT, int kNT>
__global__ __launch_bounds__(512) void mxfp4_few_kernel(int64_t steps, Lines X, Lines W,
                                                        MxEpilogue<O> E, int64_t tiles_n) {
  constexpr int kWaves = 8, kG = kGated ? 2 : 1, kB = kNT * kG;
  __shared__ v4f sums[kWaves][kMT * kB][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t tile_m = blockIdx.x / tiles_n, tile_n = blockIdx.x - tile_m * tiles_n;
  const int64_t row0 = tile_m * (16 * kMT), col0 = tile_n * (16 * kNT);
  const int frow = lane & 15, quarter = lane >> 4;
  const uint8_t *wp[kB], *wsp[kB], *xp[kMT], *xsp[kMT];
#pragma unroll
  for (int j = 0; j < kB; ++j) {
    const int64_t c = col0 + 16 * (j % kNT) + frow;
    const int64_t r = (c < E.n ? c : E.n - 1) + (j / kNT) * E.n;
    wp[j] = W.codes + r * W.ld + 32 * quarter;
    wsp[j] = W.scales + r * W.lds + 2 * quarter;
  }
#pragma unroll
  for (int i = 0; i < kMT; ++i) {
    const int64_t r = row0 + 16 * i + frow;
    xp[i] = X.codes + (r < E.m ? r : E.m - 1) * X.ld + 32 * quarter;
    xsp[i] = X.scales + (r < E.m ? r : E.m - 1) * X.lds + 2 * quarter;
  }
  v4f acc[kMT][kB];
#pragma unroll
  for (int i = 0; i < kMT; ++i)
#pragma unroll
    for (int j = 0; j < kB; ++j) acc[i][j] = v4f{0, 0, 0, 0};
  for (int64_t t = wave; t < steps; t += kWaves) {
    v4i fb[2][kB], fa[2][kMT];
    int sb[kB], sa[kMT];
#pragma unroll
    for (int j = 0; j < kB; ++j) {
      fb[0][j] = *reinterpret_cast<const v4i*>(wp[j] + t * 128);
      fb[1][j] = *reinterpret_cast<const v4i*>(wp[j] + t * 128 + 16);
      sb[j] = *reinterpret_cast<const uint16_t*>(wsp[j] + t * 8);
    }
#pragma unroll
    for (int i = 0; i < kMT; ++i) {
      fa[0][i] = *reinterpret_cast<const v4i*>(xp[i] + t * 128);
      fa[1][i] = *reinterpret_cast<const v4i*>(xp[i] + t * 128 + 16);
      sa[i] = *reinterpret_cast<const uint16_t*>(xsp[i] + t * 8);
    }
#pragma unroll
    for (int i = 0; i < kMT; ++i)
#pragma unroll
      for (int j = 0; j < kB; ++j) {
        acc[i][j] = mfma_mx<0>(fb[0][j], sb[j], fa[0][i], sa[i], acc[i][j]);
        acc[i][j] = mfma_mx<1>(fb[1][j], sb[j], fa[1][i], sa[i], acc[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < kMT; ++i)
#pragma unroll
    for (int j = 0; j < kB; ++j) sums[wave][i * kB + j][lane] = acc[i][j];
  __syncthreads();
  for (int b = wave; b < kMT * kNT; b += kWaves) {
    const int i = b / kNT, j = b % kNT;
    v4f s[2];
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      s[g] = sums[0][i * kB + j + g * kNT][lane];
#pragma unroll
      for (int v = 1; v < kWaves; ++v) s[g] += sums[v][i * kB + j + g * kNT][lane];
    }
    put4<kGated>(E, row0 + 16 * i + frow, col0 + 16 * j + 4 * quarter, s[0], s[kG - 1]);
  }
}

template <typename O, bool kGated>
int linear_t(int64_t m, int64_t n, int64_t k, const Lines& X, const Lines& W, const void* bias,
             int act, const void* residual, int64_t ldr, void* c, int64_t ldc, hipStream_t s) {
  const MxEpilogue<O> E{m, n, (const O*)bias, (const O*)residual, ldr, (O*)c, ldc, act};
  const int64_t steps = (k + 255) / 256;
  constexpr int kNT = kGated ? 1 : 2;
  const int64_t tiles_n = (n + 16 * kNT - 1) / (16 * kNT);
  const int64_t tiles_m = m <= 16 ? 1 : (m + 31) / 32;
  // a launch takes fewer than 2^32 threads, 512 a workgroup
  if (tiles_m * tiles_n >= 1 << 23) return OZK_EUNSUPPORTED;
  const dim3 grid((unsigned)(tiles_m * tiles_n)), block(512);
  if (m <= 16)
    hipLaunchKernelGGL((mxfp4_few_kernel<O, kGated, 1, kNT>), grid, block, 0, s, steps, X, W, E,
                       tiles_n);
  else
    hipLaunchKernelGGL((mxfp4_few_kernel<O, kGated, 2, kNT>), grid, block, 0, s, steps, X, W, E,
                       tiles_n);
  return hipGetLastError() == hipSuccess ? OZK_OK : OZK_EHIP;
}

template <typename O>
int linear_any(int64_t m, int64_t n, int64_t k, const Lines& X, const Lines& W, bool gated,
               const void* bias, int act, const void* residual, int64_t ldr, void* c, int64_t ldc,
               hipStream_t s) {
  return gated ? linear_t<O, true>(m, n, k, X, W, bias, act, residual, ldr, c, ldc, s)
               : linear_t<O, false>(m, n, k, X, W, bias, act, residual, ldr, c, ldc, s);
}

}  // namespace

size_t mxfp4_linear_workspace(int64_t, int64_t, int64_t, bool) { return 0; }

int launch_mxfp4_linear(int64_t m, int64_t n, int64_t k, const uint8_t* x, int64_t ldx,
                        const uint8_t* xs, int64_t ldxs, const uint8_t* w, int64_t ldw,
                        const uint8_t* ws, int64_t ldws, bool gated, const void* bias, int act,
                        const void* residual, int64_t ldr, int type, void* c, int64_t ldc, void*,
                        hipStream_t s) {
  const Lines X{x, ldx, xs, ldxs}, W{w, ldw, ws, ldws};
  switch (type) {
    case OZK_F32:
      return linear_any<float>(m, n, k, X, W, gated, bias, act, residual, ldr, c, ldc, s);
    case OZK_F16:
      return linear_any<f16_t>(m, n, k, X, W, gated, bias, act, residual, ldr, c, ldc, s);
    default:
      return linear_any<bf16_t>(m, n, k, X, W, gated, bias, act, residual, ldr, c, ldc, s);
  }
}

}  // namespace ozk
