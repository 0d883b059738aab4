// int8 linear layer: C = act(s t^T * (X W^T) + 1 b^T) + R, X m x k and W n x k int8 with K
// contiguous in both, s and t fp32 scales of their rows.  The int8 product is exact in
// int32 (k <= OZK_MAX_K); everything after it is fp32, rounded once to the output's type.
#include "activation.h"
#include "ozk_internal.h"
#include "rows.h"

namespace ozk {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef v4i v4i_bytes __attribute__((aligned(1)));

template <typename O>
struct Epilogue {
  int64_t m, n;
  const float* sx;
  const float* sw;
  const O* bias;
  const O* residual;   // may be c: an output is read by the lane that writes it, before
  int64_t ldr;
  O* c;
  int64_t ldc;
  int act;
};

// Four consecutive outputs of one row from their int32 sums.
template <typename O>
__device__ __forceinline__ void put4(const Epilogue<O>& E, int64_t row, int64_t col,
                                     const v4i& acc) {
  typedef O V __attribute__((ext_vector_type(4), aligned(sizeof(O))));
  typedef float F __attribute__((ext_vector_type(4), aligned(4)));
  if (row >= E.m || col >= E.n) return;
  const float s = E.sx[row];
  if (col + 4 <= E.n) {
    const F t = *reinterpret_cast<const F*>(E.sw + col);
    V b, r, o;
    if (E.bias) b = *reinterpret_cast<const V*>(E.bias + col);
    if (E.residual) r = *reinterpret_cast<const V*>(E.residual + row * E.ldr + col);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      float z = (float)acc[u] * s * t[u];
      if (E.bias) z += (float)b[u];
      z = activate(z, E.act);
      if (E.residual) z += (float)r[u];
      o[u] = (O)z;
    }
    *reinterpret_cast<V*>(E.c + row * E.ldc + col) = o;
    return;
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int64_t j = col + u;
    if (j >= E.n) continue;
    float z = (float)acc[u] * s * E.sw[j];
    if (E.bias) z += (float)E.bias[j];
    z = activate(z, E.act);
    if (E.residual) z += (float)E.residual[row * E.ldr + j];
    E.c[row * E.ldc + j] = (O)z;
  }
}

// 16 K bytes of a row, zero past k (any alignment).
__device__ __forceinline__ v4i load16(const int8_t* __restrict__ p, int64_t h, int64_t k) {
  if (h + 16 <= k) return *reinterpret_cast<const v4i_bytes*>(p + h);
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int u = 0; u < 16; ++u)
    if (h + u < k) w[u >> 2] |= (uint32_t)(uint8_t)p[h + u] << (8 * (u & 3));
  return v4i{(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
}

// Few rows: workgroup = 16 columns of C x 16 kMT rows, its kWaves waves splitting K in
// steps of 128 bytes taken in turn.  Operands go from global memory to the matrix core's
// registers directly: lane l of a fragment holds row l % 16 and 16 bytes of K.
template <typename O, int kMT, int kWaves>
__global__ __launch_bounds__(64 * kWaves) void int8linear_few_kernel(
    int64_t k, const int8_t* __restrict__ x, int64_t ldx, const int8_t* __restrict__ w,
    int64_t ldw, Epilogue<O> E) {
  __shared__ v4i sums[kWaves][kMT][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t tiles_n = (E.n + 15) / 16;
  const int64_t col0 = blockIdx.x % tiles_n * 16, row0 = blockIdx.x / tiles_n * 16 * kMT;
  const int64_t wr = col0 + (lane & 15) < E.n ? col0 + (lane & 15) : E.n - 1;
  const int8_t* wp = w + wr * ldw;
  const int8_t* xp[kMT];
#pragma unroll
  for (int i = 0; i < kMT; ++i) {
    const int64_t r = row0 + 16 * i + (lane & 15);
    xp[i] = x + (r < E.m ? r : E.m - 1) * ldx;
  }
  v4i acc[kMT];
#pragma unroll
  for (int i = 0; i < kMT; ++i) acc[i] = v4i{0, 0, 0, 0};
  for (int64_t h0 = (int64_t)wave * 128; h0 < k; h0 += 128 * kWaves) {
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const int64_t h = h0 + 64 * kk + 16 * (lane >> 4);
      const v4i b = load16(wp, h, k);
#pragma unroll
      for (int i = 0; i < kMT; ++i)
        acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b, load16(xp[i], h, k), acc[i], 0, 0, 0);
    }
  }
#pragma unroll
  for (int i = 0; i < kMT; ++i) sums[wave][i][lane] = acc[i];
  __syncthreads();
  for (int i = wave; i < kMT; i += kWaves) {
    v4i s = sums[0][i][lane];
#pragma unroll
    for (int v = 1; v < kWaves; ++v) s += sums[v][i][lane];
    put4(E, row0 + 16 * i + (lane & 15), col0 + 4 * (lane >> 4), s);
  }
}

template <typename O>
int int8linear_t(int64_t m, int64_t n, int64_t k, const int8_t* x, int64_t ldx, const float* sx,
                 const int8_t* w, int64_t ldw, const float* sw, const void* bias, int act,
                 const void* residual, int64_t ldr, void* c, int64_t ldc, void* workspace,
                 hipStream_t s) {
  const Epilogue<O> E{m, n, sx, sw, (const O*)bias, (const O*)residual, ldr, (O*)c, ldc, act};
  const int64_t mt = m <= 16 ? 1 : (m <= 32 ? 2 : 4);
  const int64_t tiles = (n + 15) / 16 * ((m + 16 * mt - 1) / (16 * mt));
  if (tiles > 0x7fffffff) return OZK_EUNSUPPORTED;
#define OZK_FEW(MT)                                                                        \
  hipLaunchKernelGGL((int8linear_few_kernel<O, MT, 8>), dim3((unsigned)tiles), dim3(512), 0, s, \
                     k, x, ldx, w, ldw, E)
  if (mt == 1) OZK_FEW(1);
  else if (mt == 2) OZK_FEW(2);
  else OZK_FEW(4);
#undef OZK_FEW
  return hipGetLastError() == hipSuccess ? OZK_OK : OZK_EHIP;
}

}  // namespace

size_t int8linear_workspace(int64_t, int64_t, int64_t) { return 0; }

int launch_int8linear(int64_t m, int64_t n, int64_t k, const int8_t* x, int64_t ldx,
                      const float* sx, const int8_t* w, int64_t ldw, const float* sw,
                      const void* bias, int act, const void* residual, int64_t ldr, int type,
                      void* c, int64_t ldc, void* workspace, hipStream_t s) {
  switch (type) {
    case OZK_F32:
      return int8linear_t<float>(m, n, k, x, ldx, sx, w, ldw, sw, bias, act, residual, ldr, c,
                                 ldc, workspace, s);
    case OZK_F16:
      return int8linear_t<f16_t>(m, n, k, x, ldx, sx, w, ldw, sw, bias, act, residual, ldr, c,
                                 ldc, workspace, s);
    default:
      return int8linear_t<bf16_t>(m, n, k, x, ldx, sx, w, ldw, sw, bias, act, residual, ldr, c,
                                  ldc, workspace, s);
  }
}

}  // namespace ozk
