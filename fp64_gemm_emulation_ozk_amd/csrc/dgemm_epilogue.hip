// The emulated fp64 product's epilogue, and what its gradient needs beside two products.
//
// Forward: Z = A B + 1 b^T, C = act(Z) + R.  The reconstruction finishes one output per
// lane in a register, so bias, activation and residual are applied there: C (and Z, if
// kept for the backward pass) is written once, the product alone never.  8192^2, r = 16, with
// bias, Z, gelu_tanh and residual: 0.68 ms, 2.7 GB at 4.0 TB/s; the reconstruction alone 0.41,
// 1.6 GB at 4.0.  The loads of the bias and the residual are asked for before the lift.
// Backward: G = dC * act'(Z) elementwise, db = column sums of G; dA = G B^T and dB = A^T G
// are products of the same kind.
#include "activation.h"
#include "crt_core.h"

namespace ozk {
namespace {

// Which activations a kernel holds.  Each set is its own kernel because of the registers:
// with erfc in it all ran three waves per SIMD, against six without any.
enum ActSet { kSimple, kExp, kErfc };   // none, relu; gelu_tanh, silu; gelu
inline ActSet act_set(int act) {
  return act == OZK_ACT_GELU ? kErfc
                             : (act == OZK_ACT_GELU_TANH || act == OZK_ACT_SILU ? kExp : kSimple);
}

// The residual may be C itself: a lane reads its element before it writes it.
template <ActSet kSet>
struct Finish {
  DgemmEpilogue E;
  double* c;
  int64_t ldc;
  struct Asked {
    double bias, residual;
  };
  __device__ __forceinline__ Asked ask(int64_t i, int64_t j) const {
    return {E.bias ? E.bias[j] : 0.0, E.residual ? E.residual[i * E.ldr + j] : 0.0};
  }
  __device__ __forceinline__ void operator()(int64_t i, int64_t j, double v,
                                             const Asked& a) const {
    if (E.bias) v += a.bias;
    if (E.z) E.z[i * E.ldz + j] = v;
    if (kSet == kErfc) v = activate(v, OZK_ACT_GELU);
    else if (kSet == kExp) v = activate(v, E.act == OZK_ACT_SILU ? OZK_ACT_SILU : OZK_ACT_GELU_TANH);
    else if (E.act == OZK_ACT_RELU) v = activate(v, OZK_ACT_RELU);
    if (E.residual) v += a.residual;
    c[i * ldc + j] = v;
  }
};

template <int R, ActSet kSet>
__global__ __launch_bounds__(256) void crt_epilogue_kernel(
    int64_t m, int64_t n, const int8_t* __restrict__ res, int64_t ldr, int64_t stride_r,
    const int32_t* __restrict__ ea, const int32_t* __restrict__ eb, DgemmEpilogue E, double* c,
    int64_t ldc) {
  crt_outputs<R, int8_t>(m, n, ldr, res, ldr, stride_r, ea, eb, Finish<kSet>{E, c, ldc});
}

// Two products without an epilogue in one launch: grid.y picks the one.
struct Plain {
  int64_t m, n, ldr, stride_r;
  const int8_t* res;
  const int32_t *ea, *eb;
  double* c;
  int64_t ldc;
};

struct PlainStore {
  double* c;
  int64_t ldc;
  struct Nothing {};
  __device__ __forceinline__ Nothing ask(int64_t, int64_t) const { return {}; }
  __device__ __forceinline__ void operator()(int64_t i, int64_t j, double v, Nothing) const {
    c[i * ldc + j] = v;
  }
};

template <int R>
__global__ __launch_bounds__(256) void crt_pair_kernel(Plain a, Plain b) {
  const Plain p = blockIdx.y ? b : a;
  crt_outputs<R, int8_t>(p.m, p.n, p.ldr, p.res, p.ldr, p.stride_r, p.ea, p.eb,
                         PlainStore{p.c, p.ldc});
}

template <int R>
void launch_r(dim3 grid, hipStream_t s, int64_t m, int64_t n, const int8_t* res, int64_t ldr,
              int64_t stride_r, const int32_t* ea, const int32_t* eb, const DgemmEpilogue& E,
              double* c, int64_t ldc) {
#define OZK_SET(SET)                                                                           \
  hipLaunchKernelGGL((crt_epilogue_kernel<R, SET>), grid, dim3(256), 0, s, m, n, res, ldr,     \
                     stride_r, ea, eb, E, c, ldc)
  const ActSet set = act_set(E.act);
  if (set == kErfc) OZK_SET(kErfc);
  else if (set == kExp) OZK_SET(kExp);
  else OZK_SET(kSimple);
#undef OZK_SET
}

// A short gradient's G and the whole column sums in one launch: 16 columns x 64 slices of rows per
// workgroup, slice s taking rows s, s + 64, ..., the slices added in a fixed order.  (A gradient
// of 167 x 247 x 512 took 39 us with chunks and their join, and two launches of the
// reconstruction; so 28.)  The sums alone, silu, this launch / chunks and their join, us:
//   rows            256         768         1024        1536        2048
//   256 columns    5.6 / 9.4  10.1 / 10.1  12.7 / 11.0  17.3 / 11.5  21.8 / 10.4
//   4096 columns   6.2 / 10.3 12.8 / 15.7  15.7 / 20.1  21.4 / 26.2  28.5 / 31.5
// (few columns leave compute units idle here; 1024 stands between where either is the faster).
constexpr int64_t kShortRows = 1024;

__global__ __launch_bounds__(1024) void act_grad_short_kernel(
    int64_t m, int64_t n, const double* __restrict__ dc, int64_t lddc,
    const double* __restrict__ z, int64_t ldz, int act, double* __restrict__ g,
    double* __restrict__ dbias) {
  __shared__ double sums[64][17];
  const int cl = threadIdx.x & 15, slice = threadIdx.x >> 4;
  const int64_t c = (int64_t)blockIdx.x * 16 + cl;
  double sum = 0;
  if (c < n) {
#pragma unroll 4
    for (int64_t i = slice; i < m; i += 64) {
      double v = dc[i * lddc + c];
      if (act != OZK_ACT_NONE) v *= activate_slope(z[i * ldz + c], act);
      if (g) g[i * n + c] = v;
      sum += v;
    }
  }
  sums[slice][cl] = sum;
  __syncthreads();
  if (slice < 4) {   // 64 slices to four, to one
    for (int p = 1; p < 16; ++p) sum += sums[slice + 4 * p][cl];
    sums[slice][cl] = sum;
  }
  __syncthreads();
  if (slice == 0 && c < n && dbias)
    dbias[c] = (sums[0][cl] + sums[1][cl]) + (sums[2][cl] + sums[3][cl]);
}

// Column c of a chunk of rows per thread: G, and the chunk's sum of G.  1500 x 2050 with silu:
// 19 us with eight rows' loads together, 22 to 26 with four (74 MB would take 13.5).
__global__ __launch_bounds__(256) void act_grad_kernel(
    int64_t m, int64_t n, int64_t chunk, const double* __restrict__ dc, int64_t lddc,
    const double* __restrict__ z, int64_t ldz, int act, double* __restrict__ g,
    double* __restrict__ part) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= n) return;
  const int64_t r0 = blockIdx.y * chunk, r1 = r0 + chunk < m ? r0 + chunk : m;
  double sum = 0;
  for (int64_t i0 = r0; i0 < r1; i0 += 8) {   // eight rows asked for at once
    double v[8], w[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int64_t i = i0 + u < r1 ? i0 + u : r1 - 1;
      v[u] = dc[i * lddc + c];
      w[u] = act != OZK_ACT_NONE ? z[i * ldz + c] : 0.0;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (i0 + u >= r1) break;   // uniform
      if (act != OZK_ACT_NONE) v[u] *= activate_slope(w[u], act);
      if (g) g[(i0 + u) * n + c] = v[u];
      sum += v[u];
    }
  }
  if (part) part[blockIdx.y * n + c] = sum;
}

// out[c] = the chunks' sums of column c, in a fixed order: 16 columns x 16 slices per
// workgroup, slice s adding chunks s, s + 16, ..., then the slices in order.
__global__ __launch_bounds__(256) void column_join_kernel(int64_t n, int chunks,
                                                          const double* __restrict__ part,
                                                          double* __restrict__ out) {
  __shared__ double sums[16][17];
  const int cl = threadIdx.x & 15, slice = threadIdx.x >> 4;
  const int64_t c = (int64_t)blockIdx.x * 16 + cl;
  double s = 0;
  if (c < n) {
    const double* p = part + c;
    int g = slice;
    for (; g + 112 < chunks; g += 128) {   // eight sums asked for at once
      double a[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) a[u] = p[(g + 16 * u) * n];
#pragma unroll
      for (int u = 0; u < 8; ++u) s += a[u];
    }
    for (; g < chunks; g += 16) s += p[g * n];
  }
  sums[slice][cl] = s;
  __syncthreads();
  if (slice == 0 && c < n) {
    for (int w = 1; w < 16; ++w) s += sums[w][cl];
    out[c] = s;
  }
}

__global__ __launch_bounds__(256) void zero_rows_kernel(double* __restrict__ p, int64_t rows,
                                                        int64_t cols, int64_t ld) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * cols;
       i += (int64_t)gridDim.x * 256)
    p[i / cols * ld + i % cols] = 0.0;
}

}  // namespace

int launch_zero_rows(double* p, int64_t rows, int64_t cols, int64_t ld, hipStream_t s) {
  const int64_t blocks = (rows * cols + 255) / 256;
  hipLaunchKernelGGL(zero_rows_kernel, dim3((unsigned)(blocks < 65536 ? blocks : 65536)), dim3(256),
                     0, s, p, rows, cols, ld);
  return hipGetLastError() == hipSuccess ? OZK_OK : OZK_EHIP;
}

int launch_crt_epilogue(int64_t m, int64_t n, int r, const int8_t* res, int64_t ldr,
                        int64_t stride_r, const int32_t* ea, const int32_t* eb,
                        const DgemmEpilogue& E, double* c, int64_t ldc, hipStream_t s) {
  if (m <= 0 || n <= 0) return OZK_OK;
  const dim3 grid((unsigned)crt_blocks(m, n));
  switch (r) {
#define OZK_R(R)                                                             \
  case R:                                                                    \
    launch_r<R>(grid, s, m, n, res, ldr, stride_r, ea, eb, E, c, ldc);       \
    break
    OZK_R(1); OZK_R(2); OZK_R(3); OZK_R(4); OZK_R(5); OZK_R(6); OZK_R(7); OZK_R(8); OZK_R(9);
    OZK_R(10); OZK_R(11); OZK_R(12); OZK_R(13); OZK_R(14); OZK_R(15); OZK_R(16); OZK_R(17);
    OZK_R(18); OZK_R(19); OZK_R(20);
#undef OZK_R
    default: return OZK_EINVAL;
  }
  return hipGetLastError() == hipSuccess ? OZK_OK : OZK_EHIP;
}

int launch_crt_pair(const PlaneProduct* P, int r, const int32_t* const* ea,
                    const int32_t* const* eb, double* const* c, const int64_t* ldc, hipStream_t s) {
  Plain p[2];
  int64_t blocks = 0;
  for (int o = 0; o < 2; ++o) {
    p[o] = {P[o].m, P[o].n, P[o].np, P[o].m * P[o].np, P[o].res, ea[o], eb[o], c[o], ldc[o]};
    const int64_t own = crt_blocks(P[o].m, P[o].n);
    blocks = own > blocks ? own : blocks;
  }
  const dim3 grid((unsigned)blocks, 2);
  switch (r) {
#define OZK_R(R)                                                                          \
  case R:                                                                                 \
    hipLaunchKernelGGL((crt_pair_kernel<R>), grid, dim3(256), 0, s, p[0], p[1]);          \
    break
    OZK_R(1); OZK_R(2); OZK_R(3); OZK_R(4); OZK_R(5); OZK_R(6); OZK_R(7); OZK_R(8); OZK_R(9);
    OZK_R(10); OZK_R(11); OZK_R(12); OZK_R(13); OZK_R(14); OZK_R(15); OZK_R(16); OZK_R(17);
    OZK_R(18); OZK_R(19); OZK_R(20);
#undef OZK_R
    default: return OZK_EINVAL;
  }
  return hipGetLastError() == hipSuccess ? OZK_OK : OZK_EHIP;
}

// Rows of a chunk: 16, or as many as leave at most 256 chunks.
int64_t act_grad_chunks(int64_t m) {
  const int64_t rows = (m + 255) / 256 > 16 ? (m + 255) / 256 : 16;
  return (m + rows - 1) / rows;
}

int launch_act_grad(int64_t m, int64_t n, const double* dc, int64_t lddc, const double* z,
                    int64_t ldz, int act, double* g, double* part, double* dbias,
                    hipStream_t s) {
  if (m <= kShortRows) {
    hipLaunchKernelGGL(act_grad_short_kernel, dim3((unsigned)((n + 15) / 16)), dim3(1024), 0, s, m,
                       n, dc, lddc, z, ldz, act, g, dbias);
    return hipGetLastError() == hipSuccess ? OZK_OK : OZK_EHIP;
  }
  const int64_t chunks = act_grad_chunks(m), chunk = (m + chunks - 1) / chunks;
  hipLaunchKernelGGL(act_grad_kernel, dim3((unsigned)((n + 255) / 256), (unsigned)chunks),
                     dim3(256), 0, s, m, n, chunk, dc, lddc, z, ldz, act, g,
                     dbias ? part : nullptr);
  if (dbias)
    hipLaunchKernelGGL(column_join_kernel, dim3((unsigned)((n + 15) / 16)), dim3(256), 0, s, n,
                       (int)chunks, part, dbias);
  return hipGetLastError() == hipSuccess ? OZK_OK : OZK_EHIP;
}

}  // namespace ozk
