// The gated block in emulated fp64: Z = A [Bg Bu] + 1 b^T, C = act(Zg) * Zu, and what its gradient
// needs beside two products.
//
// Forward: both projections are one product of 2 n columns (A is deconstructed once); the
// reconstruction lifts column j of the gate and column n + j of the other in the same lane, so
// that bias, activation and the product of the two happen in registers: C (and Z, if kept for the
// backward pass) is written once, the products alone never.
// Backward: G = [dC * Zu * act'(Zg), dC * act(Zg)] elementwise, db = column sums of G;
// dA = G [Bg Bu]^T and d[Bg Bu] = A^T G are products of the same kind.
#include "activation.h"
#include "crt_core.h"

namespace ozk {
namespace {

// Which activations a kernel holds, as in the ungated epilogue: each set is its own kernel because
// of the registers.
enum ActSet { kSimple, kExp, kErfc };   // none, relu; gelu_tanh, silu; gelu

template <ActSet kSet>
__device__ __forceinline__ double activate_of(double z, int act) {
  if (kSet == kErfc) return activate(z, OZK_ACT_GELU);
  if (kSet == kExp) return activate(z, act == OZK_ACT_SILU ? OZK_ACT_SILU : OZK_ACT_GELU_TANH);
  return act == OZK_ACT_RELU ? activate(z, OZK_ACT_RELU) : z;
}

// Waves as in crt_outputs, 64 columns of C a group; the second projection's residues start at any
// address, n bytes on.  Bound as the ungated reconstruction, by the latency of residues from r
// planes with vector instructions close behind: 4096 x 2 8192, r = 16, silu, Z kept 482 to 499 us
// (1.9 GB, 3.8 TB/s); no activation takes as long.  Inside the product of 64 inner values (865 us
// in all), asking for the next group's residues before this one's lift 876, 4096 workgroups in
// place of 16384 885.
template <int R, ActSet kSet>
__global__ __launch_bounds__(256) void crt_gated_kernel(
    int64_t m, int64_t n, const int8_t* __restrict__ res, int64_t ldr, int64_t stride_r,
    const int32_t* __restrict__ ea, const int32_t* __restrict__ eb, DgemmEpilogue E,
    double* __restrict__ c, int64_t ldc) {
  using S = CrtShape<R>;
  const int lane = threadIdx.x & 63;
  const int half = lane >> 5, t = (lane & 31) >> 2, u = lane & 3;
  const uint32_t sel1 = u < 2 ? 0x05040100u : 0x03020706u;
  const uint32_t sel2 = (u & 1) ? 0x03070105u : 0x06020400u;
  const v4i a_op = *reinterpret_cast<const v4i*>(&d_crt.a[R][lane][0]);
  double m_limb[4];
#pragma unroll
  for (int p = 0; p < 4; ++p) m_limb[p] = d_rns.m_limb[R][p];
  const int64_t groups_row = (n + 63) / 64, waves = (int64_t)gridDim.x * 4;
  const int64_t g0 = __builtin_amdgcn_readfirstlane(blockIdx.x * 4 + (threadIdx.x >> 6));
  const int64_t adv_i = waves / groups_row, adv_g = waves - adv_i * groups_row;
  int64_t i = g0 / groups_row, jg = g0 - i * groups_row;
  while (i < m) {
    const int64_t j0 = jg * 64, j = j0 + lane;
    WordLoads<R> raw[2];
    load_words<R>(res + i * ldr + j0, stride_r, half, t, u, raw[0]);
    load_words<R, word_any>(res + i * ldr + n + j0, stride_r, half, t, u, raw[1]);
    const int64_t jc = j < n ? j : n - 1;
    const double bias[2] = {E.bias ? E.bias[jc] : 0.0, E.bias ? E.bias[n + jc] : 0.0};
    const int32_t e_i = ea[i], f[2] = {eb[jc], eb[n + jc]};
    double z[2];
#pragma unroll
    for (int o = 0; o < 2; ++o) {
      v4i b1v, b2v;
      transpose_words<R>(raw[o], sel1, sel2, b1v, b2v);
      double x[4];
      lift_limbs<R>(a_op, b1v, b2v, m_limb, x);
      z[o] = finish<S::kL, S::kBigTop>(x, e_i + f[o], e_i == INT32_MIN || f[o] == INT32_MIN);
      if (E.bias) z[o] += bias[o];
    }
    if (j < n) {
      if (E.z) {
        E.z[i * E.ldz + j] = z[0];
        E.z[i * E.ldz + n + j] = z[1];
      }
      c[i * ldc + j] = activate_of<kSet>(z[0], E.act) * z[1];
    }
    i += adv_i;
    jg += adv_g;
    if (jg >= groups_row) {
      jg -= groups_row;
      ++i;
    }
  }
}

template <int R>
void launch_r(dim3 grid, hipStream_t s, int64_t m, int64_t n, const int8_t* res, int64_t ldr,
              int64_t stride_r, const int32_t* ea, const int32_t* eb, const DgemmEpilogue& E,
              double* c, int64_t ldc) {
#define OZK_SET(SET)                                                                           \
  hipLaunchKernelGGL((crt_gated_kernel<R, SET>), grid, dim3(256), 0, s, m, n, res, ldr,        \
                     stride_r, ea, eb, E, c, ldc)
  if (E.act == OZK_ACT_GELU) OZK_SET(kErfc);
  else if (E.act == OZK_ACT_GELU_TANH || E.act == OZK_ACT_SILU) OZK_SET(kExp);
  else OZK_SET(kSimple);
#undef OZK_SET
}

// The gradients of both projections from dC and the pre-activations.
struct Pair {
  double gate, up;
};
__device__ __forceinline__ Pair gate_grad(double dc, double zg, double zu, int act) {
  return {dc * zu * activate_slope(zg, act), dc * activate(zg, act)};
}

// A column c of both halves of G per thread, a chunk of rows per workgroup, and the chunk's sums.
// Bound by memory: 1500 x 1025 (61 MB) 17.4 us, of which launch and latency are 4.
__global__ __launch_bounds__(256) void gate_grad_kernel(
    int64_t m, int64_t n, int64_t chunk, const double* __restrict__ dc, int64_t lddc,
    const double* __restrict__ z, int64_t ldz, int act, double* __restrict__ g,
    double* __restrict__ part) {
  const int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (c >= n) return;
  const int64_t r0 = blockIdx.y * chunk, r1 = r0 + chunk < m ? r0 + chunk : m;
  Pair sum{0, 0};
  for (int64_t i0 = r0; i0 < r1; i0 += 4) {   // four rows asked for at once
    double d[4], zg[4], zu[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int64_t i = i0 + v < r1 ? i0 + v : r1 - 1;
      d[v] = dc[i * lddc + c];
      zg[v] = z[i * ldz + c];
      zu[v] = z[i * ldz + n + c];
    }
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      if (i0 + v >= r1) break;   // uniform
      const Pair p = gate_grad(d[v], zg[v], zu[v], act);
      if (g) {
        g[(i0 + v) * 2 * n + c] = p.gate;
        g[(i0 + v) * 2 * n + n + c] = p.up;
      }
      sum.gate += p.gate;
      sum.up += p.up;
    }
  }
  if (part) {
    part[blockIdx.y * 2 * n + c] = sum.gate;
    part[blockIdx.y * 2 * n + n + c] = sum.up;
  }
}

}  // namespace

int launch_crt_gated(int64_t m, int64_t n, int r, const int8_t* res, int64_t ldr, int64_t stride_r,
                     const int32_t* ea, const int32_t* eb, const DgemmEpilogue& E, double* c,
                     int64_t ldc, hipStream_t s) {
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

int launch_gate_grad(int64_t m, int64_t n, const double* dc, int64_t lddc, const double* z,
                     int64_t ldz, int act, double* g, double* part, double* dbias,
                     hipStream_t s) {
  const int64_t chunks = act_grad_chunks(m), chunk = (m + chunks - 1) / chunks;
  hipLaunchKernelGGL(gate_grad_kernel, dim3((unsigned)((n + 255) / 256), (unsigned)chunks),
                     dim3(256), 0, s, m, n, chunk, dc, lddc, z, ldz, act, g,
                     dbias ? part : nullptr);
  if (dbias) launch_column_join(2 * n, (int)chunks, part, dbias, s);
  return hipGetLastError() == hipSuccess ? OZK_OK : OZK_EHIP;
}

}  // namespace ozk
