// Small products in emulated fp64: the deconstruction of up to four operands in one launch (lines
// of at most 512 values) or two and the modular products of up to two in one.  At these sizes
// the kernels of the large path (deconstruct.hip, gemm_i8.hip) are a chain of latencies: a thread
// there converts 8 or 16 values for every modulus one after the other, walks 128 rows of a
// column, and a 256 x 256 tile per modulus leaves most of the chip empty.  Here a line's values are read once into the
// registers of many threads for its exponent, the moduli are spread over workgroups, and the
// tiles are 64 x 128 or 128 x 128.  The arithmetic per value is the same (residue_math.h).
// A product of 64^3, r = 14, takes 12 us so (three launches, one after the other's results),
// 18 with exponents and residues in launches of their own, 29 by the kernels of the large path.
#include <math.h>

#include "ozk_internal.h"
#include "residue_math.h"
#include "tile_walk.h"

namespace ozk {
namespace {

// ---------------------------------------------------------------- exponents
// Workgroup: 16 lines, 64 threads each, a line's values (at most 2048) in registers, 32 per
// thread, asked for eight at a time as far as the line goes (from a clamped place past its end:
// a load under its own guard waits its turn).  Thread t of an operand of columns takes column
// t % 16 and rows t / 16, + 64, ...; of an operand of rows a wave takes a row, values lane,
// lane + 64, ...
constexpr int kLineMax = 2048, kHeld = kLineMax / 64;

struct ExpsArgs {
  SmallOperand op[kSmallOperands];
  int count, norm;
};

__device__ __forceinline__ uint64_t max64(uint64_t a, uint64_t b) { return a > b ? a : b; }

__global__ __launch_bounds__(1024) void small_exps_kernel(ExpsArgs A) {
  __shared__ uint64_t tops[64][17];
  __shared__ double sums[64][17];
  int64_t block = blockIdx.x;
  int o = 0;
  while (o + 1 < A.count && block >= (A.op[o].lines + 15) / 16) {
    block -= (A.op[o].lines + 15) / 16;
    ++o;
  }
  const SmallOperand& P = A.op[o];
  // line of the workgroup and place in it
  const int j = P.axis ? threadIdx.x & 15 : threadIdx.x >> 6;
  const int slice = P.axis ? threadIdx.x >> 4 : threadIdx.x & 63;
  const int64_t line = block * 16 + j;
  const bool live = line < P.lines;
  const int64_t sl = P.axis ? 1 : P.ld, sk = P.axis ? P.ld : 1;
  const double* x = P.x + (live ? line : P.lines - 1) * sl;
  double a[kHeld];
  uint64_t m = 0;
#pragma unroll
  for (int u = 0; u < kHeld; ++u) a[u] = 0.0;
#pragma unroll
  for (int g = 0; g < kHeld; g += 8)
    if (64 * g < P.kdim) {   // uniform
#pragma unroll
      for (int u = g; u < g + 8; ++u) {
        const int64_t h = slice + 64 * u;
        a[u] = x[(h < P.kdim ? h : P.kdim - 1) * sk];
      }
    }
#pragma unroll
  for (int u = 0; u < kHeld; ++u) {
    if (slice + 64 * u >= P.kdim) a[u] = 0.0;
    m = max64(m, abs_bits(a[u]));
  }
  tops[slice][j] = m;
  __syncthreads();
  // 64 slices to one: 16 threads a line (threads past 256 have nothing to do)
  const int jj = threadIdx.x & 15, part = threadIdx.x >> 4;
  if (part < 16) {
    m = max64(max64(tops[part][jj], tops[part + 16][jj]),
              max64(tops[part + 32][jj], tops[part + 48][jj]));
    tops[part][jj] = m;
  }
  __syncthreads();
  m = tops[0][j];
#pragma unroll
  for (int p = 1; p < 16; ++p) m = max64(m, tops[p][j]);
  if (!A.norm) {
    if (slice == 0 && live) P.exps[line] = line_exponent(m, P.width);
    return;
  }
  // the sum of (x 2^-T)^2, T of the line's largest magnitude, in a fixed order
  const int t = line_ilogb(m);
  double s = 0.0;
#pragma unroll
  for (int u = 0; u < kHeld; ++u) {
    const double y = __builtin_ldexp(a[u], -t);
    s = __builtin_fma(y, y, s);
  }
  sums[slice][j] = s;
  __syncthreads();
  if (part < 16)
    sums[part][jj] = (sums[part][jj] + sums[part + 16][jj]) +
                     (sums[part + 32][jj] + sums[part + 48][jj]);
  __syncthreads();
  if (slice == 0 && live) {
    s = sums[0][j];
    for (int p = 1; p < 16; ++p) s += sums[p][j];
    P.exps[line] = norm_exponent(m, s, P.width);
  }
}

// ---------------------------------------------------------------- residues
// Workgroup: 16 lines x 128 K values x one group of moduli, 8 consecutive K values a thread.
struct ResidueArgs {
  SmallOperand op[kSmallOperands];
  ResidueConsts K;
  int count, groups, norm;
  int64_t kp[kSmallOperands];
};

template <bool kWide>
__device__ __forceinline__ void put_residues(const double (&a)[8], int e, const ResidueConsts& K,
                                             int l0, int l1, int8_t* dst, int64_t plane_stride) {
  Prepared p[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) p[u] = prepare_element<kWide>(a[u], e);
  for (int l = l0; l < l1; ++l) {
    uint32_t b[8];
    if (l == 0) {
#pragma unroll
      for (int u = 0; u < 8; ++u) b[u] = residue_byte_256(p[u]);
    } else {
      const double m = K.m[l], inv = K.inv[l], c = K.c32[l];
#pragma unroll
      for (int u = 0; u < 8; ++u) b[u] = residue_byte<kWide>(p[u], m, inv, c);
    }
    *reinterpret_cast<uint2*>(dst + l * plane_stride) =
        make_uint2(pack4(b[0], b[1], b[2], b[3]), pack4(b[4], b[5], b[6], b[7]));
  }
}

__global__ __launch_bounds__(256) void small_residues_kernel(ResidueArgs A) {
  int64_t block = blockIdx.x / A.groups;
  const int group = blockIdx.x % A.groups;
  int o = 0;
  for (; o + 1 < A.count; ++o) {
    const int64_t blocks = (A.op[o].lines + 15) / 16 * (A.kp[o] / 128);
    if (block < blocks) break;
    block -= blocks;
  }
  const SmallOperand& P = A.op[o];
  const int64_t steps = A.kp[o] / 128;
  // neighbouring lanes: neighbouring columns (axis 1), or K values of one row
  const int j = P.axis ? threadIdx.x & 15 : threadIdx.x >> 4;
  const int kg = P.axis ? threadIdx.x >> 4 : threadIdx.x & 15;
  const int64_t line = block / steps * 16 + j, h0 = block % steps * 128 + 8 * kg;
  if (line >= P.lines) return;
  const int e = P.exps[line];
  const int64_t sk = P.axis ? P.ld : 1;
  const double* x = P.x + line * (P.axis ? 1 : P.ld);
  double a[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) a[u] = x[(h0 + u < P.kdim ? h0 + u : P.kdim - 1) * sk];
#pragma unroll
  for (int u = 0; u < 8; ++u)
    if (h0 + u >= P.kdim || e == INT32_MIN) a[u] = 0.0;
  const int l0 = A.K.r * group / A.groups, l1 = A.K.r * (group + 1) / A.groups;
  int8_t* dst = P.planes + line * A.kp[o] + h0;
  const int64_t stride = P.lines * A.kp[o];
  if (P.wide) put_residues<true>(a, e == INT32_MIN ? 0 : e, A.K, l0, l1, dst, stride);
  else put_residues<false>(a, e == INT32_MIN ? 0 : e, A.K, l0, l1, dst, stride);
}

// Lines of at most 128 kSteps values: exponents and residues in one launch.  Workgroup: 16 lines
// x one group of moduli, the lines' values in the registers that convert them (8 consecutive K
// values a thread and step of 128).
template <int kSteps>
__global__ __launch_bounds__(256) void small_lines_kernel(ResidueArgs A) {
  __shared__ uint64_t tops[16][17];
  __shared__ double sums[16][17];
  int64_t block = blockIdx.x / A.groups;
  const int group = blockIdx.x % A.groups;
  int o = 0;
  for (; o + 1 < A.count; ++o) {
    const int64_t blocks = (A.op[o].lines + 15) / 16;
    if (block < blocks) break;
    block -= blocks;
  }
  const SmallOperand& P = A.op[o];
  const int j = P.axis ? threadIdx.x & 15 : threadIdx.x >> 4;
  const int kg = P.axis ? threadIdx.x >> 4 : threadIdx.x & 15;
  const int64_t line = block * 16 + j, at = line < P.lines ? line : P.lines - 1;
  const int64_t sk = P.axis ? P.ld : 1;
  const double* x = P.x + at * (P.axis ? 1 : P.ld);
  double a[kSteps][8];
#pragma unroll
  for (int v = 0; v < kSteps; ++v) {
#pragma unroll
    for (int u = 0; u < 8; ++u) a[v][u] = 0.0;
    if (128 * v < P.kdim) {   // uniform
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int64_t h = 128 * v + 8 * kg + u;
        a[v][u] = x[(h < P.kdim ? h : P.kdim - 1) * sk];
      }
    }
  }
  uint64_t m = 0;
#pragma unroll
  for (int v = 0; v < kSteps; ++v)
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      if (128 * v + 8 * kg + u >= P.kdim) a[v][u] = 0.0;
      m = max64(m, abs_bits(a[v][u]));
    }
  tops[kg][j] = m;
  __syncthreads();
#pragma unroll
  for (int p = 0; p < 16; ++p) m = max64(m, tops[p][j]);
  int e;
  if (A.norm) {   // as small_exps_kernel: the sum of (x 2^-T)^2 in a fixed order
    const int t = line_ilogb(m);
    double s = 0.0;
#pragma unroll
    for (int v = 0; v < kSteps; ++v)
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const double y = __builtin_ldexp(a[v][u], -t);
        s = __builtin_fma(y, y, s);
      }
    sums[kg][j] = s;
    __syncthreads();
    s = sums[0][j];
#pragma unroll
    for (int p = 1; p < 16; ++p) s += sums[p][j];
    e = norm_exponent(m, s, P.width);
  } else {
    e = line_exponent(m, P.width);
  }
  if (line >= P.lines) return;
  if (group == 0 && kg == 0) P.exps[line] = e;
  const int l0 = A.K.r * group / A.groups, l1 = A.K.r * (group + 1) / A.groups;
  const int64_t stride = P.lines * A.kp[o];
  const bool nothing = e == INT32_MIN;
#pragma unroll
  for (int v = 0; v < kSteps; ++v) {
    if (128 * v >= A.kp[o]) break;
    if (nothing)
#pragma unroll
      for (int u = 0; u < 8; ++u) a[v][u] = 0.0;
    int8_t* dst = P.planes + line * A.kp[o] + 128 * v + 8 * kg;
    if (P.wide) put_residues<true>(a[v], nothing ? 0 : e, A.K, l0, l1, dst, stride);
    else put_residues<false>(a[v], nothing ? 0 : e, A.K, l0, l1, dst, stride);
  }
}

// ---------------------------------------------------------------- modular products
struct ProductArgs {
  PlaneProduct P[2];
  int count, r;
  int tiles_m[2], tiles_n[2], blocks0;   // workgroups of the first product
  int32_t mod[kMaxModuli];
  double inv[kMaxModuli];
};

// Low byte of the symmetric residue of an exact sum v modulo an odd m: v - m round(v / m), the
// rounding read from the low word of v RN(1/m) + 1.5 2^52 (within 2^-30 of v / m, which is at
// least 1 / (2 m) from a tie).
__device__ __forceinline__ uint32_t sum_residue(int v, int m, double inv) {
  const double t = __builtin_fma((double)v, inv, kMagic);
  return (uint32_t)(v - m * (int)(uint32_t)__double_as_longlong(t));
}

template <typename TL>
__global__ __launch_bounds__(64 * TL::NW) void small_products_kernel(ProductArgs A) {
  constexpr int H = TL::TI / 2, TJ = TL::TJ;
  __shared__ __attribute__((aligned(1024))) int8_t lds[TL::S * TL::kStage];
  int id = xcd_order();
  const int o = id >= A.blocks0;
  if (o) id -= A.blocks0;
  const PlaneProduct P = A.P[o];
  const int tiles = A.tiles_m[o] * A.tiles_n[o], l = id / tiles;
  const Walk<TL> W(lds, P.m, P.n, P.kp, P.left + l * P.m * P.kp, P.kp,
                   P.right + l * P.n * P.kp, P.kp, id - l * tiles, A.tiles_m[o], A.tiles_n[o], 8,
                   0, (int)(P.kp / kStepK));
  v4i own[H][TJ];
  small_product<TL>(W, own);
  const int kh = W.wave / (TL::WR * TL::WC), wt = W.wave % (TL::WR * TL::WC);
  const int64_t row0 = W.row0 + wt / TL::WC * TL::WM + kh * 16 * H + (W.lane & 15);
  const int64_t col0 = W.col0 + wt % TL::WC * TL::WN + 4 * (W.lane >> 4);
  int8_t* res = P.res + l * P.m * P.np;
  const int mod = A.mod[l];
  const double inv = A.inv[l];
#pragma unroll
  for (int i = 0; i < H; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      const int64_t row = row0 + 16 * i, col = col0 + 16 * j;
      if (row >= P.m || col >= P.np) continue;   // np is a multiple of 64
      const v4i v = own[i][j];
      uint32_t b[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) b[u] = mod == 256 ? (uint32_t)v[u] : sum_residue(v[u], mod, inv);
      *reinterpret_cast<uint32_t*>(res + row * P.np + col) = pack4(b[0], b[1], b[2], b[3]);
    }
}

template <typename TL>
void launch_small_t(ProductArgs& A, hipStream_t s) {
  int64_t blocks = 0;
  for (int o = 0; o < A.count; ++o) {
    A.tiles_m[o] = (int)((A.P[o].m + TL::BM - 1) / TL::BM);
    A.tiles_n[o] = (int)((A.P[o].n + TL::BN - 1) / TL::BN);
    if (o == 1) A.blocks0 = (int)blocks;
    blocks += (int64_t)A.tiles_m[o] * A.tiles_n[o] * A.r;
  }
  if (A.count < 2) A.blocks0 = (int)blocks;
  hipLaunchKernelGGL((small_products_kernel<TL>), dim3((unsigned)blocks), dim3(64 * TL::NW), 0, s,
                     A);
}

// Rounds of 256 workgroups for tiles of bm x bn, and their time in microseconds.  (A launch of a
// workgroup of 512 threads a tile ends before 2^23 of them: a few rows against 2^26 columns, 16
// moduli.  gemm_i8.hip's tiles are 256 x 256 and, past one K step, walked by one workgroup a
// compute unit.)
double rounds_time(const PlaneProduct* P, int count, int r, int64_t bm, int64_t bn, double fixed,
                   double step) {
  int64_t tiles = 0, steps = 0;
  for (int o = 0; o < count; ++o) {
    tiles += (P[o].m + bm - 1) / bm * ((P[o].n + bn - 1) / bn) * r;
    steps = P[o].kp / kStepK > steps ? P[o].kp / kStepK : steps;
  }
  if (bm < 256 && tiles >= 1 << 23) return HUGE_VAL;
  return (double)((tiles + 255) / 256) * (fixed + step * (double)steps);
}

}  // namespace

// Lines of at most 2048 values, and 2^21 values in the larger operand; 2^25 where its lines have at
// most 256 values, 2^23 where both operands' lines are columns.  Whole calls with one operand of
// so many values and 64 lines of the other, r = 16, norm rule, by these kernels and by the large
// path's, microseconds:
//   values               2^20         2^21         2^22         2^23
//   rows of 2048      36.1 / 37.1  38.6 / 35.7  49.7 / 43.9  90.2 / 74.3
//   rows of 1000      32.9 / 34.9  44.8 / 43.1  68.1 / 59.9   109 / 93.9
//   columns of 1000   32.4 / 39.2  47.3 / 48.7  74.2 / 67.0   123 / 107    (rows beside them)
//   rows of 200       39.4 / 48.9  62.8 / 78.9   103 / 134    184 / 241     (2^25: 661 / 999)
//   columns of 200    38.9 / 46.9  59.0 / 64.2  95.2 / 98.1   191 / 182     (2^25: 746 / 697)
//   both columns, 2048 36.5 / 62.1 41.9 / 65.2  54.2 / 72.8  98.1 / 114
//   both columns, 1000 32.7 / 62.4 48.3 / 71.5  75.6 / 89.1   124 / 132
// (rows of the large path take one launch that keeps a row in a workgroup's registers, whatever
// its length; two operands of columns take three launches each there.)  Over 600 such cases of
// lines of 200 to 2048 values, either rule and 2^19 to 2^23.5 values, the choice costs 0.8 % on
// average, 18 % at worst.
bool small_operands(int64_t lines, int64_t kdim, bool columns) {
  const int64_t most = (int64_t)1 << (kdim <= 256 ? 25 : (columns ? 23 : 21));
  return kdim <= kLineMax && lines * kdim <= most;
}

int launch_small_deconstruct(const SmallOperand* op, int count, int r, int scaling,
                             const int64_t* kp, hipStream_t s) {
  ExpsArgs E;
  ResidueArgs R;
  E.count = R.count = count;
  E.norm = R.norm = scaling == OZK_SCALING_NORM;
  int64_t lines = 0, blocks = 0, longest = 0;
  for (int o = 0; o < count; ++o) {
    E.op[o] = R.op[o] = op[o];
    R.kp[o] = kp[o];
    const ResidueConsts* K = residue_consts(r, op[o].width);
    if (!K) return OZK_EINVAL;
    R.K = *K;
    R.op[o].wide = K->wide;
    lines += (op[o].lines + 15) / 16;
    longest = kp[o] > longest ? kp[o] : longest;
    blocks += (op[o].lines + 15) / 16 * (kp[o] / 128);
  }
  // (with eight steps a thread, 214 registers, 1024^3 took 76 us, by two launches 59)
  if (longest <= 512) {
    // moduli in up to eight groups, until there are four workgroups a compute unit
    R.groups = lines >= 1024 ? 1 : (lines >= 512 ? 2 : (lines >= 256 ? 4 : 8));
    if (R.groups > r) R.groups = 1;
    const dim3 grid((unsigned)(lines * R.groups));
    if (longest <= 128) hipLaunchKernelGGL(small_lines_kernel<1>, grid, dim3(256), 0, s, R);
    else if (longest <= 256) hipLaunchKernelGGL(small_lines_kernel<2>, grid, dim3(256), 0, s, R);
    else hipLaunchKernelGGL(small_lines_kernel<4>, grid, dim3(256), 0, s, R);
    return hipGetLastError() == hipSuccess ? OZK_OK : OZK_EHIP;
  }
  // moduli in up to four groups, until there are eight workgroups a compute unit
  R.groups = blocks >= 2048 ? 1 : (blocks >= 1024 ? 2 : 4);
  if (R.groups > r) R.groups = 1;
  hipLaunchKernelGGL(small_exps_kernel, dim3((unsigned)lines), dim3(1024), 0, s, E);
  hipLaunchKernelGGL(small_residues_kernel, dim3((unsigned)(blocks * R.groups)), dim3(256), 0, s,
                     R);
  return hipGetLastError() == hipSuccess ? OZK_OK : OZK_EHIP;
}

int launch_products(const PlaneProduct* P, int count, int r, hipStream_t s) {
  ProductArgs A;
  A.count = count;
  A.r = r;
  const CrtConsts* C = crt_consts(r);
  for (int l = 0; l < kMaxModuli; ++l) {
    A.mod[l] = l < r ? C->mod[l] : 1;
    A.inv[l] = l < r ? C->inv[l] : 1.0;
  }
  for (int o = 0; o < count; ++o) A.P[o] = P[o];
  // One round: fixed + step per 128 K values (the int8 layer's measured rounds, without the launch).
  // Whole calls, r = 16, by the small, mid and large tiles: 256^3 13.6, 15.0, 16.4; 512^3 28.7,
  // 25.5, 28.5; 768^3 55.8, 49.4, 39.8; 60 x 60 x 8192 60.6, 66.2, 106; 384 x 384 x 8192 107, 82.3,
  // 124; 1024^3 86.2, 67.7, 51.0.  Over 26 shapes of 64 to 16384 the choice costs 0.8 % on average,
  // 12 % at worst (300 x 1000 x 300: mid 30.2, large 26.9).
  const double small = rounds_time(P, count, r, 64, 128, 2.5, 0.55);
  const double mid = rounds_time(P, count, r, 128, 128, 3.8, 0.72);
  double large = 0;   // gemm_i8.hip, one launch a product
  for (int o = 0; o < count; ++o)
    large += 2.5 + rounds_time(P + o, 1, r, 256, 256, 5.0, 1.5);
  if (large < small && large < mid) {
    for (int o = 0; o < count; ++o) {
      const int st = launch_gemm_i8(P[o].m, P[o].np, P[o].kp, r, P[o].left, P[o].m * P[o].kp,
                                    P[o].right, P[o].n * P[o].kp, P[o].res, P[o].np,
                                    P[o].m * P[o].np, kEpiResidues, s);
      if (st != OZK_OK) return st;
    }
    return OZK_OK;
  }
  if (small < mid) launch_small_t<TileSmall>(A, s);
  else launch_small_t<TileMid>(A, s);
  return hipGetLastError() == hipSuccess ? OZK_OK : OZK_EHIP;
}

}  // namespace ozk
