// int8 linear layer: C = act(s t^T * (X W^T) + 1 b^T) + R, X m x k and W n x k int8 with K
// contiguous in both, s and t fp32 scales of their rows.  The int8 product is exact in
// int32 (k <= OZK_MAX_K); everything after it is fp32, rounded once to the output's type.
#include <type_traits>

#include "activation.h"
#include "lds_dma.h"
#include "ozk_internal.h"
#include "rows.h"

namespace ozk {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef v4i v4i_bytes __attribute__((aligned(1)));
typedef v4i v4i_words __attribute__((aligned(4)));

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

// sum s t + b: the sum is rounded to fp32, scaled by s, and the rest is one fma.
__device__ __forceinline__ float pre_activation(int sum, float s, float t, float b) {
  return __builtin_fmaf((float)sum * s, t, b);
}

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
      float z = pre_activation(acc[u], s, t[u], E.bias ? (float)b[u] : 0.0f);
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
    float z = pre_activation(acc[u], s, E.sw[j], E.bias ? (float)E.bias[j] : 0.0f);
    z = activate(z, E.act);
    if (E.residual) z += (float)E.residual[row * E.ldr + j];
    E.c[row * E.ldc + j] = (O)z;
  }
}

// Eight consecutive outputs of one row: one 16-byte access where a type has two bytes.
template <typename O>
__device__ __forceinline__ void put8(const Epilogue<O>& E, int64_t row, int64_t col,
                                     const v4i& lo, const v4i& hi) {
  typedef O V __attribute__((ext_vector_type(8), aligned(sizeof(O))));
  typedef float F __attribute__((ext_vector_type(8), aligned(4)));
  if (row >= E.m || col >= E.n) return;
  if (col + 8 > E.n) {
    put4(E, row, col, lo);
    put4(E, row, col + 4, hi);
    return;
  }
  const float s = E.sx[row];
  const F t = *reinterpret_cast<const F*>(E.sw + col);
  V b, r, o;
  if (E.bias) b = *reinterpret_cast<const V*>(E.bias + col);
  if (E.residual) r = *reinterpret_cast<const V*>(E.residual + row * E.ldr + col);
  float z[8];
#pragma unroll
  for (int u = 0; u < 8; ++u)
    z[u] = pre_activation(u < 4 ? lo[u & 3] : hi[u & 3], s, t[u], E.bias ? (float)b[u] : 0.0f);
#pragma unroll
  for (int u = 0; u < 8; ++u) z[u] = activate(z[u], E.act);
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    if (E.residual) z[u] += (float)r[u];
    o[u] = (O)z[u];
  }
  *reinterpret_cast<V*>(E.c + row * E.ldc + col) = o;
}

// Bytes h .. h + 15 of a row of which `left` bytes are left from p on, zero past them, at any
// alignment.  The last bytes come from the 16 that end the row, shifted down; a row shorter
// than that (`shorter`) is read byte by byte.
__device__ __forceinline__ v4i load16(const int8_t* __restrict__ p, int64_t h, int64_t left,
                                      bool shorter) {
  if (h + 16 <= left) return *reinterpret_cast<const v4i_bytes*>(p + h);
  uint64_t lo = 0, hi = 0;
  if (h < left) {
    if (!shorter) {
      const v4i v = *reinterpret_cast<const v4i_bytes*>(p + left - 16);
      lo = (uint64_t)(uint32_t)v[0] | (uint64_t)(uint32_t)v[1] << 32;
      hi = (uint64_t)(uint32_t)v[2] | (uint64_t)(uint32_t)v[3] << 32;
      const int bits = 8 * (int)(h + 16 - left);   // 8 .. 120
      if (bits >= 64) {
        lo = hi >> (bits - 64);
        hi = 0;
      } else {
        lo = lo >> bits | hi << (64 - bits);
        hi >>= bits;
      }
    } else {
#pragma unroll 1
      for (int u = (int)(left - h) - 1; u >= 0; --u) {
        hi = hi << 8 | lo >> 56;
        lo = lo << 8 | (uint8_t)p[h + u];
      }
    }
  }
  return v4i{(int)(uint32_t)lo, (int)(uint32_t)(lo >> 32), (int)(uint32_t)hi,
             (int)(uint32_t)(hi >> 32)};
}

// Four int32 partial sums of an m x n product.
__device__ __forceinline__ void put_part(int32_t* __restrict__ p, int64_t row, int64_t col,
                                         int64_t m, int64_t n, const v4i& acc) {
  if (row >= m || col >= n) return;
  if (col + 4 <= n) {
    *reinterpret_cast<v4i_words*>(p + row * n + col) = acc;
    return;
  }
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (col + u < n) p[row * n + col + u] = acc[u];
}

// Few rows: workgroup = 16 kMT rows x 16 kNT columns of C, its kWaves waves taking the K
// steps of 128 bytes in turn (of the workgroup's split of K).  Operands go from global
// memory to the matrix core's registers directly: lane l of a fragment holds row l % 16 and
// 16 bytes of K.  Whole steps run kDeep at a time, all their loads issued first: what bounds
// the kernel is the stream of W, so bytes in flight count.
template <typename O, int kMT, int kNT, int kWaves, int kDeep>
__global__ __launch_bounds__(64 * kWaves) void int8linear_few_kernel(
    int64_t k, const int8_t* __restrict__ x, int64_t ldx, const int8_t* __restrict__ w,
    int64_t ldw, Epilogue<O> E, int splits, int32_t* __restrict__ part) {
  __shared__ v4i sums[kWaves][kMT * kNT][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t tiles_n = (E.n + 16 * kNT - 1) / (16 * kNT);
  const int split = blockIdx.x % splits;
  const int64_t id = blockIdx.x / splits;
  const int64_t col0 = id % tiles_n * (16 * kNT), row0 = id / tiles_n * (16 * kMT);
  const int8_t* wp[kNT];
#pragma unroll
  for (int j = 0; j < kNT; ++j) {
    const int64_t r = col0 + 16 * j + (lane & 15);
    wp[j] = w + (r < E.n ? r : E.n - 1) * ldw + 16 * (lane >> 4);
  }
  const int8_t* xp[kMT];
#pragma unroll
  for (int i = 0; i < kMT; ++i) {
    const int64_t r = row0 + 16 * i + (lane & 15);
    xp[i] = x + (r < E.m ? r : E.m - 1) * ldx + 16 * (lane >> 4);
  }
  v4i acc[kMT][kNT];
#pragma unroll
  for (int i = 0; i < kMT; ++i)
#pragma unroll
    for (int j = 0; j < kNT; ++j) acc[i][j] = v4i{0, 0, 0, 0};
  // this workgroup's steps [t0, t1), the last one of a row perhaps short
  const int64_t steps = (k + 127) / 128, whole = k / 128;
  const int64_t t0 = steps * split / splits, t1 = steps * (split + 1) / splits;
  const int64_t t1w = t1 < whole ? t1 : whole;
  int64_t t = t0 + wave;
  for (; t + (kDeep - 1) * kWaves < t1w; t += kDeep * kWaves) {
    v4i fb[kDeep][2][kNT], fa[kDeep][2][kMT];
#pragma unroll
    for (int d = 0; d < kDeep; ++d)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t at = (t + d * kWaves) * 128 + 64 * h;
#pragma unroll
        for (int j = 0; j < kNT; ++j)
          fb[d][h][j] = *reinterpret_cast<const v4i_bytes*>(wp[j] + at);
#pragma unroll
        for (int i = 0; i < kMT; ++i)
          fa[d][h][i] = *reinterpret_cast<const v4i_bytes*>(xp[i] + at);
      }
#pragma unroll
    for (int d = 0; d < kDeep; ++d)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < kMT; ++i)
#pragma unroll
          for (int j = 0; j < kNT; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[d][h][j], fa[d][h][i],
                                                              acc[i][j], 0, 0, 0);
  }
#pragma unroll 1
  for (; t < t1; t += kWaves) {   // what is left, a short last step among it
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t at = t * 128 + 64 * h, lo = 16 * (lane >> 4);
      v4i b[kNT];
#pragma unroll
      for (int j = 0; j < kNT; ++j) b[j] = load16(wp[j] - lo, at + lo, k, k < 16);
#pragma unroll
      for (int i = 0; i < kMT; ++i) {
        const v4i a = load16(xp[i] - lo, at + lo, k, k < 16);
#pragma unroll
        for (int j = 0; j < kNT; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[j], a, acc[i][j], 0, 0, 0);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kMT; ++i)
#pragma unroll
    for (int j = 0; j < kNT; ++j) sums[wave][i * kNT + j][lane] = acc[i][j];
  __syncthreads();
  for (int b = wave; b < kMT * kNT; b += kWaves) {
    v4i s = sums[0][b][lane];
#pragma unroll
    for (int v = 1; v < kWaves; ++v) s += sums[v][b][lane];
    const int64_t row = row0 + 16 * (b / kNT) + (lane & 15);
    const int64_t col = col0 + 16 * (b % kNT) + 4 * (lane >> 4);
    if (part)
      put_part(part + split * E.m * E.n, row, col, E.m, E.n, s);
    else
      put4(E, row, col, s);
  }
}

// ------------------------------------------------------------------ tiles
// Workgroup barrier that no LDS access is moved across.
__device__ __forceinline__ void wg_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

constexpr int kStepK = 128;   // K bytes of a step: whole cache lines of every row
constexpr int kXcds = 8;

// Shape of a workgroup tile: kBM x kBN outputs by kWR x kWC waves, each wave TI x TJ blocks
// of 16 x 16, operands in a ring of kS stages of one K step.
template <int kBM, int kBN, int kWR, int kWC, int kS>
struct Tile {
  static constexpr int BM = kBM, BN = kBN, WR = kWR, WC = kWC, S = kS;
  static constexpr int NW = WR * WC;
  static constexpr int WM = BM / WR, WN = BN / WC;
  static constexpr int TI = WM / 16, TJ = WN / 16;
  static constexpr int kStage = (BM + BN) * kStepK;   // bytes
  static constexpr int kLoads = kStage / 1024 / NW;   // 1 KiB (8 rows) per wave and load
  static constexpr int kPitch = WN + 4;               // staged outputs of a wave, in words
  static constexpr int kPhase = S * kStage / NW / (16 * kPitch * 4) >= TI
                                    ? TI
                                    : (S * kStage / NW / (16 * kPitch * 4) >= TI / 2 ? TI / 2
                                                                                     : TI / 4);
  static_assert(BM % (8 * NW) == 0 && BN % (8 * NW) == 0, "loads of A and B are whole");
  static_assert(TI % kPhase == 0 && kPhase * 16 * kPitch * 4 * NW <= S * kStage, "staging fits");
  static_assert(kLoads <= TI * TJ, "a load after each MFMA of a half at most");
};

// X W^T over the K steps [t0, t1) of a tile: operand tiles go through LDS (direct loads where
// rows are 16-byte aligned and k is a multiple of 16; else through registers, zero past k).
// An LDS row is 128 bytes, its eight 16-byte chunks XORed with (row >> 1) & 7 so that the 16
// lanes of a fragment read (rows r .. r + 15, one logical chunk) cover all 64 banks.
// Per step every wave runs two halves of TI x TJ MFMAs (16 x 16 x 64); the fragments of the
// next half are read between the MFMAs of the current one.  Between the halves the wave waits
// for its loads of step t + 1 and its reads, and the barrier makes step t + 1 complete and
// step t fully read; the second half issues the loads of step t + kS into step t's stage.
template <typename O, typename TL, bool kDirect>
__global__ __launch_bounds__(64 * TL::NW) void int8linear_tile_kernel(
    int64_t k, const int8_t* __restrict__ x, int64_t ldx, const int8_t* __restrict__ w,
    int64_t ldw, Epilogue<O> E, int tiles_m, int tiles_n, int splits, int group_m,
    int32_t* __restrict__ part) {
  constexpr int BM = TL::BM, BN = TL::BN, TI = TL::TI, TJ = TL::TJ, NW = TL::NW, S = TL::S;
  constexpr int L = TL::kLoads;
  __shared__ __attribute__((aligned(1024))) int8_t lds[S * TL::kStage];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave / TL::WC, wc = wave % TL::WC;

  // Block -> (split, tile row, tile column).  The hardware deals blocks out round-robin over
  // the 8 XCDs; XCD x takes one contiguous run of the order (split, groups of group_m tile
  // rows, column, row in group), so the tiles in flight on it share panels in its L2.
  const int total = gridDim.x, per = total / kXcds, extra = total % kXcds;
  const int xcd = blockIdx.x % kXcds;
  const int id = xcd * per + (xcd < extra ? xcd : extra) + blockIdx.x / kXcds;
  const int tiles = tiles_m * tiles_n;
  const int split = id / tiles, rem = id - split * tiles;
  const int per_group = group_m * tiles_n;
  const int first = rem / per_group * group_m;
  const int gsize = tiles_m - first < group_m ? tiles_m - first : group_m;
  const int in_group = rem % per_group;
  const int64_t row0 = (int64_t)(first + in_group % gsize) * BM;
  const int64_t col0 = (int64_t)(in_group / gsize) * BN;
  const int steps = (int)((k + kStepK - 1) / kStepK);
  const int t0 = (int)((int64_t)steps * split / splits);
  const int t1 = (int)((int64_t)steps * (split + 1) / splits);
  const int nk = t1 - t0;

  // Load q of this wave: region rg = wave + NW q, rows 8 rg .. 8 rg + 7 of X (then of W);
  // lane i takes row i / 8 of it, physical chunk i % 8; rows past the matrix re-read its last.
  const int8_t* base_x = x + row0 * ldx + (int64_t)t0 * kStepK;
  const int8_t* base_w = w + col0 * ldw + (int64_t)t0 * kStepK;
  typedef typename std::conditional<kDirect, uint32_t, int64_t>::type Offset;
  Offset voff[L];   // row offset from the tile's first row
  // logical K offset of the lane's chunk: the swizzle depends on the region's parity alone,
  // which is the wave's (NW is even)
  static_assert(NW % 2 == 0, "one chunk for all loads of a lane");
  const uint32_t chunk16 = 16 * ((lane & 7) ^ ((4 * wave + (lane >> 4)) & 7));
#pragma unroll
  for (int q = 0; q < L; ++q) {
    const int rg = wave + NW * q;
    const bool is_w = rg >= BM / 8;
    const int row = 8 * (is_w ? rg - BM / 8 : rg) + (lane >> 3);
    const int64_t origin = is_w ? col0 : row0, last = (is_w ? E.n : E.m) - 1;
    const int64_t gr = origin + row < last ? origin + row : last;
    voff[q] = (Offset)((gr - origin) * (is_w ? ldw : ldx));
  }
  const uint32_t wave_lds = __builtin_amdgcn_readfirstlane(lds_address(lds) + wave * 1024);
  v4i staged[kDirect ? 1 : L];
  // K bytes left from the first byte of step t (of this split) on
  auto left = [&](int t) { return k - (int64_t)(t0 + t) * kStepK; };
  auto load = [&](int t, int q) {
    const bool is_w = wave + NW * q >= BM / 8;
    const int8_t* base = (is_w ? base_w : base_x) + (int64_t)t * kStepK;
    if constexpr (kDirect) {
      // a chunk past k re-reads the row's last one; the fragments of X are zeroed there
      const int64_t rest = left(t) - 16;
      const uint32_t c = chunk16 < rest ? chunk16 : (uint32_t)rest;
      dma16_sbase(voff[q] + c, (uint64_t)base,
                  wave_lds + (uint32_t)(t % S) * TL::kStage + q * (NW * 1024));
    } else {
      staged[q] = load16(base + voff[q], chunk16, left(t), k < 16);
    }
  };
  auto put_staged = [&](int t) {
    if constexpr (!kDirect) {
#pragma unroll
      for (int q = 0; q < L; ++q)
        *reinterpret_cast<v4i*>(lds + (t % S) * TL::kStage + (wave + NW * q) * 1024 +
                                lane * 16) = staged[q];
    }
  };

  v4i acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = v4i{0, 0, 0, 0};

  const int frow = lane & 15, fchunk = lane >> 4, sw = frow >> 1;
  const int off0 = ((0 + fchunk) ^ sw) << 4, off1 = ((4 + fchunk) ^ sw) << 4;
  const int arow = (wr * TL::WM + frow) * kStepK, brow = (BM + wc * TL::WN + frow) * kStepK;
  v4i fa[2][TI], fb[2][TJ];
  auto read = [&](int h, int t, int idx) {   // fragment idx of half h of step t
    const int8_t* st = lds + (t % S) * TL::kStage + (h ? off1 : off0);
    if (idx < TI) {
      v4i v = *reinterpret_cast<const v4i*>(st + arow + idx * 16 * kStepK);
      if (kDirect && left(t) < kStepK)   // uniform
        v = 64 * h + 16 * fchunk < left(t) ? v : v4i{0, 0, 0, 0};
      fa[h][idx] = v;
    } else {
      fb[h][idx - TI] = *reinterpret_cast<const v4i*>(st + brow + (idx - TI) * 16 * kStepK);
    }
  };
  auto wait_loads = [&](int younger) {   // this wave's loads but the youngest `younger` steps
    if constexpr (kDirect) {
      if (S > 2 && younger >= S - 2)
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(L * (S - 2)) : "memory");
      else
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
  };

  if constexpr (kDirect) {
#pragma unroll
    for (int t = 0; t < S; ++t)
      if (t < nk)
#pragma unroll
        for (int q = 0; q < L; ++q) load(t, q);
    // step 0 has landed when at most the other S - 1 steps' loads are under way
    if (nk >= S)
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(L * (S - 1)) : "memory");
    else
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  } else {
    // steps 0 and 1 go in, step 2 waits in registers
#pragma unroll
    for (int t = 0; t < 2; ++t)
      if (t < nk) {
#pragma unroll
        for (int q = 0; q < L; ++q) load(t, q);
        put_staged(t);
      }
    static_assert(kDirect || S == 2, "register staging runs two stages");
  }
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  wg_barrier();
#pragma unroll
  for (int idx = 0; idx < TI + TJ; ++idx) read(0, 0, idx);
  for (int t = 0; t < nk; ++t) {
    __builtin_amdgcn_sched_barrier(0);
    // step t + 1 waits in registers since the last step (steps 0 and 1 are in place)
    if (!kDirect && t > 0 && t + 1 < nk) put_staged(t + 1);
#pragma unroll
    for (int idx = 0; idx < TI * TJ; ++idx) {
      const int i = idx / TJ, j = idx % TJ;
      acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[0][j], fa[0][i], acc[i][j], 0, 0, 0);
      if (idx < TI + TJ) read(1, t, idx);
      __builtin_amdgcn_sched_barrier(0);
    }
    wait_loads(nk - 2 - t);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    wg_barrier();
    __builtin_amdgcn_sched_barrier(0);
    const bool more = t + 1 < nk;
    const int tl = t + (kDirect ? S : 2);
#pragma unroll
    for (int idx = 0; idx < TI * TJ; ++idx) {
      const int i = idx / TJ, j = idx % TJ;
      acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[1][j], fa[1][i], acc[i][j], 0, 0, 0);
      if (idx < TI + TJ && more) read(0, t + 1, idx);
      if (idx < L && tl < nk) load(tl, idx);
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // lane l of block (i, j): row 16 i + l % 16, columns 16 j + 4 (l / 16) .. + 3
  const int64_t wrow0 = row0 + wr * TL::WM, wcol0 = col0 + wc * TL::WN;
  if (part) {
    int32_t* p = part + (int64_t)split * E.m * E.n;
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int j = 0; j < TJ; ++j)
        put_part(p, wrow0 + 16 * i + frow, wcol0 + 16 * j + 4 * fchunk, E.m, E.n, acc[i][j]);
    return;
  }
  // Staged through this wave's part of the ring so that eight lanes finish one row of 64
  // columns, eight consecutive outputs each, and the code of the epilogue stands once.
  wg_barrier();   // every wave is past its last read
  int32_t* mine = reinterpret_cast<int32_t*>(lds) + wave * (TL::kPhase * 16 * TL::kPitch);
#pragma unroll
  for (int ph = 0; ph < TI / TL::kPhase; ++ph) {
#pragma unroll
    for (int i = 0; i < TL::kPhase; ++i)
#pragma unroll
      for (int j = 0; j < TJ; ++j)
        *reinterpret_cast<v4i*>(mine + (16 * i + frow) * TL::kPitch + 16 * j + 4 * fchunk) =
            acc[ph * TL::kPhase + i][j];
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    constexpr int kLanes = TL::WN / 8;   // lanes of a row
#pragma unroll 1
    for (int r = lane / kLanes; r < TL::kPhase * 16; r += 64 / kLanes) {
      const int c = 8 * (lane % kLanes);
      const v4i lo = *reinterpret_cast<const v4i*>(mine + r * TL::kPitch + c);
      const v4i hi = *reinterpret_cast<const v4i*>(mine + r * TL::kPitch + c + 4);
      put8(E, wrow0 + ph * TL::kPhase * 16 + r, wcol0 + c, lo, hi);
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
}

// The outputs of a product whose K was split: the partial sums added, then the epilogue.
template <typename O>
__global__ __launch_bounds__(256) void int8linear_join_kernel(Epilogue<O> E, int splits,
                                                              const int32_t* __restrict__ part) {
  const int64_t quads = (E.n + 3) / 4;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= E.m * quads) return;
  const int64_t row = id / quads, col = id % quads * 4;
  v4i s{0, 0, 0, 0};
  const int32_t* p = part + row * E.n + col;
  for (int k = 0; k < splits; ++k, p += E.m * E.n) {
    if (col + 4 <= E.n) {
      s += *reinterpret_cast<const v4i_words*>(p);
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (col + u < E.n) s[u] += p[u];
    }
  }
  put4(E, row, col, s);
}

typedef Tile<256, 256, 2, 4, 2> TileLarge;
typedef Tile<128, 128, 2, 2, 2> TileMid;

// How a product is run.  few: the kernel for few rows, mt x nt blocks of 16 x 16 a workgroup;
// else tiles of one shape.  K is split over `splits` workgroups where there are fewer tiles
// than the compute units take.
struct Plan {
  bool few, large;
  int mt, nt;
  int64_t tiles_m, tiles_n;
  int splits;
};

Plan plan_of(int64_t m, int64_t n, int64_t k) {
  Plan p{};
  const int64_t steps = (k + kStepK - 1) / kStepK;
  p.few = m <= 64;
  if (p.few) {
    p.mt = m <= 16 ? 1 : (m <= 32 ? 2 : 4);
    p.nt = m <= 16 ? 1 : 2;
    p.tiles_m = 1;
    p.tiles_n = (n + 16 * p.nt - 1) / (16 * p.nt);
    // a workgroup's eight waves take two batches of steps at least
    const int64_t s = 256 / p.tiles_n, most = steps / 64;
    p.splits = (int)(s < most ? s : most);
    if (p.splits < 1) p.splits = 1;
    return p;
  }
  p.large = (m + 255) / 256 * ((n + 255) / 256) >= 192;
  const int64_t b = p.large ? 256 : 128;
  p.tiles_m = (m + b - 1) / b;
  p.tiles_n = (n + b - 1) / b;
  p.splits = 1;
  const int64_t tiles = p.tiles_m * p.tiles_n;
  if (!p.large) {
    int64_t s = 512 / tiles;
    const int64_t most = steps / 8;
    s = s < most ? s : most;
    p.splits = s < 1 ? 1 : (s > 16 ? 16 : (int)s);
  }
  return p;
}

template <typename O, typename TL, bool kDirect>
void launch_tiles(const Plan& p, int64_t k, const int8_t* x, int64_t ldx, const int8_t* w,
                  int64_t ldw, const Epilogue<O>& E, int32_t* part, hipStream_t s) {
  const int group_m = 8;
  hipLaunchKernelGGL((int8linear_tile_kernel<O, TL, kDirect>),
                     dim3((unsigned)(p.tiles_m * p.tiles_n * p.splits)), dim3(64 * TL::NW), 0, s,
                     k, x, ldx, w, ldw, E, (int)p.tiles_m, (int)p.tiles_n, p.splits, group_m,
                     p.splits > 1 ? part : nullptr);
}

template <typename O>
int int8linear_t(int64_t m, int64_t n, int64_t k, const int8_t* x, int64_t ldx, const float* sx,
                 const int8_t* w, int64_t ldw, const float* sw, const void* bias, int act,
                 const void* residual, int64_t ldr, void* c, int64_t ldc, void* workspace,
                 hipStream_t s) {
  const Epilogue<O> E{m, n, sx, sw, (const O*)bias, (const O*)residual, ldr, (O*)c, ldc, act};
  const Plan p = plan_of(m, n, k);
  int32_t* part = static_cast<int32_t*>(workspace);
  if (p.tiles_m * p.tiles_n * p.splits > 0x7fffffff) return OZK_EUNSUPPORTED;
  // direct loads: 16-byte aligned rows and K; a lane's offset within a tile in 32 bits
  const bool direct = (((uintptr_t)x | (uintptr_t)w | (uint64_t)ldx | (uint64_t)ldw |
                        (uint64_t)k) & 15) == 0 && ldx < (1 << 24) && ldw < (1 << 24);
  if (p.few) {
#define OZK_FEW(MT, NT, DEEP)                                                                  \
  hipLaunchKernelGGL((int8linear_few_kernel<O, MT, NT, 8, DEEP>),                              \
                     dim3((unsigned)(p.tiles_n * p.splits)), dim3(512), 0, s, k, x, ldx, w, ldw, \
                     E, p.splits, p.splits > 1 ? part : nullptr)
    if (p.mt == 1) OZK_FEW(1, 1, 4);
    else if (p.mt == 2) OZK_FEW(2, 2, 2);
    else OZK_FEW(4, 2, 1);
#undef OZK_FEW
  } else if (!direct) {
    Plan q = p;
    if (p.large) {
      q.tiles_m = (m + 127) / 128;
      q.tiles_n = (n + 127) / 128;
    }
    launch_tiles<O, TileMid, false>(q, k, x, ldx, w, ldw, E, part, s);
  } else if (p.large) {
    launch_tiles<O, TileLarge, true>(p, k, x, ldx, w, ldw, E, part, s);
  } else {
    launch_tiles<O, TileMid, true>(p, k, x, ldx, w, ldw, E, part, s);
  }
  if (p.splits > 1)
    hipLaunchKernelGGL((int8linear_join_kernel<O>),
                       dim3((unsigned)((m * ((n + 3) / 4) + 255) / 256)), dim3(256), 0, s, E,
                       p.splits, part);
  return hipGetLastError() == hipSuccess ? OZK_OK : OZK_EHIP;
}

}  // namespace

size_t int8linear_workspace(int64_t m, int64_t n, int64_t k) {
  if (m <= 0 || n <= 0) return 0;
  const Plan p = plan_of(m, n, k);
  return p.splits > 1 ? (size_t)p.splits * m * n * 4 : 0;
}

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
