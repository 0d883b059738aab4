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

// One output.
template <typename O>
__device__ __forceinline__ void put1(const Epilogue<O>& E, int64_t row, int64_t col, int sum) {
  float z = pre_activation(sum, E.sx[row], E.sw[col], E.bias ? (float)E.bias[col] : 0.0f);
  z = activate(z, E.act);
  if (E.residual) z += (float)E.residual[row * E.ldr + col];
  E.c[row * E.ldc + col] = (O)z;
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
    float z[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      z[u] = pre_activation(acc[u], s, t[u], E.bias ? (float)b[u] : 0.0f);
    activate_all(z, E.act);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (E.residual) z[u] += (float)r[u];
      o[u] = (O)z[u];
    }
    *reinterpret_cast<V*>(E.c + row * E.ldc + col) = o;
    return;
  }
#pragma unroll 1
  for (int u = 0; u < 4; ++u) {
    const int64_t j = col + u;
    if (j >= E.n) break;
    put1(E, row, j, u == 0 ? acc[0] : (u == 1 ? acc[1] : acc[2]));
  }
}

// The outputs from col to the row's end, fewer than eight, from staged sums.
template <typename O>
__device__ __forceinline__ void put_ragged(const Epilogue<O>& E, int64_t row, int64_t col,
                                        const int32_t* sums) {
#pragma unroll 1
  for (int u = 0; col + u < E.n; ++u) put1(E, row, col + u, sums[u]);
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
// of 16 x 16, operands in a ring of two stages of one K step.
template <int kBM, int kBN, int kWR, int kWC>
struct Tile {
  static constexpr int BM = kBM, BN = kBN, WR = kWR, WC = kWC;
  static constexpr int S = 2;   // stages of the ring
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
};

// X W^T over the K steps [t0, t1) of a tile: operand tiles go through LDS (direct loads where
// rows are 16-byte aligned and k is a multiple of 16; else through registers, zero past k).
// An LDS row is 128 bytes, its eight 16-byte chunks XORed with (row >> 1) & 7 so that the 16
// lanes of a fragment read (rows r .. r + 15, one logical chunk) cover all 64 banks.
// Per step every wave runs quarters of 2 x TJ blocks; before the last one it waits for its
// loads of step t + 1 and for its reads of step t (the last quarter's operands are in
// registers by then), so one barrier a step makes step t + 1 complete and step t's stage free
// for step t + 2, whose loads have three quarters of a step to land.
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
      // a chunk past k re-reads the row's last one (clear_tail)
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
  v4i fa[2][2][2], fb[2][TJ];   // fa[set][K half][row block of a quarter], fb[K half][block]
  auto read_a = [&](int set, const int8_t* st, int kh, int rb, int ii) {
    fa[set][kh][ii] =
        *reinterpret_cast<const v4i*>(st + arow + (kh ? off1 : off0) + rb * 16 * kStepK);
  };
  auto read_b = [&](const int8_t* st, int kh, int j) {
    fb[kh][j] = *reinterpret_cast<const v4i*>(st + brow + (kh ? off1 : off0) + j * 16 * kStepK);
  };
  auto stage = [&](int t) { return lds + (t % S) * TL::kStage; };
  // The chunks of X past k in the row's last, short step (whole chunks: k is a multiple of
  // 16) are made zero in LDS, all waves together; what W holds there then does not count.
  auto clear_tail = [&](int t) {
    if (!kDirect || t >= nk || left(t) >= kStepK) return;
    const int first = (int)left(t) / 16;
    for (int i = threadIdx.x; i < BM * 8; i += 64 * NW) {
      const int row = i >> 3, c = i & 7;
      if (c >= first)
        *reinterpret_cast<v4i*>(stage(t) + row * kStepK + ((c ^ ((row >> 1) & 7)) << 4)) =
            v4i{0, 0, 0, 0};
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    wg_barrier();
  };
  // Quarter q (row blocks 2q and 2q + 1): MFMA idx is row block 2q + idx / (2 TJ), column block
  // (idx / 2) % TJ, K half idx % 2, a block's two halves back to back.  Its first four MFMAs
  // are followed by the reads of the next quarter's A fragments into the other set (the last
  // quarter's: row blocks 0 and 1 of stage `next`); the last quarter also replaces each B
  // fragment after its last use and issues the loads of step `tl`, if there is one.
  constexpr int NQ = TI / 2, kQuarter = 4 * TJ;
  static_assert(NQ % 2 == 0 && L <= kQuarter, "sets alternate; loads fit a quarter");
  auto quarter = [&](int q, const int8_t* st, const int8_t* next, int tl) {
    const int as = q & 1;
    const bool is_last = q == NQ - 1;
#pragma unroll
    for (int idx = 0; idx < kQuarter; ++idx) {
      const int ii = idx / (2 * TJ), j = (idx >> 1) % TJ, kh = idx & 1;
      acc[2 * q + ii][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[kh][j], fa[as][kh][ii],
                                                                 acc[2 * q + ii][j], 0, 0, 0);
      if (idx < 4) {
        if (!is_last) read_a(as ^ 1, st, idx & 1, 2 * (q + 1) + (idx >> 1), idx >> 1);
        else read_a(as ^ 1, next, idx & 1, idx >> 1, idx >> 1);
      }
      if (is_last && ii == 1) read_b(next, kh, j);
      if (is_last && (idx * L) / kQuarter != ((idx + 1) * L) / kQuarter && tl < nk)
        load(tl, (idx * L) / kQuarter);
      __builtin_amdgcn_sched_barrier(0);
      // the wave that reaches the second half of a quarter first is preferred, so the two
      // waves of a SIMD run apart
      if (idx == kQuarter / 2 - 1) __builtin_amdgcn_s_setprio(1);
    }
    __builtin_amdgcn_s_setprio(0);
  };

  if constexpr (kDirect) {
#pragma unroll
    for (int q = 0; q < L; ++q) load(0, q);
    if (nk > 1) {
#pragma unroll
      for (int q = 0; q < L; ++q) load(1, q);
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(L) : "memory");
    } else {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
  } else {
#pragma unroll
    for (int t = 0; t < 2; ++t)
      if (t < nk) {
#pragma unroll
        for (int q = 0; q < L; ++q) load(t, q);
        put_staged(t);
      }
  }
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  wg_barrier();
  clear_tail(0);
#pragma unroll
  for (int idx = 0; idx < 4; ++idx) read_a(0, lds, idx & 1, idx >> 1, idx >> 1);
#pragma unroll
  for (int j = 0; j < TJ; ++j) {
    read_b(lds, 0, j);
    read_b(lds, 1, j);
  }
  for (int t = 0; t < nk; ++t) {
    __builtin_amdgcn_sched_barrier(0);
    const int8_t* st = stage(t);
    // step t + 1 waits in registers since the last step (steps 0 and 1 are in place)
    if (!kDirect && t > 0 && t + 1 < nk) put_staged(t + 1);
#pragma unroll
    for (int q = 0; q < NQ - 1; ++q) quarter(q, st, st, nk);
    // this wave's loads of step t + 1 have landed and it has read all of step t; past the
    // barrier that holds for every wave
    if (kDirect) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    wg_barrier();
    clear_tail(t + 1);
    __builtin_amdgcn_sched_barrier(0);
    // after the last step: a harmless re-read of it
    quarter(NQ - 1, st, t + 1 < nk ? stage(t + 1) : st, t + 2);
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
  // columns, eight consecutive outputs each.  The rows' scales and residuals are asked for
  // four groups of rows ahead: an output's own work is short, the latency of its operands is
  // not.  The loop over the groups of a phase is kept a loop: written out, the epilogue does
  // not fit the instruction cache (4096 x 16384 x 4096 with gelu and residual: 1.2 ms).
  typedef O V8 __attribute__((ext_vector_type(8), aligned(sizeof(O))));
  typedef float F8 __attribute__((ext_vector_type(8), aligned(4)));
  constexpr int kLanes = TL::WN / 8, kRows = 64 / kLanes;        // lanes of a row, rows at once
  constexpr int kIters = TL::kPhase * 16 / kRows, kPhases = TI / TL::kPhase, kAhead = 4;
  const int lrow = lane / kLanes, lcol = 8 * (lane % kLanes);
  const int64_t col = wcol0 + lcol;
  const bool whole = col + 8 <= E.n;
  float t[8], b[8], s[kAhead];
  V8 res[kAhead];
  auto ahead = [&](int slot, int64_t row) {
    if (row >= E.m) return;
    s[slot] = E.sx[row];
    if (E.residual && whole)
      res[slot] = *reinterpret_cast<const V8*>(E.residual + row * E.ldr + col);
  };
#pragma unroll
  for (int u = 0; u < kAhead; ++u) ahead(u, wrow0 + u * kRows + lrow);
#pragma unroll
  for (int u = 0; u < 8; ++u) t[u] = b[u] = 0.0f;
  if (whole) {
    const F8 tv = *reinterpret_cast<const F8*>(E.sw + col);
#pragma unroll
    for (int u = 0; u < 8; ++u) t[u] = tv[u];
    if (E.bias) {
      const V8 bv = *reinterpret_cast<const V8*>(E.bias + col);
#pragma unroll
      for (int u = 0; u < 8; ++u) b[u] = (float)bv[u];
    }
  }
  wg_barrier();   // every wave is past its last read of the ring
  int32_t* mine = reinterpret_cast<int32_t*>(lds) + wave * (TL::kPhase * 16 * TL::kPitch);
#pragma unroll
  for (int ph = 0; ph < kPhases; ++ph) {
#pragma unroll
    for (int i = 0; i < TL::kPhase; ++i)
#pragma unroll
      for (int j = 0; j < TJ; ++j)
        *reinterpret_cast<v4i*>(mine + (16 * i + frow) * TL::kPitch + 16 * j + 4 * fchunk) =
            acc[ph * TL::kPhase + i][j];
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll 1
    for (int it = 0; it < kIters; ++it) {
      const int64_t row = wrow0 + (ph * kIters + it) * kRows + lrow;
      const int32_t* from = mine + (it * kRows + lrow) * TL::kPitch + lcol;
      const v4i lo = *reinterpret_cast<const v4i*>(from);
      const v4i hi = *reinterpret_cast<const v4i*>(from + 4);
      const float s0 = s[0];
      const V8 r0 = res[0];
#pragma unroll
      for (int u = 0; u + 1 < kAhead; ++u) {
        s[u] = s[u + 1];
        res[u] = res[u + 1];
      }
      if ((ph * kIters + it + kAhead) < kPhases * kIters) ahead(kAhead - 1, row + kAhead * kRows);
      if (row >= E.m) continue;
      if (!whole) {
        put_ragged(E, row, col, from);
        continue;
      }
      float z[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        z[u] = pre_activation(u < 4 ? lo[u & 3] : hi[u & 3], s0, t[u], b[u]);
      activate_all(z, E.act);
      V8 o;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (E.residual) z[u] += (float)r0[u];
        o[u] = (O)z[u];
      }
      *reinterpret_cast<V8*>(E.c + row * E.ldc + col) = o;
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

typedef Tile<256, 256, 2, 4> TileLarge;
typedef Tile<128, 128, 2, 2> TileMid;

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
