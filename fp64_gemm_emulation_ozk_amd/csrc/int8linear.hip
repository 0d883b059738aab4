// int8 linear layer: C = act(s t^T * (X W^T) + 1 b^T) + R, X m x k and W n x k int8 with K
// contiguous in both, s and t fp32 scales of their rows.  The int8 product is exact in
// int32 (k <= OZK_MAX_K); everything after it is fp32, rounded once to the output's type.
#include "activation.h"
#include "ozk_internal.h"
#include "rows.h"
#include "tile_walk.h"

namespace ozk {
namespace {

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
  z = activate32<sizeof(O) == 4>(z, E.act);
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
    activate_all<sizeof(O) == 4>(z, E.act);
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

// Bytes h .. h + 15 of a row of k, zero past k, at any alignment, in two steps so that many
// loads can be on their way: the 16 bytes at h or, where those leave the row, its last 16;
// and the shift that moves what lies past k out.  k >= 16.
__device__ __forceinline__ v4i load16(const int8_t* __restrict__ p, int64_t h, int64_t k) {
  return *reinterpret_cast<const v4i_bytes*>(p + (h + 16 <= k ? h : k - 16));
}
__device__ __forceinline__ v4i shift16(const v4i& v, int64_t h, int64_t k) {
  const int64_t over = h + 16 - k;   // bytes past k
  if (over <= 0) return v;
  if (over >= 16) return v4i{0, 0, 0, 0};
  uint64_t lo = (uint64_t)(uint32_t)v[0] | (uint64_t)(uint32_t)v[1] << 32;
  uint64_t hi = (uint64_t)(uint32_t)v[2] | (uint64_t)(uint32_t)v[3] << 32;
  const int bits = 8 * (int)over;   // 8 .. 120
  if (bits >= 64) {
    lo = hi >> (bits - 64);
    hi = 0;
  } else {
    lo = lo >> bits | hi << (64 - bits);
    hi >>= bits;
  }
  return v4i{(int)(uint32_t)lo, (int)(uint32_t)(lo >> 32), (int)(uint32_t)hi,
             (int)(uint32_t)(hi >> 32)};
}

// The bytes of a row of fewer than 16.
__device__ __forceinline__ v4i load_short(const int8_t* __restrict__ p, int64_t h, int64_t k) {
  uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int u = 0; u < 15; ++u)
    if (h + u < k) w[u >> 2] |= (uint32_t)(uint8_t)p[h + u] << (8 * (u & 3));
  return v4i{(int)w[0], (int)w[1], (int)w[2], (int)w[3]};
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

// Few rows at any alignment: workgroup = 16 kMT rows x 16 kNT columns of C, its kWaves waves
// taking the K steps of 128 bytes in turn (of the workgroup's split of K).  Operands go from
// global memory to the matrix core's registers directly: lane l of a fragment holds row
// l % 16 and 16 bytes of K.  Whole steps run kDeep at a time, all their loads issued first.
// 37 x 4100 x 1001: 7.5 us, of which a launch is 3 to 4; the 4.1 MB of W come out of the L2s.
template <typename O, int kMT, int kNT, int kWaves, int kDeep>
__global__ __launch_bounds__(64 * kWaves) void int8linear_few_kernel(
    int64_t k, const int8_t* __restrict__ x, int64_t ldx, const int8_t* __restrict__ w,
    int64_t ldw, Epilogue<O> E, int splits, int32_t* __restrict__ part) {
  __shared__ v4i sums[kWaves][kMT * kNT][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int split = blockIdx.x % splits;
  const int64_t col0 = (int64_t)(blockIdx.x / splits) * (16 * kNT), lo = 16 * (lane >> 4);
  const int8_t* wp[kNT];
#pragma unroll
  for (int j = 0; j < kNT; ++j) {
    const int64_t r = col0 + 16 * j + (lane & 15);
    wp[j] = w + (r < E.n ? r : E.n - 1) * ldw;
  }
  const int8_t* xp[kMT];
#pragma unroll
  for (int i = 0; i < kMT; ++i) {
    const int64_t r = 16 * i + (lane & 15);
    xp[i] = x + (r < E.m ? r : E.m - 1) * ldx;
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
        const int64_t at = (t + d * kWaves) * 128 + 64 * h + lo;
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
    v4i fb[2][kNT], fa[2][kMT];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t at = t * 128 + 64 * h + lo;
#pragma unroll
      for (int j = 0; j < kNT; ++j)
        fb[h][j] = k < 16 ? load_short(wp[j], at, k) : load16(wp[j], at, k);
#pragma unroll
      for (int i = 0; i < kMT; ++i)
        fa[h][i] = k < 16 ? load_short(xp[i], at, k) : load16(xp[i], at, k);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t at = t * 128 + 64 * h + lo;
      if (k >= 16) {
#pragma unroll
        for (int j = 0; j < kNT; ++j) fb[h][j] = shift16(fb[h][j], at, k);
#pragma unroll
        for (int i = 0; i < kMT; ++i) fa[h][i] = shift16(fa[h][i], at, k);
      }
#pragma unroll
      for (int i = 0; i < kMT; ++i)
#pragma unroll
        for (int j = 0; j < kNT; ++j)
          acc[i][j] =
              __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[h][j], fa[h][i], acc[i][j], 0, 0, 0);
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
    const int64_t row = 16 * (b / kNT) + (lane & 15);
    const int64_t col = col0 + 16 * (b % kNT) + 4 * (lane >> 4);
    if (part)
      put_part(part + split * E.m * E.n, row, col, E.m, E.n, s);
    else
      put4(E, row, col, s);
  }
}

// Up to 16 rows, aligned operands (as the tiles'): the same split of the work, but each wave
// streams its steps through a ring of its own in LDS by direct loads of 8 rows x 128 bytes.
// Sixteen rows x 64 bytes straight into registers, lane by lane another row, get a quarter of
// that rate (38 against 152 bytes/ns per CU from L2, 19 against 27 from HBM).  No barriers:
// a wave waits for its own loads, reads its fragments and refills the slot.  kXR rows of X
// (8 for up to 8) travel with each step.  1 x 8192 x 8192: 13.4 us, 67 MB at 5.0 TB/s (a large
// copy: 5.5); bound by HBM.
template <typename O, int kXR, int kS>
__global__ __launch_bounds__(512) void int8linear_stream_kernel(
    int64_t k, const int8_t* __restrict__ x, int64_t ldx, const int8_t* __restrict__ w,
    int64_t ldw, Epilogue<O> E, int splits, int32_t* __restrict__ part) {
  constexpr int kWaves = 8, kSlot = (16 + kXR) * 128, L = kSlot / 1024;
  __shared__ __attribute__((aligned(1024))) int8_t lds[kWaves * kS * kSlot];
  static_assert(kWaves * 1024 <= kWaves * kS * kSlot, "the sums fit the ring");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int split = blockIdx.x % splits;
  const int64_t col0 = (int64_t)(blockIdx.x / splits) * 16;
  const int steps = (int)((k + 127) / 128);
  const int t0 = (int)((int64_t)steps * split / splits) + wave;
  const int t1 = (int)((int64_t)steps * (split + 1) / splits);
  const int own = t0 < t1 ? (t1 - t0 + kWaves - 1) / kWaves : 0;   // steps t0 + 8 i
  // load q: 8 rows of W (q < 2) or X; lane i takes row i / 8, physical chunk i % 8, which
  // holds logical chunk (i % 8) ^ ((row >> 1) & 7)
  uint32_t voff[L], chunk[2];
#pragma unroll
  for (int q = 0; q < L; ++q) {
    const bool is_w = q < 2;
    const int64_t r = 8 * (is_w ? q : q - 2) + (lane >> 3);
    const int64_t last = is_w ? E.n - 1 - col0 : E.m - 1;
    voff[q] = (uint32_t)((r < last ? r : last) * (is_w ? ldw : ldx));
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) chunk[q] = 16 * ((lane & 7) ^ ((4 * q + (lane >> 4)) & 7));
  const uint32_t ring = __builtin_amdgcn_readfirstlane(lds_address(lds) + wave * (kS * kSlot));
  const int8_t* wbase = w + col0 * ldw;
  auto load = [&](int i) {
    const int64_t at = (int64_t)(t0 + kWaves * i) * 128, rest = k - at - 16;
    const uint32_t slot = ring + (uint32_t)(i % kS) * kSlot;
#pragma unroll
    for (int q = 0; q < L; ++q) {
      const uint32_t c = chunk[q & 1] < rest ? chunk[q & 1] : (uint32_t)rest;
      dma16_sbase(voff[q] + c, (uint64_t)((q < 2 ? wbase : x) + at), slot + q * 1024);
    }
  };
  const int frow = lane & 15, fchunk = lane >> 4;
  v4i acc{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < kS; ++i)
    if (i < own) load(i);
  for (int i = 0; i < own; ++i) {
    const int younger = own - 1 - i;
    if (younger >= kS - 1) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(L * (kS - 1)) : "memory");
    else if (kS > 3 && younger == 2) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(L * 2) : "memory");
    else if (kS > 2 && younger == 1) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(L) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    const int8_t* slot = lds + wave * (kS * kSlot) + (i % kS) * kSlot;
    const int xrow = frow & (kXR - 1);
    v4i fb[2], fa[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      fb[h] = *reinterpret_cast<const v4i*>(slot + frow * 128 +
                                            (((4 * h + fchunk) ^ ((frow >> 1) & 7)) << 4));
      fa[h] = *reinterpret_cast<const v4i*>(slot + (16 + xrow) * 128 +
                                            (((4 * h + fchunk) ^ ((xrow >> 1) & 7)) << 4));
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    if (i + kS < own) load(i + kS);
    const int64_t left = k - (int64_t)(t0 + kWaves * i) * 128;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (left < 128) fa[h] = 64 * h + 16 * fchunk < left ? fa[h] : v4i{0, 0, 0, 0};
      acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[h], fa[h], acc, 0, 0, 0);
    }
  }
  // every wave is past its ring: the sums take its first bytes
  __syncthreads();
  v4i* sums = reinterpret_cast<v4i*>(lds);
  sums[wave * 64 + lane] = acc;
  __syncthreads();
  if (wave) return;
#pragma unroll
  for (int v = 1; v < kWaves; ++v) acc += sums[v * 64 + lane];
  const int64_t row = frow, col = col0 + 4 * fchunk;
  if (part)
    put_part(part + split * E.m * E.n, row, col, E.m, E.n, acc);
  else
    put4(E, row, col, acc);
}

// ------------------------------------------------------------------ tiles
// A workgroup's tile and split of K in the order (split, tile).
struct Place {
  int split, tile, t0, nk;
  __device__ __forceinline__ Place(int64_t k, int tiles, int splits) {
    const int id = xcd_order(), steps = (int)((k + kStepK - 1) / kStepK);
    split = id / tiles;
    tile = id - split * tiles;
    t0 = (int)((int64_t)steps * split / splits);
    nk = (int)((int64_t)steps * (split + 1) / splits) - t0;
  }
};

// The outputs of a wave's NI x TJ blocks (lane l of block (i, j): row 16 i + l % 16, columns
// 16 j + 4 (l / 16) .. + 3), or their partial sums.  The blocks are staged through this wave's
// part `mine` of the ring so that eight lanes finish one row of 64 columns, eight consecutive
// outputs each.  The rows' scales and residuals are asked for four groups of rows ahead: an
// output's own work is short, the latency of its operands is not.  The loop over the groups
// of a phase is kept a loop: written out, the epilogue does not fit the instruction cache
// (4096 x 16384 x 4096 with gelu and residual took 1.23 ms so, 0.29 as a loop).
template <typename TL, typename O, int NI>
__device__ __forceinline__ void put_tile(const Epilogue<O>& E, const v4i (&acc)[NI][TL::TJ],
                                         int64_t wrow0, int64_t wcol0, int lane, int32_t* mine,
                                         int32_t* __restrict__ part) {
  constexpr int TJ = TL::TJ;
  const int frow = lane & 15, fchunk = lane >> 4;
  if (part) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < TJ; ++j)
        put_part(part, wrow0 + 16 * i + frow, wcol0 + 16 * j + 4 * fchunk, E.m, E.n, acc[i][j]);
    return;
  }
  typedef O V8 __attribute__((ext_vector_type(8), aligned(sizeof(O))));
  typedef float F8 __attribute__((ext_vector_type(8), aligned(4)));
  constexpr int kLanes = TL::WN / 8, kRows = 64 / kLanes;        // lanes of a row, rows at once
  constexpr int kIters = TL::kPhase * 16 / kRows, kPhases = NI / TL::kPhase, kAhead = 4;
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
  for (int u = 0; u < kAhead; ++u)
    if (u < kIters * kPhases) ahead(u, wrow0 + u * kRows + lrow);
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
      activate_all<sizeof(O) == 4>(z, E.act);
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

// The large tile, whose K steps are long: per step every wave runs quarters of 2 x TJ blocks;
// before the last one it waits for its loads of step t + 1 and for its reads of step t (the
// last quarter's operands are in registers by then), so one barrier a step makes step t + 1
// complete and step t's stage free for step t + S, whose loads have S - 1 steps to land less
// a quarter.  Two stages are enough.  8192^3 to bf16: 445 us, 2.47 POP/s; 4096 x 16384 x 4096
// with gelu and residual 290 to 300 us, 1.85 POP/s, a quarter of it the epilogues of its four
// rounds of tiles (268 MB of outputs and residual, and their instructions).
template <typename O, typename TL>
__global__ __launch_bounds__(64 * TL::NW) void int8linear_tile_kernel(
    int64_t k, const int8_t* __restrict__ x, int64_t ldx, const int8_t* __restrict__ w,
    int64_t ldw, Epilogue<O> E, int tiles_m, int tiles_n, int splits, int group_m,
    int32_t* __restrict__ part) {
  constexpr int BM = TL::BM, TI = TL::TI, TJ = TL::TJ, S = TL::S, L = TL::kLoads;
  static_assert(TL::KG == 1, "one wave for both K halves");
  __shared__ __attribute__((aligned(1024))) int8_t lds[S * TL::kStage];
  const Place p(k, tiles_m * tiles_n, splits);
  const Walk<TL> W(lds, E.m, E.n, k, x, ldx, w, ldw, p.tile, tiles_m, tiles_n, group_m, p.t0,
                   p.nk);
  const int wr = W.wave / TL::WC, wc = W.wave % TL::WC, nk = W.nk;

  v4i acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = v4i{0, 0, 0, 0};

  const int frow = W.lane & 15, fchunk = W.lane >> 4, sw = frow >> 1;
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
        W.load(tl, (idx * L) / kQuarter);
      __builtin_amdgcn_sched_barrier(0);
      // the wave that reaches the second half of a quarter first is preferred, so the two
      // waves of a SIMD run apart
      if (idx == kQuarter / 2 - 1) __builtin_amdgcn_s_setprio(1);
    }
    __builtin_amdgcn_s_setprio(0);
  };

  W.begin();
#pragma unroll
  for (int idx = 0; idx < 4; ++idx) read_a(0, lds, idx & 1, idx >> 1, idx >> 1);
#pragma unroll
  for (int j = 0; j < TJ; ++j) {
    read_b(lds, 0, j);
    read_b(lds, 1, j);
  }
  for (int t = 0; t < nk; ++t) {
    __builtin_amdgcn_sched_barrier(0);
    const int8_t* st = W.stage(t);
#pragma unroll
    for (int q = 0; q < NQ - 1; ++q) quarter(q, st, st, nk);
    // this wave's loads of step t + 1 have landed and it has read all of step t; past the
    // barrier that holds for every wave
    W.template wait_loads<S - 2>(nk - 2 - t);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    wg_barrier();
    W.clear_tail(t + 1);
    __builtin_amdgcn_sched_barrier(0);
    // after the last step: a harmless re-read of it
    quarter(NQ - 1, st, t + 1 < nk ? W.stage(t + 1) : st, t + S);
  }
  wg_barrier();   // every wave is past its last read of the ring
  put_tile<TL, O, TI>(E, acc, W.row0 + wr * TL::WM, W.col0 + wc * TL::WN, W.lane,
                      reinterpret_cast<int32_t*>(lds) + W.wave * (TL::kPhase * 16 * TL::kPitch),
                      part ? part + (int64_t)p.split * E.m * E.n : nullptr);
}

template <typename O, typename TL>
__global__ __launch_bounds__(64 * TL::NW) void int8linear_small_kernel(
    int64_t k, const int8_t* __restrict__ x, int64_t ldx, const int8_t* __restrict__ w,
    int64_t ldw, Epilogue<O> E, int tiles_m, int tiles_n, int splits, int group_m,
    int32_t* __restrict__ part) {
  constexpr int H = TL::TI / 2;
  __shared__ __attribute__((aligned(1024))) int8_t lds[TL::S * TL::kStage];
  const Place p(k, tiles_m * tiles_n, splits);
  const Walk<TL> W(lds, E.m, E.n, k, x, ldx, w, ldw, p.tile, tiles_m, tiles_n, group_m, p.t0,
                   p.nk);
  v4i own[H][TL::TJ];
  small_product<TL>(W, own);
  const int kh = W.wave / (TL::WR * TL::WC), wt = W.wave % (TL::WR * TL::WC);
  put_tile<TL, O, H>(E, own, W.row0 + wt / TL::WC * TL::WM + kh * 16 * H,
                     W.col0 + wt % TL::WC * TL::WN, W.lane,
                     reinterpret_cast<int32_t*>(lds) + W.wave * (TL::kPhase * 16 * TL::kPitch),
                     part ? part + (int64_t)p.split * E.m * E.n : nullptr);
}

// Rows of k bytes at any alignment laid out with leading dimension kp (a multiple of 16),
// zeros from k on: both operands in one launch, 16 bytes a thread.
__global__ __launch_bounds__(256) void int8linear_layout_kernel(
    int64_t m, int64_t n, int64_t k, int64_t kp, const int8_t* __restrict__ x, int64_t ldx,
    int8_t* __restrict__ xo, const int8_t* __restrict__ w, int64_t ldw,
    int8_t* __restrict__ wo) {
  const int64_t chunks = kp / 16, id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  int64_t row = id / chunks;
  const int64_t h = id % chunks * 16;
  if (row >= m + n) return;
  const bool is_w = row >= m;
  row -= is_w ? m : 0;
  const int8_t* p = is_w ? w + row * ldw : x + row * ldx;
  const v4i v = k < 16 ? load_short(p, h, k) : shift16(load16(p, h, k), h, k);
  *reinterpret_cast<v4i*>((is_w ? wo : xo) + row * kp + h) = v;
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

typedef Tile<256, 256, 2, 4, 1, 2> TileLarge;

// How a product is run: by the kernels for few rows (a workgroup takes all rows) or by tiles
// of one shape; K is split over `splits` workgroups where there are fewer tiles than the
// compute units take.
enum Shape { kStream, kFew, kSmall, kMid, kLarge };
struct Plan {
  Shape shape;
  int64_t tiles_m, tiles_n;
  int splits;
};

// Up to 16 rows: the stream kernel; unaligned, up to 64 rows, the few kernel (37 x 4100 x 1001:
// 7.5 us, against 13.8 with the operands laid out for a tile).  More rows: the tile shape and
// split of the least estimated time, in microseconds, of rounds of 256 workgroups that each
// cost `fixed` and `step` per K step.  Measured, one round of 4096 K values: small 22.7, mid
// 29, large 61 (512, 1024, 4096 x 4096 outputs), and 5.3, 7.1, 9.6 for 128.  A split costs the
// launch of the join and the partial sums' way out and back (5 TB/s).
Plan plan_of(int64_t m, int64_t n, int64_t k, bool aligned) {
  const int64_t steps = (k + kStepK - 1) / kStepK;
  if (m <= (aligned ? 16 : 64)) {
    const int64_t bn = m <= 16 ? 16 : 32;
    Plan p{aligned ? kStream : kFew, 1, (n + bn - 1) / bn, 1};
    // a workgroup's eight waves take eight steps each at least
    const int64_t s = 256 / p.tiles_n, most = steps / 64;
    p.splits = (int)(s < most ? s : most);
    if (p.splits < 1) p.splits = 1;
    return p;
  }
  struct Cost {
    Shape shape;
    int64_t bm, bn;
    double fixed, step;
  };
  const Cost costs[] = {{kSmall, 64, 128, 4.8, 0.55}, {kMid, 128, 128, 6.3, 0.72},
                        {kLarge, 256, 256, 8.2, 1.65}};
  Plan best{};
  double least = 0;
  for (const Cost& c : costs) {
    const int64_t tm = (m + c.bm - 1) / c.bm, tn = (n + c.bn - 1) / c.bn, tiles = tm * tn;
    for (int64_t sp = 1; sp <= 16 && (sp == 1 || (tiles * sp <= 256 && steps / sp >= 4)); ++sp) {
      const double rounds = (double)((tiles * sp + 255) / 256);
      double t = rounds * (c.fixed + c.step * (double)((steps + sp - 1) / sp));
      if (sp > 1) t += 3.0 + (double)sp * (double)m * (double)n * 8.0 / 5e6;
      if (least == 0 || t < least) {
        least = t;
        best = {c.shape, tm, tn, (int)sp};
      }
    }
  }
  return best;
}

size_t partial_bytes(const Plan& p, int64_t m, int64_t n) {
  return p.splits > 1 ? align256((size_t)p.splits * m * n * 4) : 0;
}

// What the tiles' direct loads take: 16-byte aligned rows, whole chunks of K, and a lane's
// offset within a tile in 32 bits.
bool rows_aligned(const int8_t* x, int64_t ldx, const int8_t* w, int64_t ldw, int64_t k) {
  return (((uintptr_t)x | (uintptr_t)w | (uint64_t)ldx | (uint64_t)ldw | (uint64_t)k) & 15) == 0 &&
         ldx < (1 << 24) && ldw < (1 << 24);
}

template <typename O, typename TL>
void launch_tiles(const Plan& p, int64_t k, const int8_t* x, int64_t ldx, const int8_t* w,
                  int64_t ldw, const Epilogue<O>& E, int32_t* part, hipStream_t s) {
  const int group_m = 8;
  const dim3 grid((unsigned)(p.tiles_m * p.tiles_n * p.splits)), block(64 * TL::NW);
  int32_t* const sums = p.splits > 1 ? part : nullptr;
  if constexpr (TL::KG == 1)
    hipLaunchKernelGGL((int8linear_tile_kernel<O, TL>), grid, block, 0, s, k, x, ldx, w, ldw, E,
                       (int)p.tiles_m, (int)p.tiles_n, p.splits, group_m, sums);
  else
    hipLaunchKernelGGL((int8linear_small_kernel<O, TL>), grid, block, 0, s, k, x, ldx, w, ldw, E,
                       (int)p.tiles_m, (int)p.tiles_n, p.splits, group_m, sums);
}

template <typename O>
int int8linear_t(int64_t m, int64_t n, int64_t k, const int8_t* x, int64_t ldx, const float* sx,
                 const int8_t* w, int64_t ldw, const float* sw, const void* bias, int act,
                 const void* residual, int64_t ldr, void* c, int64_t ldc, void* workspace,
                 hipStream_t s) {
  const Epilogue<O> E{m, n, sx, sw, (const O*)bias, (const O*)residual, ldr, (O*)c, ldc, act};
  const bool aligned = rows_aligned(x, ldx, w, ldw, k);
  const Plan p = plan_of(m, n, k, aligned);
  int32_t* part = static_cast<int32_t*>(workspace);
  // a launch takes fewer than 2^32 threads, 512 a workgroup
  if (p.tiles_m * p.tiles_n * p.splits >= 1 << 23) return OZK_EUNSUPPORTED;
  if (p.shape == kStream || p.shape == kFew) {
    const dim3 grid((unsigned)(p.tiles_n * p.splits)), block(512);
    int32_t* const sums = p.splits > 1 ? part : nullptr;
#define OZK_FEW(KERNEL) \
  hipLaunchKernelGGL(KERNEL, grid, block, 0, s, k, x, ldx, w, ldw, E, p.splits, sums)
    if (p.shape == kStream && m <= 8) OZK_FEW((int8linear_stream_kernel<O, 8, 3>));
    else if (p.shape == kStream) OZK_FEW((int8linear_stream_kernel<O, 16, 4>));
    else if (m <= 16) OZK_FEW((int8linear_few_kernel<O, 1, 1, 8, 4>));
    else if (m <= 32) OZK_FEW((int8linear_few_kernel<O, 2, 2, 8, 2>));
    else OZK_FEW((int8linear_few_kernel<O, 4, 2, 8, 1>));
#undef OZK_FEW
  } else {
    if (!aligned) {
      const int64_t kp = round_up(k, 16);
      int8_t* xo = static_cast<int8_t*>(workspace) + partial_bytes(p, m, n);
      int8_t* wo = xo + align256((size_t)m * kp);
      const int64_t blocks = ((m + n) * (kp / 16) + 255) / 256;
      if (blocks >= 1 << 24) return OZK_EUNSUPPORTED;
      hipLaunchKernelGGL(int8linear_layout_kernel, dim3((unsigned)blocks), dim3(256), 0, s, m, n,
                         k, kp, x, ldx, xo, w, ldw, wo);
      x = xo;
      w = wo;
      ldx = ldw = k = kp;
    }
    if (p.shape == kLarge) launch_tiles<O, TileLarge>(p, k, x, ldx, w, ldw, E, part, s);
    else if (p.shape == kMid) launch_tiles<O, TileMid>(p, k, x, ldx, w, ldw, E, part, s);
    else launch_tiles<O, TileSmall>(p, k, x, ldx, w, ldw, E, part, s);
  }
  if (p.splits > 1)
    hipLaunchKernelGGL((int8linear_join_kernel<O>),
                       dim3((unsigned)((m * ((n + 3) / 4) + 255) / 256)), dim3(256), 0, s, E,
                       p.splits, part);
  return hipGetLastError() == hipSuccess ? OZK_OK : OZK_EHIP;
}

}  // namespace

bool int8linear_aligned(const int8_t* x, int64_t ldx, const int8_t* w, int64_t ldw, int64_t k) {
  return rows_aligned(x, ldx, w, ldw, k);
}

size_t int8linear_workspace(int64_t m, int64_t n, int64_t k, bool aligned) {
  if (m <= 0 || n <= 0) return 0;
  const Plan p = plan_of(m, n, k, aligned);
  size_t bytes = partial_bytes(p, m, n);
  if (p.shape >= kSmall && !aligned) {
    const int64_t kp = round_up(k, 16);
    bytes += align256((size_t)m * kp) + align256((size_t)n * kp);
  }
  return bytes;
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
