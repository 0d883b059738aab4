// Tiles of exact int8 products with K contiguous in both operands (X m x k, W n x k): the way
// of the operands through LDS, and the main loop of the smaller tiles.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "lds_dma.h"

namespace ozk {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));

// Workgroup barrier that no LDS access is moved across.
__device__ __forceinline__ void wg_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

constexpr int kStepK = 128;   // K bytes of a step: whole cache lines of every row
constexpr int kXcds = 8;

// Shape of a workgroup tile: kBM x kBN outputs by kWR x kWC waves (times kKG, which split each
// K step), each wave TI x TJ blocks of 16 x 16, operands in a ring of kS stages of one K step.
template <int kBM, int kBN, int kWR, int kWC, int kKG, int kS>
struct Tile {
  static constexpr int BM = kBM, BN = kBN, WR = kWR, WC = kWC, KG = kKG, S = kS;
  static constexpr int NW = WR * WC * KG;
  static constexpr int WM = BM / WR, WN = BN / WC;
  static constexpr int TI = WM / 16, TJ = WN / 16;
  static constexpr int kStage = (BM + BN) * kStepK;   // bytes
  static constexpr int kLoads = kStage / 1024 / NW;   // 1 KiB (8 rows) per wave and load
  static constexpr int kPitch = WN + 4;               // staged outputs of a wave, in words
  // row blocks a wave finishes, and how many of them its share of the ring stages at once
  static constexpr int kOwn = TI / KG;
  static constexpr int kFit = S * kStage / NW / (16 * kPitch * 4);
  static constexpr int kPhase = kFit >= kOwn ? kOwn : (kFit >= kOwn / 2 ? kOwn / 2 : kOwn / 4);
  static_assert(BM % 16 == 0 && kStage % (1024 * NW) == 0, "loads are whole");
  static_assert(NW % 2 == 0 && BM % 16 == 0, "one chunk for all loads of a lane");
  static_assert(kOwn % kPhase == 0 && kPhase * 16 * kPitch * 4 * NW <= S * kStage, "staging fits");
  static_assert(S >= 2 && S <= 6 && kLoads * (S - 1) <= 63, "the load counter's range");
};

// A workgroup's place in the order of the launch.  The hardware deals blocks out round-robin
// over the 8 XCDs; XCD x takes one contiguous run of the order, so that neighbours in it share
// panels in its L2.
__device__ __forceinline__ int xcd_order() {
  const int total = gridDim.x, per = total / kXcds, extra = total % kXcds;
  const int xcd = blockIdx.x % kXcds;
  return xcd * per + (xcd < extra ? xcd : extra) + blockIdx.x / kXcds;
}

// A workgroup's tile: which one, its K steps, and its operands' way into the ring.  Rows are
// 16-byte aligned and k is a multiple of 16 (other operands are laid out so first).
// An LDS row is 128 bytes, its eight 16-byte chunks XORed with (row >> 1) & 7 so that the 16
// lanes of a fragment read (rows r .. r + 15, one logical chunk) cover all 64 banks.
template <typename TL>
struct Walk {
  static constexpr int BM = TL::BM, BN = TL::BN, NW = TL::NW, S = TL::S, L = TL::kLoads;
  int8_t* lds;
  int wave, lane;
  int t0, nk;              // K steps t0 .. t0 + nk - 1
  int64_t row0, col0, k;
  const int8_t* base_x;
  const int8_t* base_w;
  uint32_t voff[L];        // row offset from the tile's first row, per load
  uint32_t chunk16, wave_lds;

  // Tile `tile` of tiles_m x tiles_n in groups of group_m tile rows (column, then row in
  // group), K steps first .. first + count - 1.
  __device__ __forceinline__ Walk(int8_t* ring, int64_t m, int64_t n, int64_t kk,
                                  const int8_t* x, int64_t ldx, const int8_t* w, int64_t ldw,
                                  int tile, int tiles_m, int tiles_n, int group_m, int first,
                                  int count)
      : lds(ring), t0(first), nk(count), k(kk) {
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int per_group = group_m * tiles_n, first_m = tile / per_group * group_m;
    const int gsize = tiles_m - first_m < group_m ? tiles_m - first_m : group_m;
    const int in_group = tile % per_group;
    row0 = (int64_t)(first_m + in_group % gsize) * BM;
    col0 = (int64_t)(in_group / gsize) * BN;
    base_x = x + row0 * ldx + (int64_t)t0 * kStepK;
    base_w = w + col0 * ldw + (int64_t)t0 * kStepK;
    // Load q of this wave: region rg = wave + NW q, rows 8 rg .. 8 rg + 7 of X (then of W);
    // lane i takes row i / 8 of it, physical chunk i % 8; rows past the matrix re-read its
    // last.  The swizzle depends on the region's parity alone, which is the wave's.
    chunk16 = 16 * ((lane & 7) ^ ((4 * wave + (lane >> 4)) & 7));
#pragma unroll
    for (int q = 0; q < L; ++q) {
      const int rg = wave + NW * q;
      const bool is_w = rg >= BM / 8;
      const int row = 8 * (is_w ? rg - BM / 8 : rg) + (lane >> 3);
      const int64_t origin = is_w ? col0 : row0, last = (is_w ? n : m) - 1;
      const int64_t gr = origin + row < last ? origin + row : last;
      voff[q] = (uint32_t)((gr - origin) * (is_w ? ldw : ldx));
    }
    wave_lds = __builtin_amdgcn_readfirstlane(lds_address(lds) + wave * 1024);
  }

  // K bytes left from the first byte of step t on
  __device__ __forceinline__ int64_t left(int t) const { return k - (int64_t)(t0 + t) * kStepK; }
  __device__ __forceinline__ const int8_t* stage(int t) const {
    return lds + (t % S) * TL::kStage;
  }

  // Load q of step t.  A chunk past k re-reads the row's last one (clear_tail).
  __device__ __forceinline__ void load(int t, int q) const {
    const bool is_w = wave + NW * q >= BM / 8;
    const int8_t* base = (is_w ? base_w : base_x) + (int64_t)t * kStepK;
    const int64_t rest = left(t) - 16;
    const uint32_t c = chunk16 < rest ? chunk16 : (uint32_t)rest;
    dma16_sbase(voff[q] + c, (uint64_t)base,
                wave_lds + (uint32_t)(t % S) * TL::kStage + q * (NW * 1024));
  }

  // Waits until of this wave's loads at most those of the youngest `younger` steps are under
  // way (`most`: the number that is asked for on every step but the last ones).
  template <int kMost>
  __device__ __forceinline__ void wait_loads(int younger) const {
    if (younger >= kMost) {
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(L * kMost) : "memory");
      return;
    }
    if (kMost > 3 && younger == 3) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(L * 3) : "memory");
    else if (kMost > 2 && younger == 2) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(L * 2) : "memory");
    else if (kMost > 1 && younger == 1) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(L) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  }

  // The ring's first stages asked for, step 0 in place for every wave.
  __device__ __forceinline__ void begin() const {
#pragma unroll
    for (int t = 0; t < S; ++t)
      if (t < nk)
#pragma unroll
        for (int q = 0; q < L; ++q) load(t, q);
    wait_loads<S - 1>(nk - 1);
    wg_barrier();
    clear_tail(0);
  }

  // The chunks of X past k in the row's last, short step (whole chunks: k is a multiple of
  // 16) are made zero in LDS, all waves together; what W holds there then does not count.
  __device__ __forceinline__ void clear_tail(int t) const {
    if (t >= nk || left(t) >= kStepK) return;
    const int first = (int)left(t) / 16;
    for (int i = threadIdx.x; i < BM * 8; i += 64 * NW) {
      const int row = i >> 3, c = i & 7;
      if (c >= first)
        *reinterpret_cast<v4i*>(lds + (t % S) * TL::kStage + row * kStepK +
                                ((c ^ ((row >> 1) & 7)) << 4)) = v4i{0, 0, 0, 0};
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    wg_barrier();
  }
};

// The smaller tiles, whose K steps take a fraction of a load's latency: as many stages as
// LDS holds, and per step one barrier, one set of fragment reads and one run of MFMAs.  A
// pair of waves shares the outputs of a wave and splits each step's K bytes, 64 for either
// (two waves per SIMD cover each other's reads); the sums of both meet in LDS at the end.
// Behind the barrier of step t the wave reads step t + 1 and asks for step t + S while step
// t's MFMAs run from registers.
// Wave kh of a pair ends with row blocks kh TI / 2 .. of the wave's tile in `own`, and all waves
// past their last use of the ring.  mxfp4_small_kernel (mxfp4_linear.hip) keeps the same order.
template <typename TL>
__device__ __forceinline__ void small_product(const Walk<TL>& W, v4i (&own)[TL::TI / 2][TL::TJ]) {
  constexpr int BM = TL::BM, TI = TL::TI, TJ = TL::TJ, S = TL::S, L = TL::kLoads;
  static_assert(TL::KG == 2 && TI % 2 == 0 && L <= TI * TJ, "pairs of waves");
  int8_t* const lds = W.lds;
  const int kh = W.wave / (TL::WR * TL::WC), wt = W.wave % (TL::WR * TL::WC);
  const int wr = wt / TL::WC, wc = wt % TL::WC, nk = W.nk;

  v4i acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = v4i{0, 0, 0, 0};

  const int frow = W.lane & 15, fchunk = W.lane >> 4, sw = frow >> 1;
  const int off = ((4 * kh + fchunk) ^ sw) << 4;
  const int arow = (wr * TL::WM + frow) * kStepK + off;
  const int brow = (BM + wc * TL::WN + frow) * kStepK + off;
  v4i fa[2][TI], fb[2][TJ];
  auto read = [&](int set, int t) {
    const int8_t* st = W.stage(t);
#pragma unroll
    for (int j = 0; j < TJ; ++j)
      fb[set][j] = *reinterpret_cast<const v4i*>(st + brow + j * 16 * kStepK);
#pragma unroll
    for (int i = 0; i < TI; ++i)
      fa[set][i] = *reinterpret_cast<const v4i*>(st + arow + i * 16 * kStepK);
  };
  auto step = [&](int set, int t) {
    W.template wait_loads<S - 2>(nk - 2 - t);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    wg_barrier();
    W.clear_tail(t + 1);
    __builtin_amdgcn_sched_barrier(0);
    if (t + 1 < nk) read(set ^ 1, t + 1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int idx = 0; idx < TI * TJ; ++idx) {
      const int i = idx / TJ, j = idx % TJ;
      acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb[set][j], fa[set][i], acc[i][j], 0, 0, 0);
      if (idx < L && t + S < nk) W.load(t + S, idx);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  W.begin();
  read(0, 0);
  int t = 0;
  for (; t + 1 < nk; t += 2) {
    step(0, t);
    step(1, t + 1);
  }
  if (t < nk) step(0, t);

  // Wave kh of a pair finishes row blocks kh TI / 2 ..: the other half goes to its partner.
  wg_barrier();   // every wave is past its last read of the ring
  constexpr int H = TI / 2;
  v4i* boxes = reinterpret_cast<v4i*>(lds);   // [wave][H][TJ][lane]
  static_assert(TL::NW * H * TJ * 1024 <= S * TL::kStage, "halves fit the ring");
  #pragma unroll
  for (int i = 0; i < H; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      boxes[((W.wave * H + i) * TJ + j) * 64 + W.lane] = kh ? acc[i][j] : acc[H + i][j];
      own[i][j] = kh ? acc[H + i][j] : acc[i][j];
    }
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  wg_barrier();
  const int partner = wt + (kh ? 0 : TL::WR * TL::WC);
#pragma unroll
  for (int i = 0; i < H; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) own[i][j] += boxes[((partner * H + i) * TJ + j) * 64 + W.lane];
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  wg_barrier();
}

typedef Tile<128, 128, 2, 2, 2, 4> TileMid;
typedef Tile<64, 128, 1, 4, 2, 6> TileSmall;

}  // namespace
}  // namespace ozk
