// Linear layer and gated feed-forward block on microscaled 4-bit operands:
//   C = act(X W^T + 1 b^T) + R,   and, W = [Wg; Wu],   C = act(X Wg^T + 1 bg^T) * (X Wu^T + 1 bu^T)
// X m x k and W n (2n) x k as MX FP4 lines.  A v_mfma_scale_f32_16x16x128_f8f6f4 takes 32 codes
// and their scale from every lane, so a lane's 16 bytes of a line are one block; sums are fp32,
// and what follows them is fp32, rounded once to the output's type.
//
// Few rows are bound by the bytes of W: the stream kernel.  Many are bound by the matrix cores and
// by what feeds them: the tile kernels.  (us, bf16, MI355X; a replayed graph)
//   rows of 8192 x 8192:  1: 6.2   16: 7.0   32: 8.5   64: 11.6   128: 19.4   256: 23   512: 29
//   8192^3: 251 (4.4 PFLOP/s); 4096 x 16384 x 4096: 143, with gelu 171, with a residual 165, with
//   both 184; gated 4096 x 2 8192 x 4096: 139
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
// byte kH of its two.  Lane (row lane % 16, quarter lane / 16) gives 32 codes of its line; lane l
// of the sum holds line l % 16 of x and lines 4 (l / 16) .. + 3 of w.
template <int kH>
__device__ __forceinline__ v4f mfma_mx(const v4i& w, int sw, const v4i& x, int sx, const v4f& c) {
  const v8i w8 = {w[0], w[1], w[2], w[3], 0, 0, 0, 0};
  const v8i x8 = {x[0], x[1], x[2], x[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w8, x8, c, 4, 4, kH, sw, kH, sx);
}

// In LDS a line's step is 128 bytes, whose eight 16-byte chunks are XORed with swizzle(line).  A
// fragment read of 16 bytes a lane is served 16 lanes at a time, eight lines of one quarter and
// the other eight of its neighbour (lanes 0-3, 12-15, 20-27, and so on), which here read chunks
// two apart: these 16 fall on all 64 banks if lines 4 .. 11 of 16 have swizzles that stay among
// themselves under XOR with 2.  (With (line >> 1) & 7 alone, as where neighbours read chunks one
// apart, 0.44 of the LDS's busy cycles were conflicts.)
__device__ __forceinline__ int swizzle(int line) {
  const int x = (line >> 1) & 7;
  return x ^ ((x & 2) << 1);
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

// The outputs from col to the row's end, fewer than eight, from staged sums (gated: the other
// projection's `apart` further on).
template <bool kGated, typename O>
__device__ __forceinline__ void put_ragged(const MxEpilogue<O>& E, int64_t row, int64_t col,
                                           const float* sums, int apart) {
#pragma unroll 1
  for (int u = 0; col + u < E.n; ++u)
    put1<kGated>(E, row, col + u, sums[u], kGated ? sums[apart + u] : 0.0f);
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

// Four partial sums of a row of `wide`, the columns from col up to `end` of them.
__device__ __forceinline__ void put_part(float* __restrict__ p, int64_t row, int64_t col,
                                         int64_t m, int64_t end, int64_t wide, const v4f& acc) {
  if (row >= m || col >= end) return;
  if (col + 4 <= end) {
    *reinterpret_cast<v4f_words*>(p + row * wide + col) = acc;
    return;
  }
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (col + u < end) p[row * wide + col + u] = acc[u];
}

// Both projections' partial sums of four columns (not gated: `up` is not used).
template <bool kGated, typename O>
__device__ __forceinline__ void put_parts(const MxEpilogue<O>& E, float* __restrict__ p,
                                          int64_t row, int64_t col, const v4f& acc,
                                          const v4f& up) {
  const int64_t wide = kGated ? 2 * E.n : E.n;
  put_part(p, row, col, E.m, E.n, wide, acc);
  if constexpr (kGated)
    if (col < E.n) put_part(p + E.n, row, col, E.m, E.n, wide, up);
}

// Few rows: workgroup = 16 kNT columns of C (gated: of both projections) and all rows, its eight
// waves taking the K steps of 256 codes in turn (of the workgroup's split of K).  Each wave
// streams its steps through a ring of its own in LDS by direct loads of 8 lines x 128 bytes and
// of 32 lines' 8 scales.  No barriers: a wave waits for its own loads, reads its fragments and
// refills the slot, so that eight slots are under way even where a wave has but one.  kXR rows of
// X (8 to 64) travel with each step.
template <typename O, bool kGated, int kXR, int kNT, int kS>
__global__ __launch_bounds__(512) void mxfp4_stream_kernel(int steps, Lines X, Lines W,
                                                           MxEpilogue<O> E, int splits,
                                                           float* __restrict__ part) {
  constexpr int kG = kGated ? 2 : 1, kB = kNT * kG, kMT = kXR < 16 ? 1 : kXR / 16, kWaves = 8;
  constexpr int kRows = 16 * kB + kXR;
  constexpr int kCodes = kRows * 128, LC = kRows / 8, LS = (kRows + 31) / 32, L = LC + LS;
  constexpr int kSlot = kCodes + LS * 256;
  __shared__ __attribute__((aligned(1024))) int8_t lds[kWaves * kS * kSlot];
  static_assert(kWaves * kMT * kB * 1024 <= kWaves * kS * kSlot, "the sums fit the ring");
  static_assert(kS >= 1 && kS <= 3 && L * (kS - 1) <= 63, "the load counter's range");
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int split = blockIdx.x % splits;
  const int64_t col0 = (int64_t)(blockIdx.x / splits) * (16 * kNT);
  const int t0 = (int)((int64_t)steps * split / splits) + wave;
  const int t1 = (int)((int64_t)steps * (split + 1) / splits);
  const int own = t0 < t1 ? (t1 - t0 + kWaves - 1) / kWaves : 0;   // steps t0 + 8 i
  // line r of a step: of W's gate, of its other projection, then of X; lines past the operand
  // re-read its last
  auto line = [&](int r, bool& is_w) -> int64_t {
    is_w = r < 16 * kB;
    if (!is_w) {
      const int64_t row = r - 16 * kB;
      return row < E.m ? row : E.m - 1;
    }
    const int64_t col = col0 + r % (16 * kNT);
    return (col < E.n ? col : E.n - 1) + (kGated && r >= 16 * kNT ? E.n : 0);
  };
  // load q: lines 8 q .. 8 q + 7; lane i takes line i / 8 of them, physical chunk i % 8, which
  // holds logical chunk (i % 8) ^ swizzle(line)
  const uint8_t* from[L];
#pragma unroll
  for (int q = 0; q < LC; ++q) {
    bool is_w;
    const int64_t r = line(8 * q + (lane >> 3), is_w);
    const int chunk = 16 * ((lane & 7) ^ swizzle(8 * q + (lane >> 3)));
    from[q] = (is_w ? W.codes + r * W.ld : X.codes + r * X.ld) + (int64_t)t0 * 128 + chunk;
  }
#pragma unroll
  for (int q = 0; q < LS; ++q) {
    bool is_w;
    const int at = 32 * q + (lane >> 1);
    const int64_t r = line(at < kRows ? at : kRows - 1, is_w);
    from[LC + q] = (is_w ? W.scales + r * W.lds : X.scales + r * X.lds) + (int64_t)t0 * 8 +
                   4 * (lane & 1);
  }
  const uint32_t ring = __builtin_amdgcn_readfirstlane(lds_address(lds) + wave * (kS * kSlot));
  auto load = [&](int i) {
    const uint32_t slot = ring + (uint32_t)(i % kS) * kSlot;
#pragma unroll
    for (int q = 0; q < LC; ++q) dma16(from[q] + (int64_t)i * (kWaves * 128), slot + q * 1024);
#pragma unroll
    for (int q = 0; q < LS; ++q)
      dma4(from[LC + q] + (int64_t)i * (kWaves * 8), slot + kCodes + q * 256);
  };
  const int frow = lane & 15, quarter = lane >> 4, xrow = 16 * kB + (frow & (kXR - 1));
  v4f acc[kMT][kB];
#pragma unroll
  for (int i = 0; i < kMT; ++i)
#pragma unroll
    for (int j = 0; j < kB; ++j) acc[i][j] = v4f{0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < kS; ++i)
    if (i < own) load(i);
  for (int i = 0; i < own; ++i) {
    const int younger = own - 1 - i;
    if (younger >= kS - 1) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(L * (kS - 1)) : "memory");
    else if (kS > 2 && younger == 1) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(L) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    const int8_t* slot = lds + wave * (kS * kSlot) + (i % kS) * kSlot;
    auto codes = [&](int r, int h) {
      return *reinterpret_cast<const v4i*>(slot + r * 128 +
                                           (((2 * quarter + h) ^ swizzle(r)) << 4));
    };
    auto scale = [&](int r) -> int {
      return *reinterpret_cast<const uint16_t*>(slot + kCodes + r * 8 + 2 * quarter);
    };
    v4i fb[2][kB], fa[2][kMT];
    int sb[kB], sa[kMT];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int j = 0; j < kB; ++j) fb[h][j] = codes(16 * j + frow, h);
#pragma unroll
      for (int u = 0; u < kMT; ++u) fa[h][u] = codes(xrow + 16 * u, h);
    }
#pragma unroll
    for (int j = 0; j < kB; ++j) sb[j] = scale(16 * j + frow);
#pragma unroll
    for (int u = 0; u < kMT; ++u) sa[u] = scale(xrow + 16 * u);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    if (i + kS < own) load(i + kS);
#pragma unroll
    for (int u = 0; u < kMT; ++u)
#pragma unroll
      for (int j = 0; j < kB; ++j) {
        acc[u][j] = mfma_mx<0>(fb[0][j], sb[j], fa[0][u], sa[u], acc[u][j]);
        acc[u][j] = mfma_mx<1>(fb[1][j], sb[j], fa[1][u], sa[u], acc[u][j]);
      }
  }
  // every wave is past its ring: the sums take its first bytes
  __syncthreads();
  v4f* sums = reinterpret_cast<v4f*>(lds);
#pragma unroll
  for (int i = 0; i < kMT; ++i)
#pragma unroll
    for (int j = 0; j < kB; ++j) sums[((i * kB + j) * kWaves + wave) * 64 + lane] = acc[i][j];
  __syncthreads();
  for (int b = wave; b < kMT * kNT; b += kWaves) {
    const int i = b / kNT, j = b % kNT;
    v4f s[kG];
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      const v4f* p = sums + (i * kB + g * kNT + j) * kWaves * 64 + lane;
      s[g] = p[0];
#pragma unroll
      for (int v = 1; v < kWaves; ++v) s[g] += p[v * 64];
    }
    const int64_t row = 16 * i + frow, col = col0 + 16 * j + 4 * quarter;
    if (part)
      put_parts<kGated>(E, part + split * E.m * E.n * kG, row, col, s[0], s[kG - 1]);
    else
      put4<kGated>(E, row, col, s[0], s[kG - 1]);
  }
}

// ------------------------------------------------------------------ tiles
// Tiles as the int8 layer's (tile_walk.h), a K step being 128 bytes of each line, 256 codes.  Lane
// quarter q of a fragment takes chunks 2 q and 2 q + 1 of a line's step, so that its two scales
// are one aligned word of 16 bits.  Scales come in groups of four steps, 32 bytes a line, in a
// ring of kBufs groups behind the codes': 8 bytes of every line each step are as many requests to
// L2 again as the codes are (8192^3: 271 us so, 260 with groups and with K steps of one basic
// block).
// Gated: a wave's columns are half columns of the gate's projection and half the same columns of
// the other, so that both meet in one wave; the tile has BN / 2 columns of C.
template <typename TL, bool kGated, int kBufs>
struct MxTile {
  static constexpr int kCols = kGated ? TL::BN / 2 : TL::BN;     // of C, a tile's
  static constexpr int kWaveCols = kGated ? TL::WN / 2 : TL::WN; // and a wave's
  static constexpr int kScaleBufs = kBufs;
  static constexpr int kScaleBuf = (TL::BM + TL::BN) * 32;
  // loads of 32 lines' scales a wave and group; waves without lines of their own repeat others'
  static constexpr int kScaleLoads = (kScaleBuf / 1024 + TL::NW - 1) / TL::NW;
  static constexpr int kBytes = TL::S * TL::kStage + kBufs * kScaleBuf;
  static_assert(kScaleBuf % 1024 == 0 && kBytes <= 160 * 1024, "LDS");
  static_assert(kWaveCols % 8 == 0, "a load's lines are of one projection");
};

template <typename T, typename TL, bool kGated>
struct MxWalk {
  static constexpr int BM = TL::BM, BN = TL::BN, NW = TL::NW, S = TL::S, LC = TL::kLoads;
  static constexpr int LS = T::kScaleLoads;
  int8_t* lds;
  int wave, lane;
  int nk;                  // K steps
  int last;   // the lines' last step, from this workgroup's first, if it is the 1st, 3rd, ...
  int64_t row0, col0;      // of C
  uint64_t base[LC];       // of a load's lines (uniform)
  uint32_t voff[LC];       // a lane's offset from there
  const uint8_t* scale[LS];
  int scale_left;          // bytes of a line's scales from the lane's first on
  uint32_t wave_lds, scale_lds[LS];

  // Tile `tile` of tiles_m x tiles_n in groups of group_m tile rows (column, then row in group), K
  // steps first .. first + count - 1 of `steps`.
  __device__ __forceinline__ MxWalk(int8_t* ring, int64_t m, int64_t n, const Lines& X,
                                    const Lines& W, int tile, int tiles_m, int tiles_n,
                                    int group_m, int first, int count, int steps)
      : lds(ring), nk(count), last((steps - first) % 2 && steps > 1 ? steps - 1 - first : -1) {
    lane = threadIdx.x & 63;
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int per_group = group_m * tiles_n, first_m = tile / per_group * group_m;
    const int gsize = tiles_m - first_m < group_m ? tiles_m - first_m : group_m;
    const int in_group = tile % per_group;
    row0 = (int64_t)(first_m + in_group % gsize) * BM;
    col0 = (int64_t)(in_group / gsize) * T::kCols;
    // Load q of this wave: region rg = wave + NW q, lines 8 rg .. 8 rg + 7 of X's, then of W's;
    // lane i takes line i / 8 of it, physical chunk i % 8, which holds logical chunk (i % 8) ^
    // swizzle(line), which depends on the region's parity alone, the wave's.  Lines past the
    // matrix re-read its last.
    const uint32_t chunk = 16 * ((lane & 7) ^ swizzle(8 * wave + (lane >> 3)));
#pragma unroll
    for (int q = 0; q < LC; ++q) {
      const int rg = wave + NW * q, r = 8 * rg;
      const bool is_w = r >= BM;
      const int wr = r - BM, half = kGated && is_w ? wr % TL::WN / T::kWaveCols : 0;
      const int at = !is_w ? r : (kGated ? wr / TL::WN * T::kWaveCols + wr % T::kWaveCols : wr);
      const int64_t origin = is_w ? col0 : row0, end = (is_w ? n : m) - 1 - origin;
      const int64_t ld = is_w ? W.ld : X.ld;
      base[q] = (uint64_t)((is_w ? W.codes + half * (n * ld) : X.codes) + origin * ld +
                           (int64_t)first * 128);
      const int mine = at + (lane >> 3);
      voff[q] = (uint32_t)((mine < end ? mine : end) * ld) + chunk;
    }
    // Scales: 32 bytes of a line, four steps, by two lanes.
#pragma unroll
    for (int q = 0; q < LS; ++q) {
      const int rg = (wave + NW * q) % ((BM + BN) / 32);
      const int r = 32 * rg + (lane >> 1), wr = r - BM;
      const bool is_w = r >= BM;
      const int half = kGated && is_w ? wr % TL::WN / T::kWaveCols : 0;
      const int at = !is_w ? r : (kGated ? wr / TL::WN * T::kWaveCols + wr % T::kWaveCols : wr);
      const int64_t g = (is_w ? col0 : row0) + at, end = (is_w ? n : m) - 1;
      const int64_t l = (g < end ? g : end) + half * n;
      scale[q] = (is_w ? W.scales + l * W.lds : X.scales + l * X.lds) + (int64_t)first * 8;
      scale_lds[q] = __builtin_amdgcn_readfirstlane(lds_address(lds) + S * TL::kStage + rg * 1024);
    }
    scale_left = (steps - first) * 8;
    wave_lds = __builtin_amdgcn_readfirstlane(lds_address(lds) + wave * 1024);
  }

  __device__ __forceinline__ const int8_t* stage(int t) const {
    return lds + (t % S) * TL::kStage;
  }
  // Line 0's 8 scales of step t (a line's group is 32 bytes).
  __device__ __forceinline__ const uint8_t* scales(int t) const {
    return reinterpret_cast<const uint8_t*>(lds) + S * TL::kStage +
           (t / 4 % T::kScaleBufs) * T::kScaleBuf + t % 4 * 8 + (t == last ? 8 : 0);
  }

  // Load q of step t's codes if `more`.
  __device__ __forceinline__ void load(uint32_t more, int t, int q) const {
    dma16_sbase_if(more, voff[q], base[q] + (uint64_t)t * 128,
                   wave_lds + (uint32_t)(t % S) * TL::kStage + q * (NW * 1024));
  }
  // Load q of the scales of steps 4 g .. 4 g + 3 if `more`.  A lane whose 16 bytes would leave its
  // line takes the line's last 16: a last step that is the 1st, 3rd, ... lies 8 bytes on (`last`).
  __device__ __forceinline__ void load_scales(uint32_t more, int g, int q) const {
    const uint32_t to = scale_lds[q] + (uint32_t)(g % T::kScaleBufs) * T::kScaleBuf;
    const int at = 32 * g + 16 * (lane & 1), most = scale_left - 16;
    dma16_if(more, scale[q] + (at < most ? at : most), to);
  }

  // Behind the barrier of step t, in which the scales of group t / 4 - 1 have been read for the
  // last time where t begins a group: whether that asks for another, and which.
  __device__ __forceinline__ int next_group(int t) const { return t / 4 + T::kScaleBufs - 1; }
  __device__ __forceinline__ bool asks(int t) const {
    return t % 4 == 0 && 4 * next_group(t) < nk;
  }

  // Waits until of this wave's loads of codes at most those of the youngest `younger` steps are
  // under way (kMost: the number that is asked for on every step but the last ones), and of scales
  // at most those asked for within these steps.
  template <int kMost>
  __device__ __forceinline__ void wait_loads(int younger) const {
    constexpr int L = LC;
    if (kMost == 0 || younger >= kMost) {
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(L * kMost) : "memory");
      return;
    }
    if (kMost > 3 && younger == 3) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(L * 3) : "memory");
    else if (kMost > 2 && younger == 2) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(L * 2) : "memory");
    else if (kMost > 1 && younger == 1) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(L) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  }

  // The ring's first stages asked for, scales first, step 0 in place for every wave.
  __device__ __forceinline__ void begin() const {
    // group G is asked for at step 4 (G - kBufs + 1) and read from behind the barrier of step
    // 4 G - 1 on: 4 kBufs - 6 steps' codes later, of which S - 2 may still be under way
    static_assert(4 * T::kScaleBufs - 6 >= S - 2, "a group's scales have landed");
    if (scale_left == 8 && last < 0) {   // lines of one step: their 8 scales, no loads of 16 bytes
      for (int q = 0; q < LS; ++q) {
        const int rg = (wave + NW * q) % ((BM + BN) / 32);
        if ((lane & 1) == 0)
          *reinterpret_cast<uint2*>(lds + S * TL::kStage + rg * 1024 + 16 * lane) =
              *reinterpret_cast<const uint2*>(scale[q]);
      }
    } else {
#pragma unroll
      for (int g = 0; g < T::kScaleBufs - 1; ++g)
#pragma unroll
        for (int q = 0; q < LS; ++q) load_scales(4 * g < nk, g, q);
    }
#pragma unroll
    for (int t = 0; t < S; ++t)
#pragma unroll
      for (int q = 0; q < LC; ++q) load(t < nk, t, q);
    wait_loads<S - 1>(nk - 1);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    wg_barrier();
  }
};

// A workgroup's tile and split of K in the order (split, tile).
struct Place {
  int split, tile, t0, nk;
  __device__ __forceinline__ Place(int steps, int tiles, int splits) {
    const int id = xcd_order();
    split = id / tiles;
    tile = id - split * tiles;
    t0 = (int)((int64_t)steps * split / splits);
    nk = (int)((int64_t)steps * (split + 1) / splits) - t0;
  }
};

// The outputs of a wave's NI x TJ blocks (lane l of block (i, j): row 16 i + l % 16, columns 16 j
// + 4 (l / 16) .. + 3), or their partial sums.  A phase of the blocks is staged through this
// wave's part `mine` of the ring so that a few lanes finish one row of the wave's columns, eight
// consecutive outputs each; a phase's groups of rows are finished together, for their
// instructions' latencies, and the next phase's residuals asked for meanwhile.  The phases are a
// loop, through which the blocks move down: written out they would not fit the instruction cache.
// A residual is read once and marked so (4096 x 16384 x 4096, gelu, bf16, cold, and with a reader of
// the outputs behind: 231 -> 217 us and 280 -> 266, rows at odd elements 207 -> 199 and 260 -> 252;
// fp32 325 -> 297 and 404 -> 389).  Outputs are marked as not to be read soon behind a gate, where a
// wave's rows are half lines of memory, if they have 16 bits and rows at multiples of 16 bytes:
// 8192 x 2 4096 x 1024, bf16, silu 57.5 us so, else 61.9, with the quantiser behind 82.5 and 87 cold;
// 4096 x 2 8192 x 4096 140 and 143, 172 and 178.  Rows at odd elements 147 marked and 140 not,
// fp32 outputs 169 and 149 (cold 192 and 158); without a gate the two are the same.
template <typename TL, bool kGated, typename O, int NI>
__device__ __forceinline__ void put_tile(const MxEpilogue<O>& E, v4f (&acc)[NI][TL::TJ],
                                         int64_t wrow0, int64_t wcol0, int lane, float* mine,
                                         float* __restrict__ part) {
  constexpr int kWaveCols = kGated ? TL::WN / 2 : TL::WN;
  constexpr int TJ = TL::TJ, kPairs = kGated ? TJ / 2 : TJ;
  const int frow = lane & 15, quarter = lane >> 4;
  if (part) {
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int j = 0; j < kPairs; ++j)
        put_parts<kGated>(E, part, wrow0 + 16 * i + frow, wcol0 + 16 * j + 4 * quarter, acc[i][j],
                          acc[i][(j + kPairs) % TJ]);
    return;
  }
  typedef O V8 __attribute__((ext_vector_type(8), aligned(sizeof(O))));
  constexpr int kLanes = kWaveCols / 8, kRows = 64 / kLanes;   // lanes of a row, rows at once
  constexpr int kIters = TL::kPhase * 16 / kRows, kPhases = NI / TL::kPhase;
  static_assert(kIters >= 1 && kIters * kRows == TL::kPhase * 16, "whole groups of rows");
  const int lrow = lane / kLanes, lcol = 8 * (lane % kLanes);
  const int64_t col = wcol0 + lcol;
  const bool whole = col + 8 <= E.n;
  const bool marked = kGated && sizeof(O) == 2 &&
                      (reinterpret_cast<uintptr_t>(E.c) | (uintptr_t)E.ldc * sizeof(O)) % 16 == 0;
  // every row and column of the wave's is C's (the usual case): no checks
  const bool inside = wrow0 + 16 * NI <= E.m && wcol0 + kWaveCols <= E.n;
  const float* const from = mine + lrow * TL::kPitch + lcol;
  float b[8], bu[8];
#pragma unroll
  for (int u = 0; u < 8; ++u) b[u] = bu[u] = 0.0f;
  if (whole && E.bias) {
    const V8 bv = *reinterpret_cast<const V8*>(E.bias + col);
#pragma unroll
    for (int u = 0; u < 8; ++u) b[u] = (float)bv[u];
    if constexpr (kGated) {
      const V8 uv = *reinterpret_cast<const V8*>(E.bias + E.n + col);
#pragma unroll
      for (int u = 0; u < 8; ++u) bu[u] = (float)uv[u];
    }
  }
  V8 res[kIters];
  auto ask = [&](int64_t row0) {
    if (kGated || !E.residual || !inside) return;
#pragma unroll
    for (int it = 0; it < kIters; ++it)
      res[it] = __builtin_nontemporal_load(
          reinterpret_cast<const V8*>(E.residual + (row0 + it * kRows + lrow) * E.ldr + col));
  };
  ask(wrow0);
#pragma unroll 1
  for (int ph = 0; ph < kPhases; ++ph) {
    const int64_t row0 = wrow0 + ph * (TL::kPhase * 16);
#pragma unroll
    for (int i = 0; i < TL::kPhase; ++i)
#pragma unroll
      for (int j = 0; j < TJ; ++j)
        *reinterpret_cast<v4f*>(mine + (16 * i + frow) * TL::kPitch + 16 * j + 4 * quarter) =
            acc[i][j];
#pragma unroll
    for (int i = 0; i + TL::kPhase < NI; ++i)
#pragma unroll
      for (int j = 0; j < TJ; ++j) acc[i][j] = acc[i + TL::kPhase][j];
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (inside) {
      float z[kIters * 8], up[kGated ? kIters * 8 : 1];
#pragma unroll
      for (int it = 0; it < kIters; ++it)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float* p = from + it * kRows * TL::kPitch + 4 * h;
          const v4f v = *reinterpret_cast<const v4f*>(p);
#pragma unroll
          for (int u = 0; u < 4; ++u) z[8 * it + 4 * h + u] = v[u] + b[4 * h + u];
          if constexpr (kGated) {
            const v4f w = *reinterpret_cast<const v4f*>(p + kWaveCols);
#pragma unroll
            for (int u = 0; u < 4; ++u) up[8 * it + 4 * h + u] = w[u] + bu[4 * h + u];
          }
        }
      activate_all<sizeof(O) == 4>(z, E.act);
      if (!kGated && E.residual)
#pragma unroll
        for (int u = 0; u < kIters * 8; ++u) z[u] += (float)res[u / 8][u % 8];
      if (ph + 1 < kPhases) ask(row0 + TL::kPhase * 16);
      V8 o[kIters];
#pragma unroll
      for (int it = 0; it < kIters; ++it)
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          float y = z[8 * it + u];
          if constexpr (kGated) y *= up[8 * it + u];
          o[it][u] = (O)y;
        }
      const auto to = [&](int it) {
        return reinterpret_cast<V8*>(E.c + (row0 + it * kRows + lrow) * E.ldc + col);
      };
      if (marked) {
        asm volatile("");   // without these the compiler makes unmarked stores of both branches
#pragma unroll
        for (int it = 0; it < kIters; ++it) __builtin_nontemporal_store(o[it], to(it));
        asm volatile("");
      } else {
#pragma unroll
        for (int it = 0; it < kIters; ++it) *to(it) = o[it];
      }
    } else {
#pragma unroll 1
      for (int it = 0; it < kIters; ++it) {
        const int64_t row = row0 + it * kRows + lrow;
        const float* p = from + it * kRows * TL::kPitch;
        if (row >= E.m || col >= E.n) continue;
        if (!whole) {
          put_ragged<kGated>(E, row, col, p, kWaveCols);
          continue;
        }
        float z[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) z[u] = p[u] + b[u];
        activate_all<sizeof(O) == 4>(z, E.act);
        V8 o, r;
        if (!kGated && E.residual)
          r = *reinterpret_cast<const V8*>(E.residual + row * E.ldr + col);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          if constexpr (kGated) z[u] *= p[kWaveCols + u] + bu[u];
          else if (E.residual) z[u] += (float)r[u];
          o[u] = (O)z[u];
        }
        *reinterpret_cast<V8*>(E.c + row * E.ldc + col) = o;
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
}

// The large tile: per step every wave runs quarters of 2 x TJ blocks; before the last one it waits
// for its loads of step t + 1 and for its reads of step t (the last quarter's operands are in
// registers by then), so one barrier a step makes step t + 1 complete and step t's stage free
// for step t + S, whose loads have S - 1 steps to land less a quarter.
//
// 4096^2 x 32768 takes 224 to 230 us: the matrix instructions alone 164, the loads alone 147,
// everything but the loads 203.  The clock falls to 1.8 GHz under it.  Two workgroups a compute
// unit with tiles of 256 x 128, whose epilogues could overlap, took 338.
template <typename O, bool kGated, typename TL>
__global__ __launch_bounds__(64 * TL::NW) void mxfp4_tile_kernel(int steps, Lines X, Lines W,
                                                                 MxEpilogue<O> E, int tiles_m,
                                                                 int tiles_n, int splits,
                                                                 int group_m,
                                                                 float* __restrict__ part) {
  using T = MxTile<TL, kGated, 2>;
  constexpr int BM = TL::BM, TI = TL::TI, TJ = TL::TJ, S = TL::S, L = TL::kLoads;
  static_assert(TL::KG == 1, "one wave for both K halves");
  __shared__ __attribute__((aligned(1024))) int8_t lds[T::kBytes];
  const Place p(steps, tiles_m * tiles_n, splits);
  const MxWalk<T, TL, kGated> K(lds, E.m, E.n, X, W, p.tile, tiles_m, tiles_n, group_m, p.t0, p.nk,
                                steps);
  const int wr = K.wave / TL::WC, wc = K.wave % TL::WC, nk = K.nk;

  v4f acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = v4f{0, 0, 0, 0};

  const int frow = K.lane & 15, quarter = K.lane >> 4, sw = swizzle(frow);
  const int off0 = ((2 * quarter) ^ sw) << 4, off1 = ((2 * quarter + 1) ^ sw) << 4;
  const int aline = wr * TL::WM + frow, bline = BM + wc * TL::WN + frow;
  v4i fa[2][2][2], fb[2][TJ];   // fa[set][K half][row block of a quarter], fb[K half][block]
  int sa[2][2], sb[TJ];         // scales of both K halves
  auto two_scales = [&](int t, int line) -> int {
    return *reinterpret_cast<const uint16_t*>(K.scales(t) + line * 32 + 2 * quarter);
  };
  auto read_a = [&](int set, int t, int kh, int rb, int ii) {
    fa[set][kh][ii] = *reinterpret_cast<const v4i*>(K.stage(t) + (aline + 16 * rb) * kStepK +
                                                    (kh ? off1 : off0));
    if (kh == 0) sa[set][ii] = two_scales(t, aline + 16 * rb);
  };
  auto read_b = [&](int t, int kh, int j) {
    fb[kh][j] = *reinterpret_cast<const v4i*>(K.stage(t) + (bline + 16 * j) * kStepK +
                                              (kh ? off1 : off0));
  };
  auto read_sb = [&](int t, int j) { sb[j] = two_scales(t, bline + 16 * j); };
  // Quarter q (row blocks 2q and 2q + 1): MFMA idx is row block 2q + idx / (2 TJ), column block
  // (idx / 2) % TJ, K half idx % 2, a block's two halves back to back.  Its first four MFMAs
  // are followed by the reads of the next quarter's A fragments into the other set (the last
  // quarter's: row blocks 0 and 1 of step `next`); the last quarter also replaces each B
  // fragment after its last use and issues the loads of step t + S, if there is one (more), and of
  // scales (asks).
  constexpr int NQ = TI / 2, kQuarter = 4 * TJ;
  static_assert(NQ % 2 == 0 && L <= kQuarter, "sets alternate; loads fit a quarter");
  auto quarter_of = [&](int q, int t, int next, uint32_t more, uint32_t asks) {
    const int as = q & 1;
    const bool is_last = q == NQ - 1;
#pragma unroll
    for (int idx = 0; idx < kQuarter; ++idx) {
      const int ii = idx / (2 * TJ), j = (idx >> 1) % TJ, kh = idx & 1;
      v4f& a = acc[2 * q + ii][j];
      a = kh ? mfma_mx<1>(fb[1][j], sb[j], fa[as][1][ii], sa[as][ii], a)
             : mfma_mx<0>(fb[0][j], sb[j], fa[as][0][ii], sa[as][ii], a);
      if (idx < 4) {
        if (!is_last) read_a(as ^ 1, t, idx & 1, 2 * (q + 1) + (idx >> 1), idx >> 1);
        else read_a(as ^ 1, next, idx & 1, idx >> 1, idx >> 1);
      }
      if (is_last && ii == 1) {
        read_b(next, kh, j);
        if (kh) read_sb(next, j);
      }
      if (is_last && (idx * L) / kQuarter != ((idx + 1) * L) / kQuarter)
        K.load(more, t + S, (idx * L) / kQuarter);
      if (is_last && idx >= kQuarter - T::kScaleLoads)
        K.load_scales(asks, K.next_group(t), idx - (kQuarter - T::kScaleLoads));
      __builtin_amdgcn_sched_barrier(0);
      // the wave that reaches the second half of a quarter first is preferred, so the two
      // waves of a SIMD run apart
      if (idx == kQuarter / 2 - 1) __builtin_amdgcn_s_setprio(1);
    }
    __builtin_amdgcn_s_setprio(0);
  };

  K.begin();
#pragma unroll
  for (int idx = 0; idx < 4; ++idx) read_a(0, 0, idx & 1, idx >> 1, idx >> 1);
#pragma unroll
  for (int j = 0; j < TJ; ++j) {
    read_b(0, 0, j);
    read_b(0, 1, j);
    read_sb(0, j);
  }
  for (int t = 0; t < nk; ++t) {
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int q = 0; q < NQ - 1; ++q) quarter_of(q, t, t, 0, 0);
    // this wave's loads of step t + 1 have landed and it has read all of step t; past the
    // barrier that holds for every wave
    K.template wait_loads<S - 2>(nk - 2 - t);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    wg_barrier();
    __builtin_amdgcn_sched_barrier(0);
    // after the last step: a harmless re-read of it
    quarter_of(NQ - 1, t, t + 1 < nk ? t + 1 : t, t + S < nk, K.asks(t));
  }
  wg_barrier();   // every wave is past its last read of the ring
  put_tile<TL, kGated, O, TI>(
      E, acc, K.row0 + wr * TL::WM, K.col0 + wc * T::kWaveCols, K.lane,
      reinterpret_cast<float*>(lds) + K.wave * (TL::kPhase * 16 * TL::kPitch),
      part ? part + (int64_t)p.split * E.m * E.n * (kGated ? 2 : 1) : nullptr);
}

// The smaller tiles, whose K steps take a fraction of a load's latency: as many stages as LDS
// holds, and per step one barrier, one set of fragment reads and one run of MFMAs.  A pair of
// waves shares the outputs of a wave and splits each step's K, a block of every two; the sums of
// both meet in LDS at the end.  Behind the barrier of step t the wave reads step t + 1 and asks
// for step t + S while step t's MFMAs run from registers.  (The waits, barriers and the exchange of
// halves are small_product's in tile_walk.h, with scales beside the codes: a fault in one is to be
// looked for in the other.)
template <typename O, bool kGated, typename TL, int kBufs>
__global__ __launch_bounds__(64 * TL::NW) void mxfp4_small_kernel(int steps, Lines X, Lines W,
                                                                  MxEpilogue<O> E, int tiles_m,
                                                                  int tiles_n, int splits,
                                                                  int group_m,
                                                                  float* __restrict__ part) {
  using T = MxTile<TL, kGated, kBufs>;
  constexpr int BM = TL::BM, TI = TL::TI, TJ = TL::TJ, S = TL::S, L = TL::kLoads, H = TI / 2;
  constexpr int LS = T::kScaleLoads;
  static_assert(TL::KG == 2 && TI % 2 == 0 && L + LS <= TI * TJ, "pairs of waves");
  static_assert(TL::NW * H * TJ * 1024 <= S * TL::kStage, "halves fit the ring");
  __shared__ __attribute__((aligned(1024))) int8_t lds[T::kBytes];
  const Place p(steps, tiles_m * tiles_n, splits);
  const MxWalk<T, TL, kGated> K(lds, E.m, E.n, X, W, p.tile, tiles_m, tiles_n, group_m, p.t0, p.nk,
                                steps);
  const int kh = K.wave / (TL::WR * TL::WC), wt = K.wave % (TL::WR * TL::WC);
  const int wr = wt / TL::WC, wc = wt % TL::WC, nk = K.nk;

  v4f acc[TI][TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = v4f{0, 0, 0, 0};

  const int frow = K.lane & 15, quarter = K.lane >> 4, sw = swizzle(frow);
  const int off = ((2 * quarter + kh) ^ sw) << 4, soff = 2 * quarter + kh;
  const int aline = wr * TL::WM + frow, bline = BM + wc * TL::WN + frow;
  v4i fa[2][TI], fb[2][TJ];
  int sa[2][TI], sb[2][TJ];
  auto read = [&](int set, int t) {
    const int8_t* st = K.stage(t) + off;
    const uint8_t* sc = K.scales(t) + soff;
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      fb[set][j] = *reinterpret_cast<const v4i*>(st + (bline + 16 * j) * kStepK);
      sb[set][j] = sc[(bline + 16 * j) * 32];
    }
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      fa[set][i] = *reinterpret_cast<const v4i*>(st + (aline + 16 * i) * kStepK);
      sa[set][i] = sc[(aline + 16 * i) * 32];
    }
  };
  auto step = [&](int set, int t) {
    K.template wait_loads<S - 2>(nk - 2 - t);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    wg_barrier();
    __builtin_amdgcn_sched_barrier(0);
    read(set ^ 1, t + 1 < nk ? t + 1 : t);   // after the last step: a harmless re-read
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int idx = 0; idx < TI * TJ; ++idx) {
      const int i = idx / TJ, j = idx % TJ;
      acc[i][j] = mfma_mx<0>(fb[set][j], sb[set][j], fa[set][i], sa[set][i], acc[i][j]);
      if (idx < L) K.load(t + S < nk, t + S, idx);
      else if (idx < L + LS) K.load_scales(K.asks(t), K.next_group(t), idx - L);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  K.begin();
  read(0, 0);
  int t = 0;
  for (; t + 1 < nk; t += 2) {
    step(0, t);
    step(1, t + 1);
  }
  if (t < nk) step(0, t);

  // Wave kh of a pair finishes row blocks kh TI / 2 ..: the other half goes to its partner.
  wg_barrier();   // every wave is past its last read of the ring
  v4f own[H][TJ];
  v4f* boxes = reinterpret_cast<v4f*>(lds);   // [wave][H][TJ][lane]
#pragma unroll
  for (int i = 0; i < H; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) {
      boxes[((K.wave * H + i) * TJ + j) * 64 + K.lane] = kh ? acc[i][j] : acc[H + i][j];
      own[i][j] = kh ? acc[H + i][j] : acc[i][j];
    }
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  wg_barrier();
  const int partner = wt + (kh ? 0 : TL::WR * TL::WC);
#pragma unroll
  for (int i = 0; i < H; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) own[i][j] += boxes[((partner * H + i) * TJ + j) * 64 + K.lane];
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  wg_barrier();
  put_tile<TL, kGated, O, H>(
      E, own, K.row0 + wr * TL::WM + kh * 16 * H, K.col0 + wc * T::kWaveCols, K.lane,
      reinterpret_cast<float*>(lds) + K.wave * (TL::kPhase * 16 * TL::kPitch),
      part ? part + (int64_t)p.split * E.m * E.n * (kGated ? 2 : 1) : nullptr);
}

// The outputs of a product whose K was split: the partial sums added, then the epilogue.
template <typename O, bool kGated>
__global__ __launch_bounds__(256) void mxfp4_join_kernel(MxEpilogue<O> E, int splits,
                                                         const float* __restrict__ part) {
  constexpr int kG = kGated ? 2 : 1;
  const int64_t quads = (E.n + 3) / 4;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= E.m * quads) return;
  const int64_t row = id / quads, col = id % quads * 4;
  v4f s[kG];
#pragma unroll
  for (int g = 0; g < kG; ++g) {
    s[g] = v4f{0, 0, 0, 0};
    const float* p = part + row * (kG * E.n) + g * E.n + col;
    const int64_t apart = E.m * E.n * kG;
    if (col + 4 <= E.n) {
      int k = 0;
      for (; k + 4 <= splits; k += 4, p += 4 * apart) {   // four asked for at once
        v4f v[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) v[u] = *reinterpret_cast<const v4f_words*>(p + u * apart);
#pragma unroll
        for (int u = 0; u < 4; ++u) s[g] += v[u];
      }
      for (; k < splits; ++k, p += apart) s[g] += *reinterpret_cast<const v4f_words*>(p);
    } else {
      for (int k = 0; k < splits; ++k, p += apart)
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (col + u < E.n) s[g][u] += p[u];
    }
  }
  put4<kGated>(E, row, col, s[0], s[kG - 1]);
}

typedef Tile<256, 256, 2, 4, 1, 2> MxLarge;
typedef Tile<128, 128, 2, 2, 2, 4> MxMid;
typedef Tile<64, 128, 1, 4, 2, 5> MxSmall;

// How a product is run: by the kernel for few rows (a workgroup takes all rows) or by tiles of
// one shape; K is split over `splits` workgroups where there are fewer tiles than the compute
// units take.
enum Shape { kStream, kSmall, kMid, kLarge };
struct Plan {
  Shape shape;
  int64_t tiles_m, tiles_n;
  int splits;
};

// Up to 64 rows: the stream kernel (32 and 64 rows of 8192 x 8192: 8.5 and 11.6 us, by tiles of
// 64 rows 15.1 and 16.4; of 4096 x 4096: 4.5 and 5.8 against 10.9 and 12.3).  More rows: the tile
// shape and split of the least estimated time, in microseconds, of rounds of 256 workgroups that
// each cost `fixed` and `step` per K step.  Measured, one round of 256 and of 4096 K values:
// small 5.5 and 13.5, mid 7.9 and 19.6, large 10.4 and 36.3.  A split costs the launch of the
// join (4) and the partial sums' way out and back (128 x 4096 x 4096, small, in 1, 2, 4 and 8:
// 13.5, 14.1, 14.7, 20.6; 100 x 1024 x 8192: 21.8, 16.3, 12.3, 11.4).
Plan plan_of(int64_t m, int64_t n, int64_t k, bool gated) {
  const int64_t steps = (k + 255) / 256, wide = gated ? 2 * n : n;
  if (m <= 64) {
    // 16 columns a workgroup, or 32 where that is more than the compute units take at once (16
    // rows of 8192 x 8192: 7.0 us with 32, 9.4 with 16; of 4096 x 4096: 4.4 and 3.9)
    const int64_t bn = (n + 15) / 16 > (m <= 8 && !gated ? 512 : 256) ? 32 : 16;
    Plan p{kStream, bn / 16, (n + bn - 1) / bn, 1};
    // a workgroup's eight waves take four steps each at least
    const int64_t s = 256 / p.tiles_n, most = steps / 32;
    p.splits = (int)(s < most ? s : most);
    if (p.splits < 1) p.splits = 1;
    return p;
  }
  struct Cost {
    Shape shape;
    int64_t bm, bn;
    double fixed, step;
  };
  const Cost costs[] = {{kSmall, 64, 128, 5.0, 0.53}, {kMid, 128, 128, 7.2, 0.71},
                        {kLarge, 256, 256, 9.5, 1.75}};
  Plan best{};
  double least = 0;
  for (const Cost& c : costs) {
    const int64_t tm = (m + c.bm - 1) / c.bm, tn = (wide + c.bn - 1) / c.bn, tiles = tm * tn;
    for (int64_t sp = 1; sp <= 16 && (sp == 1 || (tiles * sp <= 256 && steps / sp >= 4)); ++sp) {
      const double rounds = (double)((tiles * sp + 255) / 256);
      double t = rounds * (c.fixed + c.step * (double)((steps + sp - 1) / sp));
      if (sp > 1) t += 4.0 + (double)sp * (double)m * (double)wide * 4.0 / 3.5e6;
      if (least == 0 || t < least) {
        least = t;
        best = {c.shape, tm, tn, (int)sp};
      }
    }
  }
  return best;
}

template <typename O, bool kGated, typename TL>
void launch_tiles(const Plan& p, int steps, const Lines& X, const Lines& W, const MxEpilogue<O>& E,
                  float* part, hipStream_t s) {
  const int group_m = 8;
  const dim3 grid((unsigned)(p.tiles_m * p.tiles_n * p.splits)), block(64 * TL::NW);
  if constexpr (TL::KG == 1)
    hipLaunchKernelGGL((mxfp4_tile_kernel<O, kGated, TL>), grid, block, 0, s, steps, X, W, E,
                       (int)p.tiles_m, (int)p.tiles_n, p.splits, group_m, part);
  else
    hipLaunchKernelGGL((mxfp4_small_kernel<O, kGated, TL, TL::S <= 4 ? 2 : 3>), grid, block, 0, s,
                       steps, X, W, E, (int)p.tiles_m, (int)p.tiles_n, p.splits, group_m, part);
}

template <typename O, bool kGated>
int linear_t(int64_t m, int64_t n, int64_t k, const Lines& X, const Lines& W, const void* bias,
             int act, const void* residual, int64_t ldr, void* c, int64_t ldc, void* workspace,
             hipStream_t s) {
  const MxEpilogue<O> E{m, n, (const O*)bias, (const O*)residual, ldr, (O*)c, ldc, act};
  const int steps = (int)((k + 255) / 256);
  const Plan p = plan_of(m, n, k, kGated);
  // a launch takes fewer than 2^32 threads, 512 a workgroup
  if (p.tiles_m * p.tiles_n * p.splits >= 1 << 23) return OZK_EUNSUPPORTED;
  float* const part = p.splits > 1 ? static_cast<float*>(workspace) : nullptr;
  if (p.shape == kStream) {
    const dim3 grid((unsigned)(p.tiles_n * p.splits)), block(512);
#define OZK_STREAM(XR, NT, S)                                                              \
  hipLaunchKernelGGL((mxfp4_stream_kernel<O, kGated, XR, NT, S>), grid, block, 0, s, steps, X, W, \
                     E, p.splits, part)
    const bool two = p.tiles_m == 2;
    if (m <= 8 && two) OZK_STREAM(8, 2, 2);
    else if (m <= 8) OZK_STREAM(8, 1, 3);
    else if (m <= 16 && two) OZK_STREAM(16, 2, kGated ? 1 : 3);
    else if (m <= 16) OZK_STREAM(16, 1, 3);
    else if (m <= 32 && two) OZK_STREAM(32, 2, kGated ? 1 : 2);
    else if (m <= 32) OZK_STREAM(32, 1, 2);
    else if (two) OZK_STREAM(64, 2, 1);
    else OZK_STREAM(64, 1, 1);
#undef OZK_STREAM
  } else if (p.shape == kLarge) {
    launch_tiles<O, kGated, MxLarge>(p, steps, X, W, E, part, s);
  } else if (p.shape == kMid) {
    launch_tiles<O, kGated, MxMid>(p, steps, X, W, E, part, s);
  } else {
    launch_tiles<O, kGated, MxSmall>(p, steps, X, W, E, part, s);
  }
  if (p.splits > 1)
    hipLaunchKernelGGL((mxfp4_join_kernel<O, kGated>),
                       dim3((unsigned)((m * ((n + 3) / 4) + 255) / 256)), dim3(256), 0, s, E,
                       p.splits, part);
  return hipGetLastError() == hipSuccess ? OZK_OK : OZK_EHIP;
}

template <typename O>
int linear_any(int64_t m, int64_t n, int64_t k, const Lines& X, const Lines& W, bool gated,
               const void* bias, int act, const void* residual, int64_t ldr, void* c, int64_t ldc,
               void* workspace, hipStream_t s) {
  return gated ? linear_t<O, true>(m, n, k, X, W, bias, act, residual, ldr, c, ldc, workspace, s)
               : linear_t<O, false>(m, n, k, X, W, bias, act, residual, ldr, c, ldc, workspace, s);
}

}  // namespace

size_t mxfp4_linear_workspace(int64_t m, int64_t n, int64_t k, bool gated) {
  const Plan p = plan_of(m, n, k, gated);
  return p.splits > 1 ? align256((size_t)p.splits * m * n * (gated ? 8 : 4)) : 0;
}

int launch_mxfp4_linear(int64_t m, int64_t n, int64_t k, const uint8_t* x, int64_t ldx,
                        const uint8_t* xs, int64_t ldxs, const uint8_t* w, int64_t ldw,
                        const uint8_t* ws, int64_t ldws, bool gated, const void* bias, int act,
                        const void* residual, int64_t ldr, int type, void* c, int64_t ldc,
                        void* workspace, hipStream_t s) {
  const Lines X{x, ldx, xs, ldxs}, W{w, ldw, ws, ldws};
  switch (type) {
    case OZK_F32:
      return linear_any<float>(m, n, k, X, W, gated, bias, act, residual, ldr, c, ldc, workspace,
                               s);
    case OZK_F16:
      return linear_any<f16_t>(m, n, k, X, W, gated, bias, act, residual, ldr, c, ldc, workspace,
                               s);
    default:
      return linear_any<bf16_t>(m, n, k, X, W, gated, bias, act, residual, ldr, c, ldc, workspace,
                                s);
  }
}

}  // namespace ozk
