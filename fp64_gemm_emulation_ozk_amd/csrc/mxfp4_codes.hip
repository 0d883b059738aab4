// Lines in microscaled 4-bit floating point (OCP MX FP4: e2m1 codes, an e8m0 scale for every 32
// values along K), written from a matrix's rows or columns and read back.
//
// A block's scale is 2^E, E = floor(log2 max |x|) - 2 held to [-127, 127], stored as E + 127: only
// the exponent field of the largest magnitude is needed, which a maximum over the magnitudes' bits
// finds.  A code is RNE(x 2^-E) on {0, 0.5, 1, 1.5, 2, 3, 4, 6}, 6 beyond, which gfx950's
// conversions to FP4 compute with the scale as their operand.
//
// Memory bounds all of them.  From operands in no cache, us: 4096 x 16384 bf16 rows 33.3, columns
// 37.5, values 25.9 (170 MB each, 5.1, 4.5 and 6.6 TB/s); 4099 x 5001 fp32 rows 20.3, columns
// 21.9, values 22.1 (93 MB).  In the last-level cache: 27, 26 and 26; 16.3, 18.1 and 16.2.
#include "ozk_internal.h"
#include "rows.h"

namespace ozk {
namespace {

typedef bf16_t v2bf __attribute__((ext_vector_type(2)));
typedef f16_t v2h __attribute__((ext_vector_type(2)));

constexpr uint32_t kNoScale = 255;   // NaN: a block with Inf or NaN, or past 2^127

// Bits of |x| that compare as the magnitudes do (of a double: the word with its exponent).
__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t magnitude(double x) {
  return (uint32_t)((uint64_t)__double_as_longlong(x) >> 32) & 0x7fffffffu;
}

// The largest magnitude of eight values (of 16 bits: two at a time).
template <typename T>
__device__ __forceinline__ uint32_t largest(const T (&v)[8]) {
  if constexpr (sizeof(T) == 2) {
    typedef uint16_t u2 __attribute__((ext_vector_type(2)));
    u2 most = {0, 0};
#pragma unroll
    for (int u = 0; u < 8; u += 2) {
      const u2 a = u2{__builtin_bit_cast(uint16_t, v[u]), __builtin_bit_cast(uint16_t, v[u + 1])} &
                   (uint16_t)0x7fff;
      most = __builtin_elementwise_max(most, a);
    }
    return most[0] > most[1] ? most[0] : most[1];
  } else {
    uint32_t most = 0;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint32_t a = magnitude(v[u]);
      most = a > most ? a : most;
    }
    return most;
  }
}

// The scale byte of a block from its largest magnitude.  A subnormal fp32 maximum has E below
// -127 in any case; a subnormal fp16 one is a normal fp32 value.
template <typename T>
__device__ __forceinline__ uint32_t scale_of(uint32_t most) {
  if constexpr (sizeof(T) == 8) {
    const int e = (int)(most >> 20) - 898;   // 1023 + 2 - 127
    return e < 0 ? 0u : (e > 254 ? kNoScale : (uint32_t)e);
  } else {
    uint32_t field;
    if constexpr (__is_same(T, f16_t))
      field = __float_as_uint((float)__builtin_bit_cast(f16_t, (uint16_t)most)) >> 23;
    else
      field = most >> (sizeof(T) == 4 ? 23 : 7);
    return field == 255 ? kNoScale : (field > 2 ? field - 2 : 0u);
  }
}

// What the conversions take as 2^E: a float of that value (2^-127 is a subnormal one).
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __uint_as_float(byte ? byte << 23 : 0x00400000u);
}

// A double as a float that rounds to the same code: |x| 2^(20 - E) cut to an integer below 2^23,
// its last bit set where something was cut off (no code's border lies between), so scale 2^20.
__device__ __forceinline__ float short_of(double x, int e) {
  const double v = __builtin_ldexp(__builtin_fabs(x), 20 - e);
  uint32_t i = (uint32_t)v;
  i |= (double)i != v ? 1u : 0u;
  const float f = (float)i;
  return (uint64_t)__double_as_longlong(x) >> 63 ? -f : f;
}

// Byte kB of `codes` becomes the codes of a (low nibble) and b.
template <int kB, typename T>
__device__ __forceinline__ uint32_t put_pair(uint32_t codes, T a, T b, uint32_t byte) {
  if constexpr (sizeof(T) == 8) {
    const int e = (int)byte - 127;
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, short_of(a, e), short_of(b, e), 0x1p20f,
                                                    kB);
  } else {
    const float s = scale_value(byte);
    if constexpr (sizeof(T) == 4)
      return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(codes, a, b, s, kB);
    else if constexpr (__is_same(T, bf16_t))
      return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(codes, v2bf{a, b}, s, kB);
    else
      return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(codes, v2h{a, b}, s, kB);
  }
}

// Eight codes; those of a block without a scale are 0.
template <typename T>
__device__ __forceinline__ uint32_t put_eight(const T (&v)[8], uint32_t byte) {
  uint32_t c = put_pair<0>(0u, v[0], v[1], byte);
  c = put_pair<1>(c, v[2], v[3], byte);
  c = put_pair<2>(c, v[4], v[5], byte);
  c = put_pair<3>(c, v[6], v[7], byte);
  return byte == kNoScale ? 0u : c;
}

// Eight values as they come from memory.
template <typename T>
struct Eight {
  static constexpr int N = Vec<T>::N;
  typename Vec<T>::type v[8 / N];
  __device__ __forceinline__ void ask(const T* p) {
#pragma unroll
    for (int q = 0; q < 8 / N; ++q)
      v[q] = *reinterpret_cast<const typename Vec<T>::type*>(p + q * N);
  }
  __device__ __forceinline__ void take(T (&out)[8]) const {
#pragma unroll
    for (int u = 0; u < 8; ++u) out[u] = v[u / N][u % N];
  }
};

// A half wave's place: unit u (256 values of a line) of a matrix of `steps` units a line.
struct Unit {
  uint32_t line, step;
  __device__ __forceinline__ Unit(uint32_t u, uint32_t steps)
      : line(u / steps), step(u - line * steps) {}
  __device__ __forceinline__ void two_on(uint32_t steps) {
    step += 2;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (step >= steps) {
        step -= steps;
        ++line;
      }
  }
};

constexpr int kUnits = 8;   // units of a wave, two at a time

// Rows: lane l of a half wave takes values 8 l .. 8 l + 7 of its unit, four lanes a block.  A wave
// takes eight units (4096 x 16384 bf16: 32.8 us cold with all of them asked for first, 36.7 with a
// branch around each load).
template <typename T>
__global__ __launch_bounds__(256) void mxfp4_rows_kernel(uint32_t rows, int64_t cols,
                                                         uint32_t steps, const T* __restrict__ x,
                                                         int64_t ldx, uint8_t* __restrict__ codes,
                                                         int64_t ldq, uint8_t* __restrict__ scales,
                                                         int64_t lds) {
  const int lane = threadIdx.x & 63, sub = lane & 31;
  const uint32_t wave = blockIdx.x * 4 + (threadIdx.x >> 6);
  Unit at(wave * kUnits + (lane >> 5), steps);
  // All units asked for first, without a branch between: lanes that the row does not fill read its
  // first values and put theirs right below.
  Eight<T> raw[kUnits / 2];
  const Unit first = at;
  if (cols >= 8) {
#pragma unroll
    for (int i = 0; i < kUnits / 2; ++i) {
      const int64_t c = (int64_t)at.step * 256 + 8 * sub;
      raw[i].ask(x + (int64_t)(at.line < rows ? at.line : rows - 1) * ldx +
                 (c + 8 <= cols ? c : 0));
      at.two_on(steps);
    }
  }
  at = first;
#pragma unroll
  for (int i = 0; i < kUnits / 2; ++i) {
    const int64_t c = (int64_t)at.step * 256 + 8 * sub;
    T v[8];
    raw[i].take(v);
    if (c + 8 > cols) {
      const T* p = x + (int64_t)(at.line < rows ? at.line : rows - 1) * ldx;
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = c + u < cols ? p[c + u] : (T)0.0f;
    }
    uint32_t most = largest(v);
    uint32_t o = dpp_mov<0xb1>(most);
    most = o > most ? o : most;
    o = dpp_mov<0x4e>(most);
    most = o > most ? o : most;
    const uint32_t byte = scale_of<T>(most);
    if (at.line < rows) {
      *reinterpret_cast<uint32_t*>(codes + (int64_t)at.line * ldq + (int64_t)at.step * 128 +
                                   4 * sub) = put_eight(v, byte);
      if ((sub & 3) == 0)
        scales[(int64_t)at.line * lds + (int64_t)at.step * 8 + (sub >> 2)] = (uint8_t)byte;
    }
    at.two_on(steps);
  }
}

// Columns: a workgroup takes 256 rows x 64 kC columns, wave w its rows 32 w .. 32 w + 31, which
// are one block of each of a lane's kC columns.  The codes meet in LDS, so that a line's 128 bytes
// leave in one store of eight lanes; a line's eight chunks are XORed with the line's number there,
// for the banks.
template <typename T, int kC>
__global__ __launch_bounds__(512) void mxfp4_cols_kernel(int64_t rows, int64_t cols,
                                                         uint32_t tiles,
                                                         const T* __restrict__ x, int64_t ldx,
                                                         uint8_t* __restrict__ codes, int64_t ldq,
                                                         uint8_t* __restrict__ scales,
                                                         int64_t lds) {
  typedef T V __attribute__((ext_vector_type(kC), aligned(sizeof(T))));
  constexpr int kLines = 64 * kC;
  __shared__ uint4 box[kLines * 8];
  __shared__ __attribute__((aligned(8))) uint8_t sbox[kLines][8];   // read as words of 8
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t id = blockIdx.x, step = id / tiles;
  const int64_t col0 = (int64_t)(id - step * tiles) * kLines, row0 = (int64_t)step * 256 + 32 * w;
  const int64_t c = col0 + kC * lane;
  // All rows asked for without a branch between: what lies past the matrix reads its last row or
  // column, and is made zero below (rows) or not stored (columns).  kC <= cols.  Whole blocks have
  // code of their own: 32 clamped row addresses did not fit the scalar registers (4096 x 16384
  // bf16 38.2 us so, else 37.5; 1500 x 2000 fp32 8.4 and 7.8).
  const int64_t from = col0 + kC <= cols ? col0 : cols - kC;   // uniform, as a row's address
  const uint32_t off = (uint32_t)((c + kC <= cols ? c : cols - kC) - from);
  V raw[32];
  if (row0 + 32 <= rows) {   // uniform
    const T* p = x + row0 * ldx + from;
#pragma unroll
    for (int r = 0; r < 32; ++r) raw[r] = *reinterpret_cast<const V*>(p + r * ldx + off);
  } else {
#pragma unroll
    for (int r = 0; r < 32; ++r) {
      const T* p = x + (row0 + r < rows ? row0 + r : rows - 1) * ldx + from;
      raw[r] = *reinterpret_cast<const V*>(p + off);
    }
  }
  T v[kC][32];
#pragma unroll
  for (int r = 0; r < 32; ++r)
#pragma unroll
    for (int u = 0; u < kC; ++u) v[u][r] = raw[r][u];
  if (kC == 2 && c + 1 == cols)   // the last column of an odd number
#pragma unroll
    for (int r = 0; r < 32; ++r) v[0][r] = raw[r][kC - 1];
  if (row0 + 32 > rows)
#pragma unroll
    for (int r = 0; r < 32; ++r)
      if (row0 + r >= rows)
#pragma unroll
        for (int u = 0; u < kC; ++u) v[u][r] = (T)0.0f;
#pragma unroll
  for (int u = 0; u < kC; ++u) {
    uint32_t most = 0;
    T part[4][8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
      for (int r = 0; r < 8; ++r) part[e][r] = v[u][8 * e + r];
      const uint32_t a = largest(part[e]);
      most = a > most ? a : most;
    }
    const uint32_t byte = scale_of<T>(most);
    uint32_t q[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) q[e] = put_eight(part[e], byte);
    const int line = kC * lane + u;
    box[line * 8 + (w ^ (line & 7))] = uint4{q[0], q[1], q[2], q[3]};
    sbox[line][w] = (uint8_t)byte;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kC; ++i) {
    const int line = 64 * i + (threadIdx.x >> 3), slot = threadIdx.x & 7;
    if (col0 + line < cols)
      *reinterpret_cast<uint4*>(codes + (col0 + line) * ldq + (int64_t)step * 128 +
                                16 * (slot ^ (line & 7))) = box[line * 8 + slot];
  }
  if (threadIdx.x < kLines && col0 + threadIdx.x < cols)
    *reinterpret_cast<uint2*>(scales + (col0 + threadIdx.x) * lds + (int64_t)step * 8) =
        *reinterpret_cast<const uint2*>(sbox[threadIdx.x]);
}

// N values of N codes in c's low bits, NaN without a scale.  fp32 holds them but for the largest
// (6 x 2^127 is Inf there), fp64 all of them.
template <int N, typename A>
__device__ __forceinline__ void take_codes(uint32_t c, uint32_t byte, A (&v)[N]) {
  const float s = sizeof(A) == 8 ? 1.0f : scale_value(byte);
  float w[8];
  const auto put = [&](int u, auto pair) {
    w[u] = pair[0];
    w[u + 1] = pair[1];
  };
  put(0, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0));
  if constexpr (N > 2) put(2, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1));
  if constexpr (N > 4) {
    put(4, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 2));
    put(6, __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 3));
  }
#pragma unroll
  for (int u = 0; u < N; ++u) {
    v[u] = byte == kNoScale ? __builtin_nanf("") : w[u];
    if constexpr (sizeof(A) == 8)
      v[u] *= __longlong_as_double((long long)(byte + 896) << 52);   // 2^(byte - 127)
  }
}

// A half wave writes a unit in 8 / N stores of 16 bytes a lane, each whole lines of memory (32
// bytes a lane in two stores of every other 16: 8192^2 to fp32 72 us).  kWhole: rows start at
// multiples of 16 bytes, so that no two stores share a line; then they are marked as not to be
// read soon.  4096 x 16384 to bf16 25.9 us so, else 32.1, and with a reader behind 58.0 and 57.5;
// 8192^2 to fp32 48.5 and 57.4, 102 and 114.  (Rows of 4099 fp32, marked: 25.3, not marked 22.0.)
template <typename T, bool kWhole>
__global__ __launch_bounds__(256) void mxfp4_values_kernel(uint32_t lines, int64_t k,
                                                           uint32_t steps,
                                                           const uint8_t* __restrict__ codes,
                                                           int64_t ldq,
                                                           const uint8_t* __restrict__ scales,
                                                           int64_t lds, T* __restrict__ out,
                                                           int64_t ldo) {
  constexpr int N = Vec<T>::N, kQ = 8 / N;
  typedef T V __attribute__((ext_vector_type(N)));
  typedef typename AccOf<T>::type A;
  const int lane = threadIdx.x & 63, sub = lane & 31;
  const uint32_t wave = blockIdx.x * 4 + (threadIdx.x >> 6);
  Unit at(wave * kUnits + (lane >> 5), steps);
  uint32_t c[kUnits / 2][kQ], s[kUnits / 2][kQ];
  const Unit first = at;
#pragma unroll
  for (int i = 0; i < kUnits / 2; ++i) {
    const uint32_t line = at.line < lines ? at.line : lines - 1;
    const uint8_t* q = codes + (int64_t)line * ldq + (int64_t)at.step * 128;
    const uint8_t* e = scales + (int64_t)line * lds + (int64_t)at.step * 8;
#pragma unroll
    for (int u = 0; u < kQ; ++u) {
      const int h = u * (32 * N) + N * sub;   // within the unit
      if constexpr (N == 8) c[i][u] = *reinterpret_cast<const uint32_t*>(q + h / 2);
      else if constexpr (N == 4) c[i][u] = *reinterpret_cast<const uint16_t*>(q + h / 2);
      else c[i][u] = q[h / 2];
      s[i][u] = e[h / 32];
    }
    at.two_on(steps);
  }
  at = first;
#pragma unroll
  for (int i = 0; i < kUnits / 2; ++i) {
    if (at.line < lines) {
#pragma unroll
      for (int u = 0; u < kQ; ++u) {
        A v[N];
        take_codes<N>(c[i][u], s[i][u], v);
        T* const row = out + (int64_t)at.line * ldo;
        const int64_t col = (int64_t)at.step * 256 + u * (32 * N) + N * sub;
        if (kWhole && col + N <= k) {
          V o;
#pragma unroll
          for (int e = 0; e < N; ++e) o[e] = (T)v[e];
          __builtin_nontemporal_store(o, reinterpret_cast<V*>(row + col));
        } else {
          store_vec(row, col, k, v);
        }
      }
    }
    at.two_on(steps);
  }
}

// Lines of a launch: fewer than 2^32 threads, units in 32 bits.
int64_t lines_at_once(int64_t steps) {
  const int64_t most = (int64_t)1 << 26;
  return steps < most ? most / steps : 1;
}

inline unsigned unit_blocks(int64_t lines, int64_t steps) {
  return (unsigned)((lines * steps + 4 * kUnits - 1) / (4 * kUnits));
}

template <typename T, int kC>
void quant_columns(int64_t rows, int64_t cols, const T* x, int64_t ldx, uint8_t* codes,
                   int64_t ldq, uint8_t* scales, int64_t lds, hipStream_t s) {
  const int64_t steps = (rows + 255) / 256;
  const int64_t tiles = (cols + 64 * kC - 1) / (64 * kC), most = 1 << 22;
  // ids are 32 bits: lines past that many tiles go in launches of their own
  for (int64_t t0 = 0; t0 < tiles; t0 += most) {
    const int64_t nt = tiles - t0 < most ? tiles - t0 : most;
    const int64_t c0 = t0 * 64 * kC, nc = cols - c0 < nt * 64 * kC ? cols - c0 : nt * 64 * kC;
    for (int64_t st0 = 0; st0 < steps; st0 += most / nt) {
      const int64_t ns = steps - st0 < most / nt ? steps - st0 : most / nt;
      hipLaunchKernelGGL((mxfp4_cols_kernel<T, kC>), dim3((unsigned)(nt * ns)), dim3(512), 0, s,
                         rows - st0 * 256, nc, (uint32_t)nt, x + st0 * 256 * ldx + c0, ldx,
                         codes + c0 * ldq + st0 * 128, ldq, scales + c0 * lds + st0 * 8, lds);
    }
  }
}

template <typename T>
int quant_t(int64_t rows, int64_t cols, const T* x, int64_t ldx, int axis, uint8_t* codes,
            int64_t ldq, uint8_t* scales, int64_t lds, hipStream_t s) {
  if (axis == 0) {
    const int64_t steps = (cols + 255) / 256, most = lines_at_once(steps);
    for (int64_t r = 0; r < rows; r += most) {
      const int64_t some = rows - r < most ? rows - r : most;
      hipLaunchKernelGGL((mxfp4_rows_kernel<T>), dim3(unit_blocks(some, steps)), dim3(256), 0, s,
                         (uint32_t)some, cols, (uint32_t)steps, x + r * ldx, ldx, codes + r * ldq,
                         ldq, scales + r * lds, lds);
    }
  } else {
    // two columns a lane, so that a wave's load of a row is 256 or 512 bytes (4099 x 5001 fp32:
    // 19.0 us, with one 22.0); of fp64 one is 512
    bool two = false;
    if constexpr (sizeof(T) <= 4) {
      two = cols > 1;
      if (two) quant_columns<T, 2>(rows, cols, x, ldx, codes, ldq, scales, lds, s);
    }
    if (!two) quant_columns<T, 1>(rows, cols, x, ldx, codes, ldq, scales, lds, s);
  }
  return hipGetLastError() == hipSuccess ? OZK_OK : OZK_EHIP;
}

template <typename T>
int values_t(int64_t lines, int64_t k, const uint8_t* codes, int64_t ldq, const uint8_t* scales,
             int64_t lds, T* out, int64_t ldo, hipStream_t s) {
  const int64_t steps = (k + 255) / 256, most = lines_at_once(steps);
  const bool whole = reinterpret_cast<uintptr_t>(out) % 16 == 0 && ldo * sizeof(T) % 16 == 0;
  for (int64_t r = 0; r < lines; r += most) {
    const int64_t some = lines - r < most ? lines - r : most;
    const dim3 grid(unit_blocks(some, steps)), block(256);
#define OZK_VALUES(WHOLE)                                                                         \
  hipLaunchKernelGGL((mxfp4_values_kernel<T, WHOLE>), grid, block, 0, s, (uint32_t)some, k,       \
                     (uint32_t)steps, codes + r * ldq, ldq, scales + r * lds, lds, out + r * ldo, \
                     ldo)
    if (whole) OZK_VALUES(true);
    else OZK_VALUES(false);
#undef OZK_VALUES
  }
  return hipGetLastError() == hipSuccess ? OZK_OK : OZK_EHIP;
}

}  // namespace

int launch_mxfp4_quant(int64_t rows, int64_t cols, int type, const void* x, int64_t ldx, int axis,
                       uint8_t* codes, int64_t ldq, uint8_t* scales, int64_t lds, hipStream_t s) {
  switch (type) {
    case OZK_F64:
      return quant_t(rows, cols, (const double*)x, ldx, axis, codes, ldq, scales, lds, s);
    case OZK_F32:
      return quant_t(rows, cols, (const float*)x, ldx, axis, codes, ldq, scales, lds, s);
    case OZK_F16:
      return quant_t(rows, cols, (const f16_t*)x, ldx, axis, codes, ldq, scales, lds, s);
    default:
      return quant_t(rows, cols, (const bf16_t*)x, ldx, axis, codes, ldq, scales, lds, s);
  }
}

int launch_mxfp4_values(int64_t lines, int64_t k, const uint8_t* codes, int64_t ldq,
                        const uint8_t* scales, int64_t lds, int type, void* out, int64_t ldo,
                        hipStream_t s) {
  switch (type) {
    case OZK_F64:
      return values_t(lines, k, codes, ldq, scales, lds, (double*)out, ldo, s);
    case OZK_F32:
      return values_t(lines, k, codes, ldq, scales, lds, (float*)out, ldo, s);
    case OZK_F16:
      return values_t(lines, k, codes, ldq, scales, lds, (f16_t*)out, ldo, s);
    default:
      return values_t(lines, k, codes, ldq, scales, lds, (bf16_t*)out, ldo, s);
  }
}

}  // namespace ozk
