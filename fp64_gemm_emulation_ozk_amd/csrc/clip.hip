// Clipping of many tensors to a global norm: N = (sum of all |x|^2)^(1/2), y = x min(1, M / N).
//
// Two passes, each one launch for up to 128 tensors, whose addresses, sizes and types travel with
// the launch (nothing is copied to the device, so a call can be captured).  The tensors are cut
// into chunks, dealt out to at most 512 workgroups (two per compute unit).  The first pass leaves
// each workgroup's sums, the second's workgroups all add them in the same order and scale.
// Squares are summed in 64 bits.  Those of fp64 values may leave its range, so they are summed
// three times, as they are and with the values scaled by 2^-600 and 2^600.
//
// Memory bounds both passes.  All of a chunk's loads are in flight at once: a thread has four of
// 16 bytes in the first pass, where eight took longer (166 -> 169 us over 1.0 GB of bf16), and
// eight in the second (406 -> 380 us with its writes of as much).  The second pass's loads and
// stores are marked as not to be read soon: the whole of 1.1 GB 581 -> 541 us, 134 MB 84 -> 68,
// 25 MB 22.5 -> 19.2; with a reader of the outputs behind 761 -> 713, 98 -> 101 and 32.8 -> 32.0
// (tensors at odd elements, 1.0 GB: bf16 630 -> 622, fp32 604 -> 582, fp64 614 -> 592).
#include "ozk_internal.h"
#include "rows.h"

namespace ozk {
namespace {

constexpr int kTensors = 128, kThreads = 512, kGroups = 512;
// Vectors of 16 bytes a thread takes of a chunk, in the pass that sums and in that which scales.
constexpr int kSumVectors = 4, kScaleVectors = 8;
static_assert(kSumVectors != kScaleVectors, "they tell the passes apart");

constexpr int chunk_bytes(int vectors) { return vectors * kThreads * 16; }

constexpr double kDown = 0x1p-600, kUp = 0x1p+600;

struct ClipTable {
  int count, chunks;
  const void* x[kTensors];
  void* out[kTensors];
  int64_t size[kTensors];
  int first[kTensors];       // a tensor's first chunk
  uint8_t type[kTensors];
};
static_assert(sizeof(ClipTable) <= 3800, "a launch's arguments take 4 KiB");

// Sums of squares: of the values, and of the values times 2^-600 and 2^600.
struct Squares {
  double mid = 0, low = 0, high = 0;
};

template <typename T>
__device__ __forceinline__ void add_square(Squares& s, T v) {
  const double d = (double)v;
  s.mid = __builtin_fma(d, d, s.mid);
  if constexpr (sizeof(T) == 8) {
    const double a = d * kDown, b = d * kUp;
    s.low = __builtin_fma(a, a, s.low);
    s.high = __builtin_fma(b, b, s.high);
  }
}

// The tensor of a chunk: the last one whose first chunk is not past it.
__device__ __forceinline__ int tensor_of(const ClipTable& A, int chunk) {
  int lo = 0, hi = A.count;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (A.first[mid] <= chunk) lo = mid;
    else hi = mid;
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// f(vector, how many of its elements, its first element) over the chunk's vectors of 16 bytes,
// kV loads of a thread at once; its last, short vector's elements alone.
template <int kV, typename T, typename F>
__device__ __forceinline__ void each_vector(const T* x, int64_t size, int chunk, F f) {
  constexpr int N = Vec<T>::N;
  typedef typename Vec<T>::type V;
  // which chunk is the last is compared in 32 bits: of a 64-bit comparison of uniform values this
  // compiler (clang of ROCm 7.2) took the branch from vcc and the selected count from a stale scc
  // (in the code of the library's other kernels every select and branch follows what sets its scc)
  constexpr int most = chunk_bytes(kV) / (int)sizeof(T);
  const int64_t begin = (int64_t)chunk * most;
  const T* p = x + begin;
  if (chunk < (int)((size - 1) / most)) {
    V v[kV];
#pragma unroll
    for (int q = 0; q < kV; ++q) {
      const V* at = reinterpret_cast<const V*>(p + (q * kThreads + threadIdx.x) * N);
      if constexpr (kV == kScaleVectors) v[q] = __builtin_nontemporal_load(at);
      else v[q] = *at;
    }
#pragma unroll
    for (int q = 0; q < kV; ++q) f(v[q], N, begin + (q * kThreads + threadIdx.x) * N);
    return;
  }
  const int count = (int)(size - begin);   // 1 .. most
  for (int e = threadIdx.x * N; e < count; e += kThreads * N) {
    if (e + N <= count) {
      f(*reinterpret_cast<const V*>(p + e), N, begin + e);
    } else {
      V v;
#pragma unroll
      for (int u = 0; u < N; ++u) v[u] = e + u < count ? p[e + u] : (T)0.0f;
      f(v, count - e, begin + e);
    }
  }
}

template <typename T>
__device__ __forceinline__ void sum_chunk(const ClipTable& A, int t, int chunk, Squares& sum) {
  Squares s;
  each_vector<kSumVectors>((const T*)A.x[t], A.size[t], chunk,
                           [&](const typename Vec<T>::type& v, int, int64_t) {
#pragma unroll
                             for (int u = 0; u < Vec<T>::N; ++u) add_square(s, v[u]);
                           });
  sum.mid += s.mid;
  // of the other types nothing is past the range but Inf itself, and nothing below 2^-298
  sum.low += sizeof(T) == 8 ? s.low : s.mid * kDown * kDown;
  sum.high += s.high;
}

__device__ __forceinline__ double block_sum(double v, double* slot) {
  return row_all<kThreads>(v, SumOp(), slot);
}

__global__ __launch_bounds__(kThreads) void clip_sums_kernel(ClipTable A,
                                                             double* __restrict__ part) {
  __shared__ double slots[3][kThreads / 64];
  Squares s;
  for (int c = blockIdx.x; c < A.chunks; c += gridDim.x) {
    const int t = tensor_of(A, c);
    const int chunk = c - A.first[t];
    switch (A.type[t]) {
      case OZK_F64: sum_chunk<double>(A, t, chunk, s); break;
      case OZK_F32: sum_chunk<float>(A, t, chunk, s); break;
      case OZK_F16: sum_chunk<f16_t>(A, t, chunk, s); break;
      default: sum_chunk<bf16_t>(A, t, chunk, s); break;
    }
  }
  const double mid = block_sum(s.mid, slots[0]);
  const double low = block_sum(s.low, slots[1]);
  const double high = block_sum(s.high, slots[2]);
  if (threadIdx.x == 0) {
    part[3 * blockIdx.x] = mid;
    part[3 * blockIdx.x + 1] = low;
    part[3 * blockIdx.x + 2] = high;
  }
}

// M / N as one number, and for fp64 values where it is subnormal, so that it holds few bits or
// none, as 2^-512 coef 2^-512, coef = M 2^512 / (N 2^-512), or 0 for coef elsewhere.  A value times
// 2^-512 loses bits only below 2^-510, where its output is 0.  The other types' outputs are below
// 2^-894 there, 0 in any of them.
struct Factor {
  double whole, coef;
};
__device__ __forceinline__ Factor factor_of(double max_norm, double total) {
  const double c = max_norm / total;
  return {c, c < 0x1p-1022 ? (max_norm * 0x1p512) / (total * 0x1p-512) : 0.0};
}

// kSteps: the factor in its parts (taken so for all values, 1.0 GB of fp64 takes 519 us for 516).
template <typename T, bool kSteps = false>
__device__ __forceinline__ void scale_chunk(const ClipTable& A, int t, int chunk,
                                            Factor by) {
  T* out = (T*)A.out[t];
  each_vector<kScaleVectors>(
      (const T*)A.x[t], A.size[t], chunk,
      [&](const typename Vec<T>::type& v, int count, int64_t at) {
        typename Vec<T>::type o;
#pragma unroll
        for (int u = 0; u < Vec<T>::N; ++u) {
          // to 16 bits by way of fp32, which is off a direct rounding by 2^-24 at most
          if constexpr (kSteps) o[u] = v[u] * 0x1p-512 * by.coef * 0x1p-512;
          else if constexpr (sizeof(T) == 8) o[u] = v[u] * by.whole;
          else o[u] = (T)(float)((double)v[u] * by.whole);
        }
        if (count == Vec<T>::N) {
          __builtin_nontemporal_store(o, reinterpret_cast<typename Vec<T>::type*>(out + at));
        } else {
#pragma unroll
          for (int u = 0; u < Vec<T>::N; ++u)
            if (u < count) out[at + u] = o[u];
        }
      });
}

// in_place: every out is its x, so that a norm within the bound leaves nothing to do.  Chunks are
// taken from the last: of what the first pass read, that may still be in the last-level cache.
__global__ __launch_bounds__(kThreads) void clip_scale_kernel(ClipTable A,
                                                              const double* __restrict__ part,
                                                              int parts, double max_norm,
                                                              int in_place,
                                                              double* __restrict__ norm) {
  __shared__ double slots[3][kThreads / 64];
  Squares s;
  for (int i = threadIdx.x; i < parts; i += kThreads) {
    s.mid += part[3 * i];
    s.low += part[3 * i + 1];
    s.high += part[3 * i + 2];
  }
  const double mid = block_sum(s.mid, slots[0]);
  const double low = block_sum(s.low, slots[1]);
  const double high = block_sum(s.high, slots[2]);
  // Where the squares' sum is past the range, what the scaled sum loses is below 2^-474 in
  // magnitude; where it is below 2^-900, no value times 2^600 passes 2^150.
  double total;
  if (__builtin_isinf(mid)) total = __builtin_sqrt(low) * kUp;
  else if (mid < 0x1p-900) total = __builtin_sqrt(high) * kDown;
  else total = __builtin_sqrt(mid);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = total;
  const bool clips = total > max_norm && !__builtin_isinf(total);
  if (!clips && in_place) return;
  const Factor by = clips ? factor_of(max_norm, total) : Factor{1.0, 0.0};
  for (int c = A.chunks - 1 - (int)blockIdx.x; c >= 0; c -= gridDim.x) {
    const int t = tensor_of(A, c);
    const int chunk = c - A.first[t];
    switch (A.type[t]) {
      case OZK_F64:
        if (by.coef == 0.0) scale_chunk<double>(A, t, chunk, by);
        else scale_chunk<double, true>(A, t, chunk, by);
        break;
      case OZK_F32: scale_chunk<float>(A, t, chunk, by); break;
      case OZK_F16: scale_chunk<f16_t>(A, t, chunk, by); break;
      default: scale_chunk<bf16_t>(A, t, chunk, by); break;
    }
  }
}

int64_t element_size(int type) { return type == OZK_F64 ? 8 : (type == OZK_F32 ? 4 : 2); }

// The tensors [t, t + returned) of a launch: those that are not empty, up to kTensors of them,
// in chunks of `bytes`.
int64_t fill_table(ClipTable& A, int64_t t, int64_t count, const void* const* x, void* const* out,
                   const int64_t* sizes, const int* types, int64_t bytes, bool* in_place) {
  A.count = A.chunks = 0;
  int64_t i = t;
  for (; i < count && A.count < kTensors; ++i) {
    if (sizes[i] == 0) continue;
    A.x[A.count] = x[i];
    A.out[A.count] = out[i];
    A.size[A.count] = sizes[i];
    A.type[A.count] = (uint8_t)types[i];
    A.first[A.count] = A.chunks;
    A.chunks += (int)((sizes[i] * element_size(types[i]) + bytes - 1) / bytes);
    *in_place = *in_place && x[i] == out[i];
    ++A.count;
  }
  return i - t;
}

}  // namespace

size_t clip_norm_workspace(int64_t count) {
  return align256((size_t)((count + kTensors - 1) / kTensors) * kGroups * 3 * 8);
}

int launch_clip_norm(int64_t count, const void* const* x, void* const* out, const int64_t* sizes,
                     const int* types, double max_norm, double* norm, void* workspace,
                     hipStream_t s) {
  double* part = static_cast<double*>(workspace);
  ClipTable A;
  int parts = 0;
  bool in_place = true;
  for (int64_t t = 0; t < count;) {
    t += fill_table(A, t, count, x, out, sizes, types, chunk_bytes(kSumVectors), &in_place);
    if (A.chunks == 0) continue;
    const int groups = A.chunks < kGroups ? A.chunks : kGroups;
    hipLaunchKernelGGL(clip_sums_kernel, dim3(groups), dim3(kThreads), 0, s, A,
                       part + 3 * (int64_t)parts);
    parts += groups;
  }
  bool first = true;
  for (int64_t t = 0; t < count || first;) {
    t += fill_table(A, t, count, x, out, sizes, types, chunk_bytes(kScaleVectors), &in_place);
    if (A.chunks == 0 && !(first && t >= count)) continue;
    const int groups = A.chunks < kGroups ? (A.chunks > 0 ? A.chunks : 1) : kGroups;
    hipLaunchKernelGGL(clip_scale_kernel, dim3(groups), dim3(kThreads), 0, s, A, part, parts,
                       max_norm, in_place ? 1 : 0, first ? norm : nullptr);
    first = false;
  }
  return hipGetLastError() == hipSuccess ? OZK_OK : OZK_EHIP;
}

}  // namespace ozk
