// The reconstruction of [TME4] abstract as a launch of its own: the outputs of crt_core.h
// stored to C.
#include "crt_core.h"

namespace ozk {
namespace {

struct Store {
  double* c;
  int64_t ldc;
  struct Nothing {};
  __device__ __forceinline__ Nothing ask(int64_t, int64_t) const { return {}; }
  __device__ __forceinline__ void operator()(int64_t i, int64_t j, double v, Nothing) const {
    c[i * ldc + j] = v;
  }
};

template <int R, typename T>
__global__ __launch_bounds__(256) void crt_kernel(int64_t m, int64_t n, const T* __restrict__ res,
                                                  int64_t ldr, int64_t stride_r,
                                                  const int32_t* __restrict__ ea,
                                                  const int32_t* __restrict__ eb,
                                                  double* __restrict__ c, int64_t ldc) {
  crt_outputs<R, T>(m, n, n, res, ldr, stride_r, ea, eb, Store{c, ldc});
}

template <int R>
void launch_r(dim3 grid, hipStream_t s, int64_t m, int64_t n, const void* res, int is_i32,
              int64_t ldr, int64_t stride_r, const int32_t* ea, const int32_t* eb, double* c,
              int64_t ldc) {
  if (is_i32)
    hipLaunchKernelGGL((crt_kernel<R, int32_t>), grid, dim3(256), 0, s, m, n,
                       (const int32_t*)res, ldr, stride_r, ea, eb, c, ldc);
  else
    hipLaunchKernelGGL((crt_kernel<R, int8_t>), grid, dim3(256), 0, s, m, n, (const int8_t*)res,
                       ldr, stride_r, ea, eb, c, ldc);
}

template <int... Rs>
struct Dispatch;

template <>
struct Dispatch<> {
  static void go(int, dim3, hipStream_t, int64_t, int64_t, const void*, int, int64_t, int64_t,
                 const int32_t*, const int32_t*, double*, int64_t) {}
};

template <int R0, int... Rs>
struct Dispatch<R0, Rs...> {
  static void go(int r, dim3 g, hipStream_t s, int64_t m, int64_t n, const void* res, int i32,
                 int64_t ldr, int64_t sr, const int32_t* ea, const int32_t* eb, double* c,
                 int64_t ldc) {
    if (r == R0)
      launch_r<R0>(g, s, m, n, res, i32, ldr, sr, ea, eb, c, ldc);
    else
      Dispatch<Rs...>::go(r, g, s, m, n, res, i32, ldr, sr, ea, eb, c, ldc);
  }
};

}  // namespace

int launch_crt(int64_t m, int64_t n, int r, const void* res, int res_is_i32, int64_t ldr,
               int64_t stride_r, const int32_t* ea, const int32_t* eb, double* c, int64_t ldc,
               hipStream_t s) {
  if (m <= 0 || n <= 0) return OZK_OK;
  if (r < 1 || r > kMaxModuli) return OZK_EINVAL;
  dim3 grid((unsigned)crt_blocks(m, n));
  Dispatch<1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15, 16, 17, 18, 19, 20>::go(
      r, grid, s, m, n, res, res_is_i32, ldr, stride_r, ea, eb, c, ldc);
  return hipGetLastError() == hipSuccess ? OZK_OK : OZK_EHIP;
}

}  // namespace ozk
