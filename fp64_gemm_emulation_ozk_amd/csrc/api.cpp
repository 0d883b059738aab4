// extern "C" entry points of libozk.so: argument validation (before any HIP call),
// workspace carving, and the stream-ordered launch sequence of each operation.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <new>

#include "ozk_internal.h"

using namespace ozk;

namespace {

inline hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Workspace carving: consecutive 256-byte aligned regions.
struct Carver {
  char* base;
  size_t off = 0;
  explicit Carver(void* b) : base(static_cast<char*>(b)) {}
  void* take(size_t bytes) {
    void* p = base ? base + off : nullptr;
    off += align256(bytes);
    return p;
  }
};

// Scratch of one operand's deconstruction beyond its planes and exponents: the line
// maxima of the max rule, or the chunk partials of the norm rule; the larger of the two,
// so that one workspace query serves both rules.  None for rows the fused kernel takes.
size_t deconstruct_scratch(int64_t rows, int64_t cols, int axis) {
  if (axis == 0 && rows_fused_supported(cols)) return 0;
  const int64_t lines = axis == 0 ? rows : cols;
  const size_t maxb = align256((size_t)lines * 8);
  const size_t part = 2 * align256((size_t)lines * norm_chunks(rows, cols, axis) * 8);
  return maxb > part ? maxb : part;
}

struct DgemmLayout {
  int64_t kp;
  size_t planes_a, planes_b, residues, exps_a, exps_b, scr_a, scr_b;
  size_t total() const {
    return align256(planes_a) + align256(planes_b) + align256(residues) + align256(exps_a) +
           align256(exps_b) + align256(scr_a) + align256(scr_b);
  }
};

DgemmLayout dgemm_layout(int64_t m, int64_t n, int64_t k, int r) {
  DgemmLayout L;
  // K padded to whole 128-byte rows: the products then stream whole cache lines.
  L.kp = round_up(k, 2 * kPlaneK);
  L.planes_a = (size_t)r * m * L.kp;
  L.planes_b = (size_t)r * n * L.kp;
  L.residues = (size_t)r * m * n;
  L.exps_a = (size_t)m * 4;
  L.exps_b = (size_t)n * 4;
  L.scr_a = deconstruct_scratch(m, k, 0);
  L.scr_b = deconstruct_scratch(k, n, 1);
  return L;
}

int check_r(int r) { return (r >= 1 && r <= kMaxModuli) ? OZK_OK : OZK_EINVAL; }

// First pass of a column deconstruction: the column maxima (max rule, into scratch as
// maxbits) or the norm-rule exponents (chunk partials in scratch, exponents into exps).
int cols_prep(const double* x, int64_t rows, int64_t cols, int64_t ldx, int scaling, int width,
              void* scratch, int32_t* exps, hipStream_t s) {
  int st;
  if (scaling == OZK_SCALING_NORM) {
    Carver cv(scratch);
    const size_t n = (size_t)cols * norm_chunks(rows, cols, 1) * 8;
    uint64_t* pmax = static_cast<uint64_t*>(cv.take(n));
    double* ps = static_cast<double*>(cv.take(n));
    return launch_norm_exps(x, rows, cols, ldx, 1, width, pmax, ps, exps, s);
  }
  uint64_t* maxbits = static_cast<uint64_t*>(scratch);
  if ((st = launch_fill_u64(maxbits, cols, 0, s)) != OZK_OK) return st;
  return launch_absmax(x, rows, cols, ldx, 1, maxbits, s);
}

// Deconstruct one operand (axis 0: per-row, axis 1: per-column) into planes by either
// scaling rule; width is P (max rule) or alpha (norm rule) of this operand and scratch
// holds deconstruct_scratch(rows, cols, axis) bytes.
int deconstruct_impl(const double* x, int64_t rows, int64_t cols, int64_t ldx, int axis, int r,
                     int scaling, int width, int8_t* planes, int64_t ldp, int64_t plane_stride,
                     int32_t* exps, void* scratch, hipStream_t s) {
  int st;
  if (axis == 0 && rows_fused_supported(cols))
    return launch_residues_rows_fused(x, rows, cols, ldx, r, scaling, width, planes, ldp,
                                      plane_stride, exps, s);
  const int norm = scaling == OZK_SCALING_NORM;
  if (axis == 1) {
    if ((st = cols_prep(x, rows, cols, ldx, scaling, width, scratch, exps, s)) != OZK_OK)
      return st;
    return launch_residues(x, rows, cols, ldx, 1, r, width,
                           static_cast<const uint64_t*>(scratch), planes, ldp, plane_stride,
                           exps, norm, s);
  }
  if (norm) {
    Carver cv(scratch);
    const size_t n = (size_t)rows * norm_chunks(rows, cols, 0) * 8;
    uint64_t* pmax = static_cast<uint64_t*>(cv.take(n));
    double* ps = static_cast<double*>(cv.take(n));
    if ((st = launch_norm_exps(x, rows, cols, ldx, 0, width, pmax, ps, exps, s)) != OZK_OK)
      return st;
    return launch_residues(x, rows, cols, ldx, 0, r, width, nullptr, planes, ldp,
                           plane_stride, exps, 1, s);
  }
  uint64_t* maxbits = static_cast<uint64_t*>(scratch);
  if ((st = launch_fill_u64(maxbits, rows, 0, s)) != OZK_OK) return st;
  if ((st = launch_absmax(x, rows, cols, ldx, 0, maxbits, s)) != OZK_OK) return st;
  return launch_residues(x, rows, cols, ldx, 0, r, width, maxbits, planes, ldp, plane_stride,
                         exps, 0, s);
}

// Both operands of a product: B's first pass, then A's rows and B's residues in one
// launch where that applies, else one operand after the other.
int deconstruct_operands(const double* A, int64_t m, int64_t k, int64_t lda, const double* B,
                         int64_t n, int64_t ldb, int r, int scaling, int wa, int wb,
                         int8_t* planes_a, int8_t* planes_b, int64_t kp, int32_t* exps_a,
                         int32_t* exps_b, void* scr_a, void* scr_b, hipStream_t s) {
  int st;
  if (!rows_fused_supported(k) || k > 8192) {
    if ((st = deconstruct_impl(A, m, k, lda, 0, r, scaling, wa, planes_a, kp, m * kp, exps_a,
                               scr_a, s)))
      return st;
    return deconstruct_impl(B, k, n, ldb, 1, r, scaling, wb, planes_b, kp, n * kp, exps_b,
                            scr_b, s);
  }
  if ((st = cols_prep(B, k, n, ldb, scaling, wb, scr_b, exps_b, s)) != OZK_OK) return st;
  st = launch_deconstruct_pair(A, m, k, lda, B, n, ldb, r, scaling, wa, wb,
                               static_cast<const uint64_t*>(scr_b), planes_a, planes_b, kp,
                               exps_a, exps_b, s);
  if (st != OZK_EUNSUPPORTED) return st;
  if ((st = launch_residues_rows_fused(A, m, k, lda, r, scaling, wa, planes_a, kp, m * kp,
                                       exps_a, s)))
    return st;
  return launch_residues(B, k, n, ldb, 1, r, wb, static_cast<const uint64_t*>(scr_b), planes_b,
                         kp, n * kp, exps_b, scaling == OZK_SCALING_NORM, s);
}

}  // namespace

extern "C" {

int ozk_version(void) { return 100; }

const char* ozk_status_string(int status) {
  switch (status) {
    case OZK_OK: return "success";
    case OZK_EINVAL: return "invalid argument";
    case OZK_EWORKSPACE: return "workspace missing or too small";
    case OZK_ERANGE: return "inner dimension out of range for exact products or the bit budget";
    case OZK_EHIP: return "HIP launch failed";
    case OZK_EUNSUPPORTED: return "unsupported request";
    case OZK_ENOSCRATCH:
      return "request needs more scratch than the allocation-free entry point holds";
    default: return "unknown status";
  }
}

int ozk_moduli(int r, int32_t* out) { return moduli_list(r, out); }

int ozk_scaling_bits(int r, int64_t k, int32_t* pa, int32_t* pb) {
  int a = 0, b = 0;
  int st = scaling_bits(r, k, &a, &b);
  if (st != OZK_OK) return st;
  if (pa) *pa = a;
  if (pb) *pb = b;
  return OZK_OK;
}

int ozk_scaling_bits_ex(int r, int64_t k, int scaling, int32_t* pa, int32_t* pb) {
  int a = 0, b = 0;
  int st = scaling_widths(scaling, r, k, &a, &b);
  if (st != OZK_OK) return st;
  if (pa) *pa = a;
  if (pb) *pb = b;
  return OZK_OK;
}

int64_t ozk_planes_ld(int64_t k) { return k <= 0 ? 0 : round_up(k, kPlaneK); }

int ozk_deconstruct_workspace_size(int64_t rows, int64_t cols, int axis, size_t* bytes) {
  if (!bytes || rows < 0 || cols < 0 || (axis != 0 && axis != 1)) return OZK_EINVAL;
  *bytes = deconstruct_scratch(rows, cols, axis);
  return OZK_OK;
}

int ozk_deconstruct_ex(const double* x, int64_t rows, int64_t cols, int64_t ldx, int axis,
                       int r, int64_t k_budget, int scaling, int8_t* planes, int64_t ldp,
                       int64_t plane_stride, int32_t* exps, void* workspace,
                       size_t workspace_bytes, void* stream) {
  if (axis != 0 && axis != 1) return OZK_EINVAL;
  if (scaling != OZK_SCALING_MAX && scaling != OZK_SCALING_NORM) return OZK_EINVAL;
  if (check_r(r) != OZK_OK) return OZK_EINVAL;
  if (rows < 0 || cols < 0 || ldx < (cols > 0 ? cols : 1)) return OZK_EINVAL;
  const int64_t K = axis == 0 ? cols : rows;
  const int64_t lines = axis == 0 ? rows : cols;
  if (ldp < K || ldp % kPlaneK != 0 || ldp <= 0) return OZK_EINVAL;
  if (plane_stride < lines * ldp || plane_stride % kPlaneK != 0) return OZK_EINVAL;
  int wa = 0, wb = 0;
  int st = scaling_widths(scaling, r, k_budget, &wa, &wb);
  if (st != OZK_OK) return st;
  if (lines == 0) return OZK_OK;
  if (!planes || !exps || (K > 0 && !x)) return OZK_EINVAL;
  if (!aligned(planes, 16)) return OZK_EINVAL;
  const size_t need = deconstruct_scratch(rows, cols, axis);
  if (need > workspace_bytes || (need > 0 && !workspace)) return OZK_EWORKSPACE;
  if (need > 0 && !aligned(workspace, 8)) return OZK_EINVAL;
  return deconstruct_impl(x, rows, cols, ldx, axis, r, scaling, axis == 0 ? wa : wb, planes,
                          ldp, plane_stride, exps, workspace, as_stream(stream));
}

int ozk_deconstruct(const double* x, int64_t rows, int64_t cols, int64_t ldx, int axis, int r,
                    int64_t k_budget, int8_t* planes, int64_t ldp, int64_t plane_stride,
                    int32_t* exps, void* workspace, size_t workspace_bytes, void* stream) {
  return ozk_deconstruct_ex(x, rows, cols, ldx, axis, r, k_budget, OZK_SCALING_MAX, planes, ldp,
                            plane_stride, exps, workspace, workspace_bytes, stream);
}

int ozk_modular_products(int64_t m, int64_t n, int64_t kp, int r, const int8_t* pa,
                         int64_t stride_a, const int8_t* pb, int64_t stride_b,
                         int32_t* products, int64_t ldp_out, int64_t stride_p, void* stream) {
  if (check_r(r) != OZK_OK) return OZK_EINVAL;
  if (m < 0 || n < 0 || kp <= 0 || kp % kPlaneK != 0) return OZK_EINVAL;
  if (kp > round_up(OZK_MAX_K, kPlaneK)) return OZK_ERANGE;
  if (ldp_out < (n > 0 ? n : 1) || stride_p < m * ldp_out) return OZK_EINVAL;
  if (stride_a < m * kp || stride_b < n * kp) return OZK_EINVAL;
  if (stride_a % 16 || stride_b % 16) return OZK_EINVAL;
  if (m == 0 || n == 0) return OZK_OK;
  if (!pa || !pb || !products || !aligned(pa, 16) || !aligned(pb, 16)) return OZK_EINVAL;
  return launch_gemm_i8(m, n, kp, r, pa, stride_a, pb, stride_b, products, ldp_out, stride_p,
                        kEpiProducts, as_stream(stream));
}

int ozk_modular_residues(int64_t m, int64_t n, int64_t kp, int r, const int8_t* pa,
                         int64_t stride_a, const int8_t* pb, int64_t stride_b, int8_t* residues,
                         int64_t ldr, int64_t stride_r, void* stream) {
  if (check_r(r) != OZK_OK) return OZK_EINVAL;
  if (m < 0 || n < 0 || kp <= 0 || kp % kPlaneK != 0) return OZK_EINVAL;
  if (kp > round_up(OZK_MAX_K, kPlaneK)) return OZK_ERANGE;
  if (ldr < (n > 0 ? n : 1) || stride_r < m * ldr) return OZK_EINVAL;
  if (stride_a < m * kp || stride_b < n * kp) return OZK_EINVAL;
  if (stride_a % 16 || stride_b % 16) return OZK_EINVAL;
  if (m == 0 || n == 0) return OZK_OK;
  if (!pa || !pb || !residues || !aligned(pa, 16) || !aligned(pb, 16)) return OZK_EINVAL;
  return launch_gemm_i8(m, n, kp, r, pa, stride_a, pb, stride_b, residues, ldr, stride_r,
                        kEpiResidues, as_stream(stream));
}

int ozk_reconstruct(int64_t m, int64_t n, int r, const int32_t* products, int64_t ldp_in,
                    int64_t stride_p, const int32_t* exps_a, const int32_t* exps_b, double* C,
                    int64_t ldc, void* stream) {
  if (check_r(r) != OZK_OK) return OZK_EINVAL;
  if (m < 0 || n < 0) return OZK_EINVAL;
  if (ldp_in < (n > 0 ? n : 1) || stride_p < m * ldp_in || ldc < (n > 0 ? n : 1))
    return OZK_EINVAL;
  if (m == 0 || n == 0) return OZK_OK;
  if (!products || !exps_a || !exps_b || !C) return OZK_EINVAL;
  return launch_crt(m, n, r, products, 1, ldp_in, stride_p, exps_a, exps_b, C, ldc,
                    as_stream(stream));
}

int ozk_dgemm_workspace_size(int64_t m, int64_t n, int64_t k, int r, size_t* bytes) {
  if (!bytes || m < 0 || n < 0 || k < 1 || check_r(r) != OZK_OK) return OZK_EINVAL;
  if (k > OZK_MAX_K) return OZK_ERANGE;
  *bytes = dgemm_layout(m, n, k, r).total();
  return OZK_OK;
}

int ozk_dgemm_ex(int64_t m, int64_t n, int64_t k, const double* A, int64_t lda,
                 const double* B, int64_t ldb, double* C, int64_t ldc, int r, int scaling,
                 void* workspace, size_t workspace_bytes, void* stream) {
  return ozk_dgemm_ex_timed(m, n, k, A, lda, B, ldb, C, ldc, r, scaling, workspace,
                            workspace_bytes, stream, nullptr, nullptr);
}

int ozk_dgemm_ex_timed(int64_t m, int64_t n, int64_t k, const double* A, int64_t lda,
                       const double* B, int64_t ldb, double* C, int64_t ldc, int r, int scaling,
                       void* workspace, size_t workspace_bytes, void* stream,
                       void* gemm_start, void* gemm_stop) {
  if ((gemm_start == nullptr) != (gemm_stop == nullptr)) return OZK_EINVAL;
  if (check_r(r) != OZK_OK) return OZK_EINVAL;
  if (scaling != OZK_SCALING_MAX && scaling != OZK_SCALING_NORM) return OZK_EINVAL;
  if (m < 0 || n < 0 || k < 1) return OZK_EINVAL;
  if (k > OZK_MAX_K) return OZK_ERANGE;
  if (lda < k || ldb < (n > 0 ? n : 1) || ldc < (n > 0 ? n : 1)) return OZK_EINVAL;
  int wa = 0, wb = 0;
  int st = scaling_widths(scaling, r, k, &wa, &wb);
  if (st != OZK_OK) return st;
  if (m == 0 || n == 0) return OZK_OK;
  if (!A || !B || !C) return OZK_EINVAL;
  const DgemmLayout L = dgemm_layout(m, n, k, r);
  if (!workspace || workspace_bytes < L.total()) return OZK_EWORKSPACE;
  if (!aligned(workspace, 256)) return OZK_EINVAL;
  if ((size_t)m * n > (size_t)0x7fffffffffffull) return OZK_EUNSUPPORTED;
  Carver cv(workspace);
  int8_t* planes_a = static_cast<int8_t*>(cv.take(L.planes_a));
  int8_t* planes_b = static_cast<int8_t*>(cv.take(L.planes_b));
  int8_t* residues = static_cast<int8_t*>(cv.take(L.residues));
  int32_t* exps_a = static_cast<int32_t*>(cv.take(L.exps_a));
  int32_t* exps_b = static_cast<int32_t*>(cv.take(L.exps_b));
  void* scr_a = cv.take(L.scr_a);
  void* scr_b = cv.take(L.scr_b);
  hipStream_t s = as_stream(stream);
  const int64_t kp = L.kp;
  if ((st = deconstruct_operands(A, m, k, lda, B, n, ldb, r, scaling, wa, wb, planes_a,
                                 planes_b, kp, exps_a, exps_b, scr_a, scr_b, s)))
    return st;
  if ((st = launch_gemm_i8(m, n, kp, r, planes_a, m * kp, planes_b, n * kp, residues, n, m * n,
                           kEpiResidues, s, static_cast<hipEvent_t>(gemm_start),
                           static_cast<hipEvent_t>(gemm_stop))))
    return st;
  return launch_crt(m, n, r, residues, 0, n, m * n, exps_a, exps_b, C, ldc, s);
}

int ozk_dgemm(int64_t m, int64_t n, int64_t k, const double* A, int64_t lda, const double* B,
              int64_t ldb, double* C, int64_t ldc, int r, void* workspace,
              size_t workspace_bytes, void* stream) {
  return ozk_dgemm_ex(m, n, k, A, lda, B, ldb, C, ldc, r, OZK_SCALING_MAX, workspace,
                      workspace_bytes, stream);
}

}  // extern "C"

// ---------------------------------------------------------------- emulated DGEMV
namespace {

struct GemvLayout {
  int64_t kp;
  bool digits;   // on the fly through base-256 digits (scaling bits of A <= 50)
  size_t x_planes, x_exps, x_max, res, a_exps, a_max, xd, corr, part;
  size_t total() const {
    return align256(x_planes) + align256(x_exps) + align256(x_max) + align256(res) +
           align256(a_exps) + align256(a_max) + align256(xd) + align256(corr) +
           align256(part);
  }
};

GemvLayout gemv_layout(int64_t m, int64_t k, int64_t nrhs, int r, int mode) {
  GemvLayout L;
  L.kp = round_up(k, kPlaneK);
  L.x_planes = (size_t)r * nrhs * L.kp;
  L.x_exps = (size_t)nrhs * 4;
  L.x_max = (size_t)nrhs * 8;
  L.res = (size_t)r * m * nrhs;
  L.a_exps = mode == 0 ? (size_t)m * 4 : 0;
  L.a_max = mode == 0 ? (size_t)m * 8 : 0;
  int pa = 0, pb = 0;
  L.digits = mode == 0 && scaling_bits(r, k, &pa, &pb) == OZK_OK &&
             gemv_digits_supported(pa, (int64_t)r * nrhs);
  L.xd = L.corr = L.part = 0;
  if (L.digits) gemv_digits_workspace(m, L.kp, r, nrhs, &L.xd, &L.corr, &L.part);
  return L;
}

}  // namespace

extern "C" {

int ozk_dgemv_workspace_size(int64_t m, int64_t k, int64_t nrhs, int r, int mode,
                             size_t* bytes) {
  if (!bytes || m < 0 || k < 1 || nrhs < 1 || nrhs > 32 || check_r(r) != OZK_OK) return OZK_EINVAL;
  if (mode != 0 && mode != 1) return OZK_EINVAL;
  if (k > OZK_MAX_K) return OZK_ERANGE;
  *bytes = gemv_layout(m, k, nrhs, r, mode).total();
  return OZK_OK;
}

}  // extern "C"

namespace ozk {

int dgemv_validate(int64_t m, int64_t k, int64_t nrhs, const double* A, int64_t lda,
                   const int8_t* A_planes, int64_t ldp, int64_t plane_stride,
                   const int32_t* A_exps, const double* X, int64_t ldx, const double* Y,
                   int64_t ldy, int r, int mode) {
  if (check_r(r) != OZK_OK || (mode != 0 && mode != 1)) return OZK_EINVAL;
  if (m < 0 || k < 1 || nrhs < 1 || nrhs > 32) return OZK_EINVAL;
  if (k > OZK_MAX_K) return OZK_ERANGE;
  if (ldx < nrhs || ldy < nrhs) return OZK_EINVAL;
  int pa = 0, pb = 0;
  int st = scaling_bits(r, k, &pa, &pb);
  if (st != OZK_OK) return st;
  const int64_t kp = round_up(k, kPlaneK);
  if (mode == 0) {
    if (lda < k) return OZK_EINVAL;
  } else {
    if (ldp < kp || ldp % kPlaneK != 0 || plane_stride < m * ldp || plane_stride % 16 != 0)
      return OZK_EINVAL;
  }
  if (m == 0) return OZK_OK;
  if (!X || !Y) return OZK_EINVAL;
  if (mode == 0 && !A) return OZK_EINVAL;
  if (mode == 1 && (!A_planes || !A_exps || !aligned(A_planes, 16))) return OZK_EINVAL;
  return OZK_OK;
}

}  // namespace ozk

extern "C" {

int ozk_dgemv(int64_t m, int64_t k, int64_t nrhs, const double* A, int64_t lda,
              const int8_t* A_planes, int64_t ldp, int64_t plane_stride, const int32_t* A_exps,
              const double* X, int64_t ldx, double* Y, int64_t ldy, int r, int mode,
              void* workspace, size_t workspace_bytes, void* stream) {
  int st = dgemv_validate(m, k, nrhs, A, lda, A_planes, ldp, plane_stride, A_exps, X, ldx, Y,
                          ldy, r, mode);
  if (st != OZK_OK || m == 0) return st;
  int pa = 0, pb = 0;
  scaling_bits(r, k, &pa, &pb);
  const GemvLayout L = gemv_layout(m, k, nrhs, r, mode);
  if (!workspace || workspace_bytes < L.total()) return OZK_EWORKSPACE;
  if (!aligned(workspace, 256)) return OZK_EINVAL;
  Carver cv(workspace);
  int8_t* x_planes = static_cast<int8_t*>(cv.take(L.x_planes));
  int32_t* x_exps = static_cast<int32_t*>(cv.take(L.x_exps));
  uint64_t* x_max = static_cast<uint64_t*>(cv.take(L.x_max));
  int8_t* res = static_cast<int8_t*>(cv.take(L.res));
  int32_t* a_exps = static_cast<int32_t*>(cv.take(L.a_exps));
  uint64_t* a_max = static_cast<uint64_t*>(cv.take(L.a_max));
  int8_t* xd = static_cast<int8_t*>(cv.take(L.xd));
  int32_t* corr = static_cast<int32_t*>(cv.take(L.corr));
  int8_t* part = static_cast<int8_t*>(cv.take(L.part));
  hipStream_t s = as_stream(stream);
  const int64_t kp = L.kp;
  if ((st = deconstruct_impl(X, k, nrhs, ldx, 1, r, OZK_SCALING_MAX, pb, x_planes, kp, nrhs * kp,
                             x_exps, x_max, s)))
    return st;
  const int32_t* ea = A_exps;
  if (mode == 0) {
    if (!ea) {
      if ((st = launch_line_exps(A, m, k, lda, 0, pa, a_max, a_exps, s))) return st;
      ea = a_exps;
    }
    if (L.digits)
      st = launch_gemv_digits(A, m, k, lda, ea, r, x_planes, kp, nrhs * kp, (int)nrhs, xd, corr,
                              part, res, s);
    else
      st = launch_gemv_fly(A, m, k, lda, ea, r, pa, x_planes, kp, nrhs * kp, (int)nrhs, res, s);
  } else {
    st = launch_gemv_stored(m, kp, r, A_planes, ldp, plane_stride, x_planes, nrhs * kp,
                            (int)nrhs, res, s);
  }
  if (st) return st;
  return launch_crt(m, nrhs, r, res, 0, nrhs, m * nrhs, ea, x_exps, Y, ldy, s);
}

// ---------------------------------------------------------------- FP4-limb INT8 GEMM
int ozk_fp4limb_pack(const int8_t* x, int64_t rows, int64_t cols, int64_t ldx, int axis,
                     uint8_t* planes, int64_t ldp_bytes, int64_t plane_stride, void* stream) {
  if (axis != 0 && axis != 1) return OZK_EINVAL;
  if (rows < 0 || cols < 0 || ldx < (cols > 0 ? cols : 1)) return OZK_EINVAL;
  const int64_t K = axis == 0 ? cols : rows;
  const int64_t lines = axis == 0 ? rows : cols;
  if (ldp_bytes <= 0 || ldp_bytes % 32 != 0 || 2 * ldp_bytes < K) return OZK_EINVAL;
  if (plane_stride < lines * ldp_bytes || plane_stride % 16 != 0) return OZK_EINVAL;
  if (lines == 0) return OZK_OK;
  if (!planes || (K > 0 && !x) || !aligned(planes, 16)) return OZK_EINVAL;
  return launch_fp4_pack(x, rows, cols, ldx, axis, planes, ldp_bytes, plane_stride,
                         as_stream(stream));
}

int ozk_fp4limb_products(int64_t m, int64_t n, int64_t ldp_bytes, const uint8_t* planes_a,
                         int64_t stride_a, const uint8_t* planes_b, int64_t stride_b,
                         int32_t* products, int64_t ldp_out, int64_t stride_p, void* stream) {
  if (m < 0 || n < 0 || ldp_bytes <= 0 || ldp_bytes % 32 != 0) return OZK_EINVAL;
  if (2 * ldp_bytes > round_up(OZK_MAX_K, kPlaneK)) return OZK_ERANGE;
  if (stride_a < m * ldp_bytes || stride_b < n * ldp_bytes || stride_a % 16 || stride_b % 16)
    return OZK_EINVAL;
  if (ldp_out < (n > 0 ? n : 1) || stride_p < m * ldp_out) return OZK_EINVAL;
  if (m == 0 || n == 0) return OZK_OK;
  if (!planes_a || !planes_b || !products || !aligned(planes_a, 16) || !aligned(planes_b, 16))
    return OZK_EINVAL;
  return launch_fp4_products(m, n, ldp_bytes, planes_a, stride_a, planes_b, stride_b, products,
                             ldp_out, stride_p, as_stream(stream));
}

int ozk_int8gemm_fp4limb_workspace_size(int64_t m, int64_t n, int64_t k, size_t* bytes) {
  if (!bytes || m < 0 || n < 0 || k < 1) return OZK_EINVAL;
  if (k > OZK_MAX_K) return OZK_ERANGE;
  const int64_t ldpb = round_up(k, 2 * kPlaneK) / 2;  // K steps of 128 codes
  *bytes = align256((size_t)3 * m * ldpb) + align256((size_t)3 * n * ldpb);
  return OZK_OK;
}

int ozk_int8gemm_fp4limb(int64_t m, int64_t n, int64_t k, const int8_t* A, int64_t lda,
                         const int8_t* B, int64_t ldb, int32_t* C, int64_t ldc, void* workspace,
                         size_t workspace_bytes, void* stream) {
  if (m < 0 || n < 0 || k < 1) return OZK_EINVAL;
  if (k > OZK_MAX_K) return OZK_ERANGE;
  if (lda < k || ldb < (n > 0 ? n : 1) || ldc < (n > 0 ? n : 1)) return OZK_EINVAL;
  if (m == 0 || n == 0) return OZK_OK;
  if (!A || !B || !C) return OZK_EINVAL;
  size_t need = 0;
  ozk_int8gemm_fp4limb_workspace_size(m, n, k, &need);
  if (!workspace || workspace_bytes < need) return OZK_EWORKSPACE;
  if (!aligned(workspace, 256)) return OZK_EINVAL;
  const int64_t ldpb = round_up(k, 2 * kPlaneK) / 2;  // K steps of 128 codes
  Carver cv(workspace);
  uint8_t* pa = static_cast<uint8_t*>(cv.take((size_t)3 * m * ldpb));
  uint8_t* pb = static_cast<uint8_t*>(cv.take((size_t)3 * n * ldpb));
  hipStream_t s = as_stream(stream);
  int st;
  if ((st = launch_fp4_pack(A, m, k, lda, 0, pa, ldpb, m * ldpb, s))) return st;
  if ((st = launch_fp4_pack(B, k, n, ldb, 1, pb, ldpb, n * ldpb, s))) return st;
  return launch_fp4_gemm(m, n, ldpb, pa, m * ldpb, pb, n * ldpb, C, ldc, s);
}

// ---------------------------------------------------------------- 6-product FP4 INT8 GEMM
int64_t ozk_fp4awe_line_bytes(int64_t k) { return k <= 0 ? 0 : awe_line_bytes(k); }

int ozk_fp4awe_pack(const int8_t* x, int64_t rows, int64_t cols, int64_t ldx, int axis,
                    uint8_t* planes, int64_t ld_line, void* stream) {
  if (axis != 0 && axis != 1) return OZK_EINVAL;
  if (rows < 0 || cols < 0 || ldx < (cols > 0 ? cols : 1)) return OZK_EINVAL;
  const int64_t K = axis == 0 ? cols : rows;
  const int64_t lines = axis == 0 ? rows : cols;
  if (K > OZK_MAX_K) return OZK_ERANGE;
  if (ld_line < awe_line_bytes(K > 0 ? K : 1) || ld_line % 16 != 0) return OZK_EINVAL;
  if (lines == 0 || K == 0) return OZK_OK;
  if (!planes || !x || !aligned(planes, 16)) return OZK_EINVAL;
  return launch_awe_pack(x, rows, cols, ldx, axis, planes, ld_line, as_stream(stream));
}

int ozk_fp4awe_products(int64_t m, int64_t n, int64_t k, const uint8_t* planes_a, int64_t lda,
                        const uint8_t* planes_b, int64_t ldb, int32_t* products,
                        int64_t ldp_out, int64_t stride_p, void* stream) {
  if (m < 0 || n < 0 || k < 1) return OZK_EINVAL;
  if (k > OZK_MAX_K) return OZK_ERANGE;
  const int64_t line = awe_line_bytes(k);
  if (lda < line || ldb < line || lda % 16 || ldb % 16) return OZK_EINVAL;
  if (ldp_out < (n > 0 ? n : 1) || stride_p < m * ldp_out) return OZK_EINVAL;
  if (m == 0 || n == 0) return OZK_OK;
  if (!planes_a || !planes_b || !products || !aligned(planes_a, 16) || !aligned(planes_b, 16))
    return OZK_EINVAL;
  return launch_awe_products(m, n, line / 192, planes_a, lda, planes_b, ldb, products, ldp_out,
                             stride_p, as_stream(stream));
}

int ozk_int8gemm_fp4awe_workspace_size(int64_t m, int64_t n, int64_t k, size_t* bytes) {
  if (!bytes || m < 0 || n < 0 || k < 1) return OZK_EINVAL;
  if (k > OZK_MAX_K) return OZK_ERANGE;
  const int64_t line = awe_line_bytes(k);
  *bytes = align256((size_t)m * line) + align256((size_t)n * line);
  return OZK_OK;
}

int ozk_int8gemm_fp4awe(int64_t m, int64_t n, int64_t k, const int8_t* A, int64_t lda,
                        const int8_t* B, int64_t ldb, int32_t* C, int64_t ldc, void* workspace,
                        size_t workspace_bytes, void* stream) {
  if (m < 0 || n < 0 || k < 1) return OZK_EINVAL;
  if (k > OZK_MAX_K) return OZK_ERANGE;
  if (lda < k || ldb < (n > 0 ? n : 1) || ldc < (n > 0 ? n : 1)) return OZK_EINVAL;
  if (m == 0 || n == 0) return OZK_OK;
  if (!A || !B || !C) return OZK_EINVAL;
  size_t need = 0;
  ozk_int8gemm_fp4awe_workspace_size(m, n, k, &need);
  if (!workspace || workspace_bytes < need) return OZK_EWORKSPACE;
  if (!aligned(workspace, 256)) return OZK_EINVAL;
  const int64_t line = awe_line_bytes(k);
  Carver cv(workspace);
  uint8_t* pa = static_cast<uint8_t*>(cv.take((size_t)m * line));
  uint8_t* pb = static_cast<uint8_t*>(cv.take((size_t)n * line));
  hipStream_t s = as_stream(stream);
  int st;
  if ((st = launch_awe_pack(A, m, k, lda, 0, pa, line, s))) return st;
  if ((st = launch_awe_pack(B, k, n, ldb, 1, pb, line, s))) return st;
  return launch_awe_gemm(m, n, line / 192, pa, line, pb, line, C, ldc, s);
}

// ---------------------------------------------------------------- 4-product FP4 INT4 x INT8 GEMM
int64_t ozk_fp4awe4_line_bytes(int64_t k) { return k <= 0 ? 0 : awe4_line_bytes(k); }

int ozk_fp4awe4_pack(const int8_t* x, int64_t rows, int64_t cols, int64_t ldx, int axis,
                     int int4, uint8_t* planes, int64_t ld_line, void* stream) {
  if (axis != 0 && axis != 1) return OZK_EINVAL;
  if (int4 != 0 && int4 != 1) return OZK_EINVAL;
  if (rows < 0 || cols < 0 || ldx < (cols > 0 ? cols : 1)) return OZK_EINVAL;
  const int64_t K = axis == 0 ? cols : rows;
  const int64_t lines = axis == 0 ? rows : cols;
  if (K > OZK_MAX_K) return OZK_ERANGE;
  if (ld_line < awe4_line_bytes(K > 0 ? K : 1) || ld_line % 16 != 0) return OZK_EINVAL;
  if (lines == 0 || K == 0) return OZK_OK;
  if (!planes || !x || !aligned(planes, 16)) return OZK_EINVAL;
  return launch_awe4_pack(x, rows, cols, ldx, axis, int4, planes, ld_line, as_stream(stream));
}

int ozk_fp4awe4_products(int64_t m, int64_t n, int64_t k, const uint8_t* planes_a,
                         int64_t lda, const uint8_t* planes_b, int64_t ldb, int32_t* products,
                         int64_t ldp_out, int64_t stride_p, void* stream) {
  if (m < 0 || n < 0 || k < 1) return OZK_EINVAL;
  if (k > OZK_MAX_K) return OZK_ERANGE;
  const int64_t line = awe4_line_bytes(k);
  if (lda < line || ldb < line || lda % 16 || ldb % 16) return OZK_EINVAL;
  if (ldp_out < (n > 0 ? n : 1) || stride_p < m * ldp_out) return OZK_EINVAL;
  if (m == 0 || n == 0) return OZK_OK;
  if (!planes_a || !planes_b || !products || !aligned(planes_a, 16) || !aligned(planes_b, 16))
    return OZK_EINVAL;
  return launch_awe4_products(m, n, line / 128, planes_a, lda, planes_b, ldb, products,
                              ldp_out, stride_p, as_stream(stream));
}

int ozk_int4int8gemm_fp4awe_workspace_size(int64_t m, int64_t n, int64_t k, size_t* bytes) {
  if (!bytes || m < 0 || n < 0 || k < 1) return OZK_EINVAL;
  if (k > OZK_MAX_K) return OZK_ERANGE;
  const int64_t line = awe4_line_bytes(k);
  *bytes = align256((size_t)m * line) + align256((size_t)n * line);
  return OZK_OK;
}

int ozk_int4int8gemm_fp4awe(int64_t m, int64_t n, int64_t k, const int8_t* A, int64_t lda,
                            const int8_t* B, int64_t ldb, int32_t* C, int64_t ldc,
                            void* workspace, size_t workspace_bytes, void* stream) {
  if (m < 0 || n < 0 || k < 1) return OZK_EINVAL;
  if (k > OZK_MAX_K) return OZK_ERANGE;
  if (lda < k || ldb < (n > 0 ? n : 1) || ldc < (n > 0 ? n : 1)) return OZK_EINVAL;
  if (m == 0 || n == 0) return OZK_OK;
  if (!A || !B || !C) return OZK_EINVAL;
  size_t need = 0;
  ozk_int4int8gemm_fp4awe_workspace_size(m, n, k, &need);
  if (!workspace || workspace_bytes < need) return OZK_EWORKSPACE;
  if (!aligned(workspace, 256)) return OZK_EINVAL;
  const int64_t line = awe4_line_bytes(k);
  Carver cv(workspace);
  uint8_t* pa = static_cast<uint8_t*>(cv.take((size_t)m * line));
  uint8_t* pb = static_cast<uint8_t*>(cv.take((size_t)n * line));
  hipStream_t s = as_stream(stream);
  int st;
  if ((st = launch_awe4_pack(A, m, k, lda, 0, 1, pa, line, s))) return st;
  if ((st = launch_awe4_pack(B, k, n, ldb, 1, 0, pb, line, s))) return st;
  return launch_awe4_gemm(m, n, line / 128, pa, line, pb, line, C, ldc, s);
}

}  // extern "C"

// ---------------------------------------------------------------- emulated SpMV (CSR)
namespace {

struct SpmvLayout {
  size_t x_res, x_exp, x_partial, res, row_exps;
  size_t total() const {
    return align256(x_res) + align256(x_exp) + align256(x_partial) + align256(res) +
           align256(row_exps);
  }
};

SpmvLayout spmv_layout(int64_t rows, int64_t cols, int r) {
  SpmvLayout L;
  L.x_res = (size_t)cols * (r <= 16 ? 16 : 32);
  L.x_exp = 4;
  L.x_partial = (size_t)((cols + 2047) / 2048) * 8;
  L.res = (size_t)r * rows;
  L.row_exps = (size_t)rows * 4;
  return L;
}

}  // namespace

extern "C" {

int ozk_spmv_csr_workspace_size(int64_t rows, int64_t cols, int r, size_t* bytes) {
  if (!bytes || rows < 0 || cols < 1 || check_r(r) != OZK_OK) return OZK_EINVAL;
  *bytes = spmv_layout(rows, cols, r).total();
  return OZK_OK;
}

int ozk_spmv_csr(int64_t rows, int64_t cols, int64_t nnz, const int32_t* row_ptr,
                 const int32_t* col_idx, const double* vals, int64_t max_row_nnz,
                 const double* x, double* y, int r, void* workspace, size_t workspace_bytes,
                 void* stream) {
  if (check_r(r) != OZK_OK) return OZK_EINVAL;
  if (rows < 0 || cols < 1 || nnz < 0 || max_row_nnz < 1) return OZK_EINVAL;
  if (nnz > 0x7fffffffll || rows > 0x7ffffffell || cols > 0x7fffffffll) return OZK_EUNSUPPORTED;
  if (max_row_nnz > OZK_MAX_K) return OZK_ERANGE;
  int pa = 0, pb = 0;
  int st = scaling_bits(r, max_row_nnz, &pa, &pb);
  if (st != OZK_OK) return st;
  if (rows == 0) return OZK_OK;
  if (!row_ptr || !x || !y || (nnz > 0 && (!col_idx || !vals))) return OZK_EINVAL;
  const SpmvLayout L = spmv_layout(rows, cols, r);
  if (!workspace || workspace_bytes < L.total()) return OZK_EWORKSPACE;
  if (!aligned(workspace, 256)) return OZK_EINVAL;
  Carver cv(workspace);
  int8_t* x_res = static_cast<int8_t*>(cv.take(L.x_res));
  int32_t* x_exp = static_cast<int32_t*>(cv.take(L.x_exp));
  uint64_t* x_partial = static_cast<uint64_t*>(cv.take(L.x_partial));
  int8_t* res = static_cast<int8_t*>(cv.take(L.res));
  int32_t* row_exps = static_cast<int32_t*>(cv.take(L.row_exps));
  hipStream_t s = as_stream(stream);
  if ((st = launch_spmv(rows, cols, nnz, row_ptr, col_idx, vals, max_row_nnz, x, r, pa, pb,
                        x_partial, x_exp, x_res, res, row_exps, s)))
    return st;
  // y as a 1 x rows matrix: output j scaled by x's exponent plus row j's
  return launch_crt(1, rows, r, res, 0, rows, rows, x_exp, row_exps, y, rows, s);
}

}  // extern "C"

// ---------------------------------------------------------------- emulated DGEMM: epilogue
namespace {

bool act_ok(int act) { return act >= OZK_ACT_NONE && act <= OZK_ACT_SILU; }

// A product of the epilogue's or the gradient's: `left` (its lines along left_axis) times
// `right`, inner dimension K, rows x cols outputs.
struct Product {
  int64_t rows, cols, K;
  const double* left;
  int64_t left_rows, left_cols, ldl;
  int left_axis;
  const double* right;
  int64_t right_rows, right_cols, ldr;
  int right_axis;
  int64_t least_np = 0;   // a row of residues holds as many at least
};

// Workspace of a product.  The rows of residues are padded to 64 so that every store of the
// modular products and every load of the reconstruction is a whole vector (1500 x 2050 x
// 1001: 133.6 -> 68 us a product); the padding's columns are products with whatever lines
// follow the right planes, which therefore end in as many lines more.
struct ProductLayout {
  int64_t kp, np;
  size_t planes_l, planes_r, residues, exps_l, exps_r, scr_l, scr_r;
  size_t total() const {
    return align256(planes_l) + align256(planes_r) + align256(residues) + align256(exps_l) +
           align256(exps_r) + align256(scr_l) + align256(scr_r);
  }
};

ProductLayout product_layout(const Product& P, int r) {
  ProductLayout L;
  L.kp = round_up(P.K, 2 * kPlaneK);
  L.np = round_up(P.cols, 64);
  if (L.np < P.least_np) L.np = P.least_np;
  L.planes_l = (size_t)r * P.rows * L.kp;
  L.planes_r = ((size_t)r * P.cols + (L.np - P.cols)) * L.kp;
  L.residues = (size_t)r * P.rows * L.np;
  L.exps_l = (size_t)P.rows * 4;
  L.exps_r = (size_t)P.cols * 4;
  L.scr_l = deconstruct_scratch(P.left_rows, P.left_cols, P.left_axis);
  L.scr_r = deconstruct_scratch(P.right_rows, P.right_cols, P.right_axis);
  return L;
}

bool small(const Product& P) {
  return small_operands(P.rows > P.cols ? P.rows : P.cols, P.K,
                        P.left_axis == 1 && P.right_axis == 1);
}

// Whether a gradient's two products are run as one: small ones, and those of which one list of
// tiles is estimated to save 15 %, if what both hold stays in the last-level cache of 256 MB.
// Whole gradients, r = 16, one after the other and as one, us: 1500 x 2050 x 1001 253 and 239,
// 900 x 1500 x 1300 175 and 159, 700 x 1400 x 2000 (r = 14) 176 and 156.  Where 2 % are to be
// saved the two differ by 2 % either way; 5000 x 600 x 500 (12 % to be saved) took 211 and 220.
// Past the cache the first product's residues are gone before they are reconstructed: 2048^3,
// 439 MB, 413 and 456.
bool joined(const Product& a, const Product& b, int r) {
  if (small(a) && small(b)) return true;
  const ProductLayout la = product_layout(a, r), lb = product_layout(b, r);
  if (la.total() + lb.total() > (size_t)256 << 20) return false;
  const PlaneProduct both[2] = {{a.rows, a.cols, la.np, la.kp, nullptr, nullptr, nullptr},
                                {b.rows, b.cols, lb.np, lb.kp, nullptr, nullptr, nullptr}};
  const double apart = products_time(both, 1, r) + products_time(both + 1, 1, r);
  return products_time(both, 2, r) < 0.85 * apart;
}

// A product in its workspace, and what becomes of it.
struct Job {
  Product P;
  DgemmEpilogue E;
  double* out;
  int64_t ldo;
  bool gated = false;   // out: P.cols / 2 columns
  ProductLayout L{};
  int8_t *pl = nullptr, *pr = nullptr, *res = nullptr;
  int32_t *el = nullptr, *er = nullptr;
  void *scr_l = nullptr, *scr_r = nullptr;
  void place(Carver& cv, int r) {
    L = product_layout(P, r);
    pl = static_cast<int8_t*>(cv.take(L.planes_l));
    pr = static_cast<int8_t*>(cv.take(L.planes_r));
    res = static_cast<int8_t*>(cv.take(L.residues));
    el = static_cast<int32_t*>(cv.take(L.exps_l));
    er = static_cast<int32_t*>(cv.take(L.exps_r));
    scr_l = cv.take(L.scr_l);
    scr_r = cv.take(L.scr_r);
  }
  int reconstruct(int r, hipStream_t s) const {
    if (gated)
      return launch_crt_gated(P.rows, P.cols / 2, r, res, L.np, P.rows * L.np, el, er, E, out, ldo,
                              s);
    return launch_crt_epilogue(P.rows, P.cols, r, res, L.np, P.rows * L.np, el, er, E, out, ldo,
                               s);
  }
};

// One or two products in emulated fp64, each with its epilogue.  Small ones run together, each
// in a workspace of its own (in `workspace` one after the other), and so do those that `joined`
// names if `bytes` of workspace hold both; others one after the other, over the same workspace.
int run_jobs(Job* jobs, int count, int r, int scaling, void* workspace, size_t bytes,
             hipStream_t s) {
  int st, wl = 0, wr = 0;
  bool together = true;
  for (int i = 0; i < count; ++i) together = together && small(jobs[i].P);
  // two are the gradient's, without an epilogue
  const auto finish_two = [&](const PlaneProduct* prod) -> int {
    if (const int e = launch_products(prod, 2, r, s)) return e;
    const int32_t* const ea[2] = {jobs[0].el, jobs[1].el};
    const int32_t* const eb[2] = {jobs[0].er, jobs[1].er};
    double* const out[2] = {jobs[0].out, jobs[1].out};
    const int64_t ldo[2] = {jobs[0].ldo, jobs[1].ldo};
    return launch_crt_pair(prod, r, ea, eb, out, ldo, s);
  };
  if (together) {
    SmallOperand op[kSmallOperands];
    PlaneProduct prod[2];
    int64_t kp[kSmallOperands];
    Carver cv(workspace);
    for (int i = 0; i < count; ++i) {
      Job& J = jobs[i];
      const Product& P = J.P;
      if ((st = scaling_widths(scaling, r, P.K, &wl, &wr))) return st;
      J.place(cv, r);
      op[2 * i] = {P.left, P.rows, P.K, P.ldl, P.left_axis, wl, 0, J.pl, J.el};
      op[2 * i + 1] = {P.right, P.cols, P.K, P.ldr, P.right_axis, wr, 0, J.pr, J.er};
      kp[2 * i] = kp[2 * i + 1] = J.L.kp;
      prod[i] = {P.rows, P.cols, J.L.np, J.L.kp, J.pl, J.pr, J.res};
    }
    if ((st = launch_small_deconstruct(op, 2 * count, r, scaling, kp, s))) return st;
    if (count == 2) return finish_two(prod);
    if ((st = launch_products(prod, count, r, s))) return st;
    return jobs[0].reconstruct(r, s);
  }
  const bool join = count == 2 && joined(jobs[0].P, jobs[1].P, r) &&
                    product_layout(jobs[0].P, r).total() +
                            product_layout(jobs[1].P, r).total() <= bytes;
  PlaneProduct prod[2];
  Carver cv(workspace);
  for (int i = 0; i < count; ++i) {
    Job& J = jobs[i];
    const Product& P = J.P;
    if ((st = scaling_widths(scaling, r, P.K, &wl, &wr))) return st;
    if (!join) cv = Carver(workspace);
    J.place(cv, r);
    const int64_t sl = P.rows * J.L.kp, sr = P.cols * J.L.kp;   // plane strides
    if (small(P)) {
      const SmallOperand op[2] = {{P.left, P.rows, P.K, P.ldl, P.left_axis, wl, 0, J.pl, J.el},
                                  {P.right, P.cols, P.K, P.ldr, P.right_axis, wr, 0, J.pr, J.er}};
      const int64_t kp[2] = {J.L.kp, J.L.kp};
      st = launch_small_deconstruct(op, 2, r, scaling, kp, s);
    } else if (P.left_axis == 0 && P.right_axis == 1) {
      st = deconstruct_operands(P.left, P.rows, P.K, P.ldl, P.right, P.cols, P.ldr, r, scaling,
                                wl, wr, J.pl, J.pr, J.L.kp, J.el, J.er, J.scr_l, J.scr_r, s);
    } else {
      st = deconstruct_impl(P.left, P.left_rows, P.left_cols, P.ldl, P.left_axis, r, scaling, wl,
                            J.pl, J.L.kp, sl, J.el, J.scr_l, s);
      if (st == OZK_OK)
        st = deconstruct_impl(P.right, P.right_rows, P.right_cols, P.ldr, P.right_axis, r,
                              scaling, wr, J.pr, J.L.kp, sr, J.er, J.scr_r, s);
    }
    if (st != OZK_OK) return st;
    prod[i] = {P.rows, P.cols, J.L.np, J.L.kp, J.pl, J.pr, J.res};
    if (join) continue;
    if ((st = launch_products(&prod[i], 1, r, s))) return st;
    if ((st = J.reconstruct(r, s))) return st;
  }
  return join ? finish_two(prod) : OZK_OK;
}

// C = A B: rows of A against columns of B.
Product forward_product(int64_t m, int64_t n, int64_t k, const double* A, int64_t lda,
                        const double* B, int64_t ldb) {
  return {m, n, k, A, m, k, lda, 0, B, k, n, ldb, 1};
}

// The same for both projections of a gated block, B k x 2 n: the reconstruction reads whole groups
// of 64 residues from column 0 and from column n on.
Product gated_product(int64_t m, int64_t n, int64_t k, const double* A, int64_t lda,
                      const double* B, int64_t ldb) {
  Product P = forward_product(m, 2 * n, k, A, lda, B, ldb);
  P.least_np = 2 * round_up(n, 64);
  return P;
}

// dA = G B^T: rows of G against rows of B; dB = A^T G: columns of A against columns of G.
Product grad_a(int64_t m, int64_t n, int64_t k, const double* g, int64_t ldg,
                   const double* B, int64_t ldb) {
  return {m, k, n, g, m, n, ldg, 0, B, k, n, ldb, 0};
}
Product grad_b(int64_t m, int64_t n, int64_t k, const double* A, int64_t lda,
                   const double* g, int64_t ldg) {
  return {k, n, m, A, m, k, lda, 1, g, m, n, ldg, 1};
}

// Workspace of the gradient: G, the chunks' sums of its columns, and the two products' (side
// by side where they run together, else the larger one).  Of products that are not small the
// larger one's is enough (least): then they run one after the other.
struct EpilogueGradLayout {
  size_t g, part, products, least_products;
  size_t before() const { return align256(g) + align256(part); }   // the products'
  size_t total() const { return before() + align256(products); }
  size_t least() const { return before() + align256(least_products); }
};

EpilogueGradLayout epilogue_grad_layout(int64_t m, int64_t n, int64_t k, int r) {
  EpilogueGradLayout L;
  L.g = (size_t)m * n * 8;
  L.part = (size_t)act_grad_chunks(m > 0 ? m : 1) * n * 8;
  const Product pa = grad_a(m, n, k, nullptr, n, nullptr, n);
  const Product pb = grad_b(m, n, k, nullptr, k, nullptr, n);
  const size_t a = product_layout(pa, r).total(), b = product_layout(pb, r).total();
  L.least_products = small(pa) && small(pb) ? a + b : (a > b ? a : b);
  L.products = joined(pa, pb, r) ? a + b : L.least_products;
  return L;
}

}  // namespace

extern "C" {

int ozk_dgemm_epilogue_workspace_size(int64_t m, int64_t n, int64_t k, int r, size_t* bytes) {
  if (!bytes || m < 0 || n < 0 || k < 1 || check_r(r) != OZK_OK) return OZK_EINVAL;
  if (k > OZK_MAX_K) return OZK_ERANGE;
  *bytes = product_layout(forward_product(m, n, k, nullptr, k, nullptr, n), r).total();
  return OZK_OK;
}

int ozk_dgemm_epilogue(int64_t m, int64_t n, int64_t k, const double* A, int64_t lda,
                       const double* B, int64_t ldb, const double* bias, int act,
                       const double* residual, int64_t ldr, double* Z, int64_t ldz, double* C,
                       int64_t ldc, int r, int scaling, void* workspace, size_t workspace_bytes,
                       void* stream) {
  if (check_r(r) != OZK_OK || !act_ok(act)) return OZK_EINVAL;
  if (scaling != OZK_SCALING_MAX && scaling != OZK_SCALING_NORM) return OZK_EINVAL;
  if (m < 0 || n < 0 || k < 1) return OZK_EINVAL;
  if (k > OZK_MAX_K) return OZK_ERANGE;
  const int64_t n1 = n > 0 ? n : 1;
  if (lda < k || ldb < n1 || ldc < n1 || (residual && ldr < n1) || (Z && ldz < n1))
    return OZK_EINVAL;
  int wa = 0, wb = 0;
  int st = scaling_widths(scaling, r, k, &wa, &wb);
  if (st != OZK_OK) return st;
  if (m == 0 || n == 0) return OZK_OK;
  if (!A || !B || !C) return OZK_EINVAL;
  const Product P = forward_product(m, n, k, A, lda, B, ldb);
  if (!workspace || workspace_bytes < product_layout(P, r).total()) return OZK_EWORKSPACE;
  if (!aligned(workspace, 256)) return OZK_EINVAL;
  if ((size_t)m * n > (size_t)0x7fffffffffffull) return OZK_EUNSUPPORTED;
  Job job{P, {bias, residual, ldr, Z, ldz, act}, C, ldc};
  return run_jobs(&job, 1, r, scaling, workspace, workspace_bytes, as_stream(stream));
}

int ozk_dgemm_epilogue_grad_workspace_size(int64_t m, int64_t n, int64_t k, int r,
                                           size_t* bytes) {
  if (!bytes || m < 0 || n < 0 || k < 1 || check_r(r) != OZK_OK) return OZK_EINVAL;
  if (m > OZK_MAX_K || n > OZK_MAX_K || k > OZK_MAX_K) return OZK_ERANGE;
  *bytes = epilogue_grad_layout(m, n, k, r).total();
  return OZK_OK;
}

int ozk_dgemm_epilogue_grad(int64_t m, int64_t n, int64_t k, const double* dC, int64_t lddc,
                            const double* A, int64_t lda, const double* B, int64_t ldb,
                            const double* Z, int64_t ldz, int act, double* dA, int64_t ldda,
                            double* dB, int64_t lddb, double* dbias, int r, int scaling,
                            void* workspace, size_t workspace_bytes, void* stream) {
  if (check_r(r) != OZK_OK || !act_ok(act)) return OZK_EINVAL;
  if (scaling != OZK_SCALING_MAX && scaling != OZK_SCALING_NORM) return OZK_EINVAL;
  if (m < 0 || n < 0 || k < 1) return OZK_EINVAL;
  if (m > OZK_MAX_K || n > OZK_MAX_K || k > OZK_MAX_K) return OZK_ERANGE;
  const int64_t n1 = n > 0 ? n : 1;
  if (lddc < n1 || (act != OZK_ACT_NONE && ldz < n1)) return OZK_EINVAL;
  if ((dA && (ldda < k || ldb < n1)) || (dB && (lddb < n1 || lda < k))) return OZK_EINVAL;
  int wa = 0, wb = 0, st;
  if (m == 0 || n == 0) {   // sums of no terms
    hipStream_t s = as_stream(stream);
    if (m > 0 && dA && (st = launch_zero_rows(dA, m, k, ldda, s))) return st;
    if (n > 0 && dB && (st = launch_zero_rows(dB, k, n, lddb, s))) return st;
    if (n > 0 && dbias && (st = launch_zero_rows(dbias, 1, n, n, s))) return st;
    return OZK_OK;
  }
  if (dA && (st = scaling_widths(scaling, r, n, &wa, &wb))) return st;
  if (dB && (st = scaling_widths(scaling, r, m, &wa, &wb))) return st;
  if (!dA && !dB && !dbias) return OZK_OK;
  if (!dC || (act != OZK_ACT_NONE && !Z) || (dA && !B) || (dB && !A)) return OZK_EINVAL;
  const EpilogueGradLayout L = epilogue_grad_layout(m, n, k, r);
  if (!workspace || workspace_bytes < L.least()) return OZK_EWORKSPACE;
  if (!aligned(workspace, 256)) return OZK_EINVAL;
  Carver cv(workspace);
  double* g = static_cast<double*>(cv.take(L.g));
  double* part = static_cast<double*>(cv.take(L.part));
  const size_t room = workspace_bytes - L.before();
  void* products = cv.take(room);
  hipStream_t s = as_stream(stream);
  // without an activation G is dC itself
  const bool own_g = act != OZK_ACT_NONE && (dA || dB);
  if ((own_g || dbias) &&
      (st = launch_act_grad(m, n, dC, lddc, Z, ldz, act, own_g ? g : nullptr, part, dbias, s)))
    return st;
  const double* gp = own_g ? g : dC;
  const int64_t ldg = own_g ? n : lddc;
  const DgemmEpilogue none{nullptr, nullptr, 0, nullptr, 0, OZK_ACT_NONE};
  Job jobs[2];
  int count = 0;
  if (dA) jobs[count++] = Job{grad_a(m, n, k, gp, ldg, B, ldb), none, dA, ldda};
  if (dB) jobs[count++] = Job{grad_b(m, n, k, A, lda, gp, ldg), none, dB, lddb};
  return count ? run_jobs(jobs, count, r, scaling, products, room, s) : OZK_OK;
}

// ---------------------------------------------------------------- gated block in emulated fp64
int ozk_dgemm_gated_workspace_size(int64_t m, int64_t n, int64_t k, int r, size_t* bytes) {
  if (!bytes || m < 0 || n < 0 || k < 1 || check_r(r) != OZK_OK) return OZK_EINVAL;
  if (k > OZK_MAX_K) return OZK_ERANGE;
  if (n >= (int64_t)1 << 40) return OZK_EUNSUPPORTED;
  *bytes = product_layout(gated_product(m, n, k, nullptr, k, nullptr, 2 * n), r).total();
  return OZK_OK;
}

int ozk_dgemm_gated(int64_t m, int64_t n, int64_t k, const double* A, int64_t lda, const double* B,
                    int64_t ldb, const double* bias, int act, double* Z, int64_t ldz, double* C,
                    int64_t ldc, int r, int scaling, void* workspace, size_t workspace_bytes,
                    void* stream) {
  if (check_r(r) != OZK_OK || !act_ok(act)) return OZK_EINVAL;
  if (scaling != OZK_SCALING_MAX && scaling != OZK_SCALING_NORM) return OZK_EINVAL;
  if (m < 0 || n < 0 || k < 1) return OZK_EINVAL;
  if (k > OZK_MAX_K) return OZK_ERANGE;
  if (n >= (int64_t)1 << 40) return OZK_EUNSUPPORTED;
  const int64_t n1 = n > 0 ? n : 1;
  if (lda < k || ldb < 2 * n1 || ldc < n1 || (Z && ldz < 2 * n1)) return OZK_EINVAL;
  int wa = 0, wb = 0;
  int st = scaling_widths(scaling, r, k, &wa, &wb);
  if (st != OZK_OK) return st;
  if (m == 0 || n == 0) return OZK_OK;
  if (!A || !B || !C) return OZK_EINVAL;
  const Product P = gated_product(m, n, k, A, lda, B, ldb);
  if (!workspace || workspace_bytes < product_layout(P, r).total()) return OZK_EWORKSPACE;
  if (!aligned(workspace, 256)) return OZK_EINVAL;
  if ((size_t)m * n > (size_t)0x3fffffffffffull) return OZK_EUNSUPPORTED;
  Job job{P, {bias, nullptr, 0, Z, ldz, act}, C, ldc, true};
  return run_jobs(&job, 1, r, scaling, workspace, workspace_bytes, as_stream(stream));
}

int ozk_dgemm_gated_grad_workspace_size(int64_t m, int64_t n, int64_t k, int r, size_t* bytes) {
  if (n > OZK_MAX_K / 2) return bytes && m >= 0 && k >= 1 && check_r(r) == OZK_OK ? OZK_ERANGE
                                                                                  : OZK_EINVAL;
  return ozk_dgemm_epilogue_grad_workspace_size(m, 2 * n, k, r, bytes);
}

int ozk_dgemm_gated_grad(int64_t m, int64_t n, int64_t k, const double* dC, int64_t lddc,
                         const double* A, int64_t lda, const double* B, int64_t ldb,
                         const double* Z, int64_t ldz, int act, double* dA, int64_t ldda,
                         double* dB, int64_t lddb, double* dbias, int r, int scaling,
                         void* workspace, size_t workspace_bytes, void* stream) {
  if (check_r(r) != OZK_OK || !act_ok(act)) return OZK_EINVAL;
  if (scaling != OZK_SCALING_MAX && scaling != OZK_SCALING_NORM) return OZK_EINVAL;
  if (m < 0 || n < 0 || k < 1) return OZK_EINVAL;
  if (m > OZK_MAX_K || n > OZK_MAX_K / 2 || k > OZK_MAX_K) return OZK_ERANGE;
  const int64_t n1 = n > 0 ? n : 1, w = 2 * n;
  if (lddc < n1 || ldz < 2 * n1) return OZK_EINVAL;
  if ((dA && (ldda < k || ldb < 2 * n1)) || (dB && (lddb < 2 * n1 || lda < k))) return OZK_EINVAL;
  int wa = 0, wb = 0, st;
  hipStream_t s = as_stream(stream);
  if (m == 0 || n == 0) {   // sums of no terms
    if (m > 0 && dA && (st = launch_zero_rows(dA, m, k, ldda, s))) return st;
    if (n > 0 && dB && (st = launch_zero_rows(dB, k, w, lddb, s))) return st;
    if (n > 0 && dbias && (st = launch_zero_rows(dbias, 1, w, w, s))) return st;
    return OZK_OK;
  }
  if (dA && (st = scaling_widths(scaling, r, w, &wa, &wb))) return st;
  if (dB && (st = scaling_widths(scaling, r, m, &wa, &wb))) return st;
  if (!dA && !dB && !dbias) return OZK_OK;
  if (!dC || !Z || (dA && !B) || (dB && !A)) return OZK_EINVAL;
  const EpilogueGradLayout L = epilogue_grad_layout(m, w, k, r);
  if (!workspace || workspace_bytes < L.least()) return OZK_EWORKSPACE;
  if (!aligned(workspace, 256)) return OZK_EINVAL;
  Carver cv(workspace);
  double* g = static_cast<double*>(cv.take(L.g));
  double* part = static_cast<double*>(cv.take(L.part));
  const size_t room = workspace_bytes - L.before();
  void* products = cv.take(room);
  if ((st = launch_gate_grad(m, n, dC, lddc, Z, ldz, act, dA || dB ? g : nullptr, part, dbias, s)))
    return st;
  const DgemmEpilogue none{nullptr, nullptr, 0, nullptr, 0, OZK_ACT_NONE};
  Job jobs[2];
  int count = 0;
  if (dA) jobs[count++] = Job{grad_a(m, w, k, g, w, B, ldb), none, dA, ldda};
  if (dB) jobs[count++] = Job{grad_b(m, w, k, A, lda, g, w), none, dB, lddb};
  return count ? run_jobs(jobs, count, r, scaling, products, room, s) : OZK_OK;
}

// ---------------------------------------------------------------- int8 linear layer
int ozk_int8linear_workspace_size(int64_t m, int64_t n, int64_t k, int aligned, size_t* bytes) {
  if (!bytes || m < 0 || n < 0 || k < 1 || (aligned != 0 && aligned != 1)) return OZK_EINVAL;
  if (k > OZK_MAX_K) return OZK_ERANGE;
  if (m > 0x7fffffffll || n > 0x7fffffffll) return OZK_EUNSUPPORTED;
  // operands of a K that allows it may be aligned, and run in another way than unaligned ones
  const size_t tiled = k % 16 == 0 ? int8linear_workspace(m, n, k, true) : 0;
  const size_t any = int8linear_workspace(m, n, k, false);
  *bytes = k % 16 == 0 && (aligned || tiled > any) ? tiled : any;
  return OZK_OK;
}

int ozk_int8linear(int64_t m, int64_t n, int64_t k, const int8_t* X, int64_t ldx,
                   const float* scale_x, const int8_t* W, int64_t ldw, const float* scale_w,
                   const void* bias, int act, const void* residual, int64_t ldr, int type,
                   void* C, int64_t ldc, void* workspace, size_t workspace_bytes, void* stream) {
  if (!act_ok(act) || (type != OZK_F32 && type != OZK_F16 && type != OZK_BF16))
    return OZK_EINVAL;
  if (m < 0 || n < 0 || k < 1) return OZK_EINVAL;
  if (k > OZK_MAX_K) return OZK_ERANGE;
  const int64_t n1 = n > 0 ? n : 1;
  if (ldx < k || ldw < k || ldc < n1 || (residual && ldr < n1)) return OZK_EINVAL;
  if (m == 0 || n == 0) return OZK_OK;
  if (!X || !scale_x || !W || !scale_w || !C) return OZK_EINVAL;
  const size_t e = type == OZK_F32 ? 4 : 2;
  if (!aligned(scale_x, 4) || !aligned(scale_w, 4) || !aligned(bias, e) ||
      !aligned(residual, e) || !aligned(C, e))
    return OZK_EINVAL;
  if (m > 0x7fffffffll || n > 0x7fffffffll) return OZK_EUNSUPPORTED;
  const size_t need = int8linear_workspace(m, n, k, int8linear_aligned(X, ldx, W, ldw, k));
  if (need > workspace_bytes || (need > 0 && !workspace)) return OZK_EWORKSPACE;
  if (need > 0 && !aligned(workspace, 256)) return OZK_EINVAL;
  return launch_int8linear(m, n, k, X, ldx, scale_x, W, ldw, scale_w, bias, act, residual, ldr,
                           type, C, ldc, workspace, as_stream(stream));
}

// ---------------------------------------------------------------- rows: codes, layer norm
static int check_rows(int64_t rows, int64_t cols, int type) {
  if (type < OZK_F64 || type > OZK_BF16 || rows < 0 || cols < 1) return OZK_EINVAL;
  if (rows > 0x7fffffffll || cols > 0x7fffffffll) return OZK_EUNSUPPORTED;
  return OZK_OK;
}
static size_t type_size(int type) { return type == OZK_F64 ? 8 : type == OZK_F32 ? 4 : 2; }

int ozk_int8quant_rows(int64_t rows, int64_t cols, int type, const void* x, int64_t ldx, int norm,
                       const void* gamma, const void* beta, double eps, int8_t* q, int64_t ldq,
                       float* scale, void* stream) {
  int st = check_rows(rows, cols, type);
  if (st != OZK_OK) return st;
  if ((norm != 0 && norm != 1) || ldx < cols || ldq < cols) return OZK_EINVAL;
  if (norm ? !(eps >= 0.0) : (gamma != nullptr || beta != nullptr)) return OZK_EINVAL;
  if (rows == 0) return OZK_OK;
  const size_t e = type_size(type);
  if (!x || !q || !scale || !aligned(x, e) || !aligned(gamma, e) || !aligned(beta, e) ||
      !aligned(scale, 4))
    return OZK_EINVAL;
  return launch_int8quant(rows, cols, type, x, ldx, norm, gamma, beta, eps, q, ldq, scale,
                          as_stream(stream));
}

int ozk_layernorm(int64_t rows, int64_t cols, int type, const void* x, int64_t ldx,
                  const void* gamma, const void* beta, double eps, void* y, int64_t ldy,
                  void* mean, void* rstd, void* stream) {
  int st = check_rows(rows, cols, type);
  if (st != OZK_OK) return st;
  if (ldx < cols || ldy < cols || !(eps >= 0.0)) return OZK_EINVAL;
  if (rows == 0) return OZK_OK;
  const size_t e = type_size(type), a = e > 4 ? e : 4;
  if (!x || !y || !aligned(x, e) || !aligned(y, e) || !aligned(gamma, e) || !aligned(beta, e) ||
      !aligned(mean, a) || !aligned(rstd, a))
    return OZK_EINVAL;
  return launch_layernorm(rows, cols, type, x, ldx, gamma, beta, eps, y, ldy, mean, rstd,
                          as_stream(stream));
}

int ozk_layernorm_backward_workspace_size(int64_t rows, int64_t cols, int type, size_t* bytes) {
  if (!bytes) return OZK_EINVAL;
  int st = check_rows(rows, cols, type);
  if (st != OZK_OK) return st;
  *bytes = align256((size_t)layernorm_backward_groups(rows) * 2 * cols *
                    (type == OZK_F64 ? 8 : 4));
  return OZK_OK;
}

int ozk_layernorm_backward(int64_t rows, int64_t cols, int type, const void* dy, int64_t lddy,
                           const void* x, int64_t ldx, const void* gamma, const void* mean,
                           const void* rstd, void* dx, int64_t lddx, void* dgamma, void* dbeta,
                           void* workspace, size_t workspace_bytes, void* stream) {
  size_t need = 0;
  int st = ozk_layernorm_backward_workspace_size(rows, cols, type, &need);
  if (st != OZK_OK) return st;
  if (ldx < cols || lddy < cols || (dx && lddx < cols)) return OZK_EINVAL;
  const size_t e = type_size(type), a = e > 4 ? e : 4;
  if (rows > 0 && (!dy || !x || !mean || !rstd)) return OZK_EINVAL;
  if (!aligned(dy, e) || !aligned(x, e) || !aligned(gamma, e) || !aligned(mean, a) ||
      !aligned(rstd, a) || !aligned(dx, e) || !aligned(dgamma, e) || !aligned(dbeta, e))
    return OZK_EINVAL;
  if (rows == 0) dx = nullptr;   // the sums over no rows are zero
  if (!dx && !dgamma && !dbeta) return OZK_OK;
  if (rows > 0 && (dgamma || dbeta)) {
    if (!workspace || workspace_bytes < need) return OZK_EWORKSPACE;
    if (!aligned(workspace, 256)) return OZK_EINVAL;
  }
  return launch_layernorm_backward(rows, cols, type, dy, lddy, x, ldx, gamma, mean, rstd, dx,
                                   lddx, dgamma, dbeta, workspace, as_stream(stream));
}

// ---------------------------------------------------------------- MX FP4
int64_t ozk_mxfp4_line_bytes(int64_t k) { return k > 0 ? (k + 255) / 256 * 128 : 0; }
int64_t ozk_mxfp4_scale_bytes(int64_t k) { return k > 0 ? (k + 255) / 256 * 8 : 0; }

// Lines of codes and scales over k values as the kernels read and write them.
static bool lines_ok(int64_t k, const void* codes, int64_t ldq, const void* scales, int64_t lds) {
  return codes && scales && aligned(codes, 16) && aligned(scales, 8) && ldq % 16 == 0 &&
         lds % 8 == 0 && ldq >= ozk_mxfp4_line_bytes(k) && lds >= ozk_mxfp4_scale_bytes(k);
}

int ozk_mxfp4_quant(int64_t rows, int64_t cols, int type, const void* x, int64_t ldx, int axis,
                    uint8_t* codes, int64_t ldq, uint8_t* scales, int64_t lds, void* stream) {
  if (type < OZK_F64 || type > OZK_BF16 || (axis != 0 && axis != 1)) return OZK_EINVAL;
  if (rows < 0 || cols < 0 || (axis ? rows : cols) < 1 || ldx < (cols > 0 ? cols : 1))
    return OZK_EINVAL;
  if (rows > 0x7fffffffll || cols > 0x7fffffffll) return OZK_EUNSUPPORTED;
  if (rows == 0 || cols == 0) return OZK_OK;
  if (!x || !aligned(x, type_size(type)) || !lines_ok(axis ? rows : cols, codes, ldq, scales, lds))
    return OZK_EINVAL;
  return launch_mxfp4_quant(rows, cols, type, x, ldx, axis, codes, ldq, scales, lds,
                            as_stream(stream));
}

int ozk_mxfp4_values(int64_t lines, int64_t k, const uint8_t* codes, int64_t ldq,
                     const uint8_t* scales, int64_t lds, int type, void* out, int64_t ldo,
                     void* stream) {
  if (type < OZK_F64 || type > OZK_BF16 || lines < 0 || k < 1 || ldo < k) return OZK_EINVAL;
  if (lines > 0x7fffffffll || k > 0x7fffffffll) return OZK_EUNSUPPORTED;
  if (lines == 0) return OZK_OK;
  if (!out || !aligned(out, type_size(type)) || !lines_ok(k, codes, ldq, scales, lds))
    return OZK_EINVAL;
  return launch_mxfp4_values(lines, k, codes, ldq, scales, lds, type, out, ldo, as_stream(stream));
}

// The checks of both products that depend on sizes alone.
static int check_mx(int64_t m, int64_t n, int64_t k) {
  if (m < 0 || n < 0 || k < 1) return OZK_EINVAL;
  if (k > OZK_MX_MAX_K) return OZK_ERANGE;
  if (m > 0x7fffffffll || n > 0x3fffffffll) return OZK_EUNSUPPORTED;
  return OZK_OK;
}

static int mx_workspace(int64_t m, int64_t n, int64_t k, bool gated, size_t* bytes) {
  if (!bytes) return OZK_EINVAL;
  const int st = check_mx(m, n, k);
  if (st == OZK_OK) *bytes = m > 0 && n > 0 ? mxfp4_linear_workspace(m, n, k, gated) : 0;
  return st;
}

static int mx_product(int64_t m, int64_t n, int64_t k, const uint8_t* X, int64_t ldx,
                      const uint8_t* scale_x, int64_t ldsx, const uint8_t* W, int64_t ldw,
                      const uint8_t* scale_w, int64_t ldsw, bool gated, const void* bias, int act,
                      const void* residual, int64_t ldr, int type, void* C, int64_t ldc,
                      void* workspace, size_t workspace_bytes, void* stream) {
  if (!act_ok(act) || (type != OZK_F32 && type != OZK_F16 && type != OZK_BF16)) return OZK_EINVAL;
  const int st = check_mx(m, n, k);
  if (st != OZK_OK) return st;
  const int64_t n1 = n > 0 ? n : 1;
  if (ldc < n1 || (residual && ldr < n1)) return OZK_EINVAL;
  if (m == 0 || n == 0) return OZK_OK;
  const size_t e = type == OZK_F32 ? 4 : 2;
  if (!lines_ok(k, X, ldx, scale_x, ldsx) || !lines_ok(k, W, ldw, scale_w, ldsw) || !C ||
      !aligned(bias, e) || !aligned(residual, e) || !aligned(C, e))
    return OZK_EINVAL;
  // a lane's offset within a tile is 32 bits
  const int64_t far = 1 << 24;
  if (ldx >= far || ldw >= far || ldsx >= far || ldsw >= far) return OZK_EUNSUPPORTED;
  const size_t need = mxfp4_linear_workspace(m, n, k, gated);
  if (need > workspace_bytes || (need > 0 && !workspace)) return OZK_EWORKSPACE;
  if (need > 0 && !aligned(workspace, 256)) return OZK_EINVAL;
  return launch_mxfp4_linear(m, n, k, X, ldx, scale_x, ldsx, W, ldw, scale_w, ldsw, gated, bias,
                             act, residual, ldr, type, C, ldc, workspace, as_stream(stream));
}

int ozk_mxfp4_linear_workspace_size(int64_t m, int64_t n, int64_t k, size_t* bytes) {
  return mx_workspace(m, n, k, false, bytes);
}

int ozk_mxfp4_linear(int64_t m, int64_t n, int64_t k, const uint8_t* X, int64_t ldx,
                     const uint8_t* scale_x, int64_t ldsx, const uint8_t* W, int64_t ldw,
                     const uint8_t* scale_w, int64_t ldsw, const void* bias, int act,
                     const void* residual, int64_t ldr, int type, void* C, int64_t ldc,
                     void* workspace, size_t workspace_bytes, void* stream) {
  return mx_product(m, n, k, X, ldx, scale_x, ldsx, W, ldw, scale_w, ldsw, false, bias, act,
                    residual, ldr, type, C, ldc, workspace, workspace_bytes, stream);
}

int ozk_mxfp4_gated_workspace_size(int64_t m, int64_t n, int64_t k, size_t* bytes) {
  return mx_workspace(m, n, k, true, bytes);
}

int ozk_mxfp4_gated(int64_t m, int64_t n, int64_t k, const uint8_t* X, int64_t ldx,
                    const uint8_t* scale_x, int64_t ldsx, const uint8_t* W, int64_t ldw,
                    const uint8_t* scale_w, int64_t ldsw, const void* bias, int act, int type,
                    void* C, int64_t ldc, void* workspace, size_t workspace_bytes, void* stream) {
  return mx_product(m, n, k, X, ldx, scale_x, ldsx, W, ldw, scale_w, ldsw, true, bias, act, nullptr,
                    0, type, C, ldc, workspace, workspace_bytes, stream);
}

// ---------------------------------------------------------------- clipping
int ozk_clip_norm_workspace_size(int64_t count, size_t* bytes) {
  if (!bytes || count < 0) return OZK_EINVAL;
  if (count > 0x7fffff) return OZK_EUNSUPPORTED;
  *bytes = clip_norm_workspace(count);
  return OZK_OK;
}

namespace {
struct Span {
  uintptr_t from, to;
  int64_t tensor;
  bool operator<(const Span& o) const { return from < o.from; }
};

// Whether an output, norm among them, overlaps another, or an input other than the one it is.
// spans: count + 1 of them.
bool clip_overlaps(int64_t count, const void* const* x, void* const* out, const int64_t* sizes,
                   const int* types, const double* norm, Span* spans) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(norm);
  int64_t n = 0;
  spans[n++] = {at, at + sizeof(double), -1};
  for (int64_t i = 0; i < count; ++i)
    if (sizes[i] > 0) {
      const uintptr_t p = reinterpret_cast<uintptr_t>(out[i]);
      spans[n++] = {p, p + sizes[i] * type_size(types[i]), i};
    }
  std::sort(spans, spans + n);
  for (int64_t i = 1; i < n; ++i)
    if (spans[i].from < spans[i - 1].to) return true;
  for (int64_t i = 0; i < count; ++i) {
    if (sizes[i] == 0) continue;
    const uintptr_t p = reinterpret_cast<uintptr_t>(x[i]), e = p + sizes[i] * type_size(types[i]);
    // the first output that ends past p (they are in order and apart)
    const Span* s = std::lower_bound(spans, spans + n, p,
                                     [](const Span& a, uintptr_t v) { return a.to <= v; });
    for (; s < spans + n && s->from < e; ++s)
      if (s->tensor != i || s->from != p) return true;
  }
  return false;
}
}  // namespace

int ozk_clip_norm(int64_t count, const void* const* x, void* const* out, const int64_t* sizes,
                  const int* types, double max_norm, double* norm, void* workspace,
                  size_t workspace_bytes, void* stream) {
  if (count < 0 || !(max_norm >= 0.0) || !norm || !aligned(norm, 8)) return OZK_EINVAL;
  if (count > 0x7fffff) return OZK_EUNSUPPORTED;
  if (count > 0 && (!x || !out || !sizes || !types)) return OZK_EINVAL;
  int64_t bytes = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (types[i] < OZK_F64 || types[i] > OZK_BF16 || sizes[i] < 0) return OZK_EINVAL;
    if (sizes[i] == 0) continue;
    const size_t e = type_size(types[i]);
    if (!x[i] || !out[i] || !aligned(x[i], e) || !aligned(out[i], e)) return OZK_EINVAL;
    // chunks are counted in 32 bits
    if (sizes[i] >= ((int64_t)1 << 44) / (int64_t)e) return OZK_EUNSUPPORTED;
    bytes += sizes[i] * e + 32768;
    if (bytes >= (int64_t)1 << 45) return OZK_EUNSUPPORTED;
  }
  const size_t need = clip_norm_workspace(count);
  if (need > workspace_bytes || (need > 0 && !workspace)) return OZK_EWORKSPACE;
  if (need > 0 && !aligned(workspace, 256)) return OZK_EINVAL;
  if (count > 0) {
    Span few[65];
    Span* spans = count <= 64 ? few : new (std::nothrow) Span[count + 1];
    if (!spans) return OZK_EUNSUPPORTED;
    const bool bad = clip_overlaps(count, x, out, sizes, types, norm, spans);
    if (spans != few) delete[] spans;
    if (bad) return OZK_EINVAL;
  }
  return launch_clip_norm(count, x, out, sizes, types, max_norm, norm, workspace,
                          as_stream(stream));
}

}  // extern "C"
