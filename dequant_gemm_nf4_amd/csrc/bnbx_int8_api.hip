// C entry points of libbnbx_int8 (declared in include/bnbx_int8.h): argument
// checks on the host and kernel launches.
#include "../../include/bnbx_int8.h"
#include "bnbx_int8.hpp"

namespace bnbx {
namespace {

bool aligned8(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

int status8(hipError_t e) {
  return e == hipSuccess ? BNBX_OK : e == hipErrorNotSupported ? BNBX_E_UNSUPPORTED : BNBX_E_HIP;
}

// `empty`: rows may be 0 (their buffers are then not looked at).
int check_rows8(const bnbx_int8_rows* q, bool empty) {
  if (q == nullptr || q->rows < 0 || q->cols < 1) return BNBX_E_INVAL;
  if (q->rows == 0 && !empty) return BNBX_E_INVAL;
  if (q->dtype != BNBX_DTYPE_BF16 && q->dtype != BNBX_DTYPE_F16) return BNBX_E_INVAL;
  if (q->ld < ((int64_t)q->cols + 15) / 16 * 16) return BNBX_E_INVAL;
  if (q->rows > 0 && (q->codes == nullptr || q->scale == nullptr)) return BNBX_E_INVAL;
  if (q->ld % 16 != 0 || !aligned8(q->codes, 16) || !aligned8(q->scale, 4)) return BNBX_E_ALIGN;
  if (q->ld >= ((int64_t)1 << 23)) return BNBX_E_UNSUPPORTED;   // a tile's rows in 31 bits
  return BNBX_OK;
}

// The products count rows to the end of a last tile in 31 bits.
bool too_many(int rows) { return rows > INT32_MAX - 511; }

// Whether bnbx_gemm_int8 and bnbx_linear_int8 have a launch for a product.
bool int8_gemm_takes(int M, int N, int K) {
  if (too_many(M) || too_many(N)) return false;
  return int8_few_takes(M, K) ? int8_few_fits(N) : int8_gemm_fits(M, N, K);
}

// Rows of `bytes`-wide values: `cols` of them at p + r * ld.
int check_matrix8(const void* p, int64_t ld, int64_t rows, int64_t cols, size_t bytes) {
  if (rows > 0 && p == nullptr) return BNBX_E_INVAL;
  if (ld < cols) return BNBX_E_INVAL;
  return aligned8(p, bytes) ? BNBX_OK : BNBX_E_ALIGN;
}

// Gradients, which the kernels copy in 16-byte pieces.
int check_dy8(const uint16_t* dy, int64_t ld, int64_t rows, int64_t cols) {
  const int s = check_matrix8(dy, ld, rows, cols, 16);
  if (s != BNBX_OK) return s;
  if (ld % 8 != 0) return BNBX_E_ALIGN;
  return ld >= ((int64_t)1 << 22) ? BNBX_E_UNSUPPORTED : BNBX_OK;   // a tile's rows in 31 bits
}

int check_workspace8(const void* ws, size_t bytes, size_t need) {
  if (need == 0) return BNBX_OK;
  if (ws == nullptr || bytes < need) return BNBX_E_WORKSPACE;
  return aligned8(ws, 16) ? BNBX_OK : BNBX_E_ALIGN;
}

Int8Rows rows8(const bnbx_int8_rows* q) {
  return Int8Rows{q->codes, q->scale, q->ld, q->rows, q->cols};
}

int64_t padded(int64_t cols) { return (cols + 15) / 16 * 16; }

// X's codes and scales at the start of a workspace.
size_t codes_bytes(int64_t M, int K) {
  return whole256((size_t)M * padded(K)) + whole256((size_t)M * sizeof(float));
}

}  // namespace

int int8_cus() {
  static const int n = [] {
    int dev = 0, v = 0;
    const bool ok = hipGetDevice(&dev) == hipSuccess &&
                    hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) ==
                        hipSuccess;
    return ok && v > 0 ? v : 256;
  }();
  return n;
}

}  // namespace bnbx

using namespace bnbx;

extern "C" {

int bnbx_quantize_rows_int8(const uint16_t* x, int64_t ldx, const bnbx_int8_rows* q,
                            void* stream) {
  int s = check_rows8(q, true);
  if (s != BNBX_OK) return s;
  s = check_matrix8(x, ldx, q->rows, q->cols, 2);
  if (s != BNBX_OK) return s;
  return status8(launch_quantize_rows(x, ldx, rows8(q), q->dtype == BNBX_DTYPE_F16,
                                      (hipStream_t)stream));
}

int bnbx_dequantize_rows_int8(const bnbx_int8_rows* q, uint16_t* out, int64_t ldo, void* stream) {
  int s = check_rows8(q, true);
  if (s != BNBX_OK) return s;
  s = check_matrix8(out, ldo, q->rows, q->cols, 2);
  if (s != BNBX_OK) return s;
  return status8(launch_dequantize_rows(rows8(q), out, ldo, q->dtype == BNBX_DTYPE_F16,
                                        (hipStream_t)stream));
}

size_t bnbx_gemm_int8_workspace_bytes(int M, int N, int K) {
  if (M < 1 || N < 1 || K < 1 || K > BNBX_INT8_MAX_COLS || int8_few_takes(M, K)) return 0;
  return int8_gemm_takes(M, N, K) ? int8_gemm_workspace(M, N, K) : 0;
}

int bnbx_gemm_int8(const bnbx_int8_rows* x, const bnbx_int8_rows* w, uint16_t* y, int64_t ldy,
                   void* workspace, size_t workspace_bytes, void* stream) {
  int s = check_rows8(x, true);
  if (s != BNBX_OK) return s;
  s = check_rows8(w, false);
  if (s != BNBX_OK) return s;
  if (x->cols != w->cols || x->dtype != w->dtype) return BNBX_E_INVAL;
  s = check_matrix8(y, ldy, x->rows, w->rows, 2);
  if (s != BNBX_OK) return s;
  if (x->cols > BNBX_INT8_MAX_COLS || !int8_gemm_takes(x->rows, w->rows, x->cols))
    return BNBX_E_UNSUPPORTED;
  if (x->rows == 0) return BNBX_OK;
  const bool f16 = x->dtype == BNBX_DTYPE_F16;
  if (int8_few_takes(x->rows, x->cols))
    return status8(launch_int8_few(nullptr, 0, rows8(x), rows8(w), y, ldy, f16,
                                   (hipStream_t)stream));
  s = check_workspace8(workspace, workspace_bytes, int8_gemm_workspace(x->rows, w->rows, x->cols));
  if (s != BNBX_OK) return s;
  return status8(launch_int8_gemm(rows8(x), rows8(w), y, ldy, f16,
                                  workspace, (hipStream_t)stream));
}

size_t bnbx_linear_int8_workspace_bytes(int M, int N, int K, int saved) {
  if (M < 1 || N < 1 || K < 1 || K > BNBX_INT8_MAX_COLS || int8_few_takes(M, K)) return 0;
  return (saved ? 0 : codes_bytes(M, K)) + int8_gemm_workspace(M, N, K);
}

int bnbx_linear_int8(const uint16_t* x, int64_t ldx, int M, const bnbx_int8_rows* w,
                     const bnbx_int8_rows* saved, uint16_t* y, int64_t ldy, void* workspace,
                     size_t workspace_bytes, void* stream) {
  int s = check_rows8(w, false);
  if (s != BNBX_OK) return s;
  const int N = w->rows, K = w->cols;
  if (M < 0) return BNBX_E_INVAL;
  s = check_matrix8(x, ldx, M, K, 2);
  if (s != BNBX_OK) return s;
  s = check_matrix8(y, ldy, M, N, 2);
  if (s != BNBX_OK) return s;
  if (saved != nullptr) {
    s = check_rows8(saved, true);
    if (s != BNBX_OK) return s;
    if (saved->rows != M || saved->cols != K || saved->dtype != w->dtype) return BNBX_E_INVAL;
  }
  if (K > BNBX_INT8_MAX_COLS || !int8_gemm_takes(M, N, K)) return BNBX_E_UNSUPPORTED;
  if (M == 0) return BNBX_OK;
  s = check_workspace8(workspace, workspace_bytes,
                       bnbx_linear_int8_workspace_bytes(M, N, K, saved != nullptr));
  if (s != BNBX_OK) return s;
  const bool f16 = w->dtype == BNBX_DTYPE_F16;
  Int8Rows q{nullptr, nullptr, 0, M, K};
  if (int8_few_takes(M, K)) {
    if (saved != nullptr) q = rows8(saved);
    return status8(launch_int8_few(x, ldx, q, rows8(w), y, ldy, f16, (hipStream_t)stream));
  }
  uint8_t* ws = (uint8_t*)workspace;
  if (saved != nullptr) {
    q = rows8(saved);
  } else {
    q = Int8Rows{(int8_t*)ws, (float*)(ws + whole256((size_t)M * padded(K))), padded(K), M, K};
    ws += codes_bytes(M, K);
  }
  const hipError_t e = launch_quantize_rows(x, ldx, q, f16, (hipStream_t)stream);
  if (e != hipSuccess) return status8(e);
  return status8(launch_int8_gemm(q, rows8(w), y, ldy, f16, ws, (hipStream_t)stream));
}

size_t bnbx_gemm_int8_dx_workspace_bytes(int M, int N, int K) {
  if (M < 1 || N < 1 || K < 1) return 0;
  return int8_grad_workspace(M, K, N);
}

int bnbx_gemm_int8_dx(const uint16_t* dy, int64_t lddy, int M, const bnbx_int8_rows* w,
                      uint16_t* dx, int64_t lddx, void* workspace, size_t workspace_bytes,
                      void* stream) {
  int s = check_rows8(w, false);
  if (s != BNBX_OK) return s;
  if (M < 0) return BNBX_E_INVAL;
  s = check_matrix8(dx, lddx, M, w->cols, 2);
  if (s != BNBX_OK) return s;
  s = check_dy8(dy, lddy, M, w->rows);
  if (s != BNBX_OK) return s;
  if (too_many(M) || too_many(w->rows)) return BNBX_E_UNSUPPORTED;
  if (M == 0) return BNBX_OK;
  s = check_workspace8(workspace, workspace_bytes, int8_grad_workspace(M, w->cols, w->rows));
  if (s != BNBX_OK) return s;
  const bool f16 = w->dtype == BNBX_DTYPE_F16;
  const GradGemm g{dy, lddy, M, rows8(w), dx, lddx, f16 ? kOutF16 : kOutBf16};
  return status8(launch_int8_grad(g, false, f16, workspace, (hipStream_t)stream));
}

size_t bnbx_gemm_int8_dw_workspace_bytes(int M, int N, int K) {
  if (M < 0 || N < 1 || K < 1) return 0;
  return int8_grad_workspace(N, K, M);
}

int bnbx_gemm_int8_dw(const uint16_t* dy, int64_t lddy, int N, const bnbx_int8_rows* x, void* dw,
                      int64_t lddw, int out_dtype, void* workspace, size_t workspace_bytes,
                      void* stream) {
  int s = check_rows8(x, true);
  if (s != BNBX_OK) return s;
  if (N < 1) return BNBX_E_INVAL;
  if (out_dtype != BNBX_DTYPE_F32 && out_dtype != x->dtype) return BNBX_E_INVAL;
  s = check_matrix8(dw, lddw, N, x->cols, out_dtype == BNBX_DTYPE_F32 ? 4 : 2);
  if (s != BNBX_OK) return s;
  s = check_dy8(dy, lddy, x->rows, N);
  if (s != BNBX_OK) return s;
  if (too_many(N) || too_many(x->rows)) return BNBX_E_UNSUPPORTED;
  s = check_workspace8(workspace, workspace_bytes, int8_grad_workspace(N, x->cols, x->rows));
  if (s != BNBX_OK) return s;
  const bool f16 = x->dtype == BNBX_DTYPE_F16;
  const GradGemm g{dy, lddy, N, rows8(x), dw, lddw, out_dtype};
  return status8(launch_int8_grad(g, true, f16, workspace, (hipStream_t)stream));
}

}  // extern "C"
