/*
 * bnbx_int8.h -- C ABI of libbnbx_int8.so: the 8-bit linear layer and its
 * training from 8-bit activations, for MI355X (gfx950).
 *
 * A matrix is held as rows of int8 codes with one fp32 scale a row: a weight
 * [N, K] has a scale for each output channel, activations [M, K] one for each
 * token.  The codes that the forward product reads are also what the backward
 * pass keeps of the activations (one byte a value instead of two):
 *   bnbx_quantize_rows_int8     16-bit rows -> codes and scales
 *   bnbx_dequantize_rows_int8   codes -> 16-bit values
 *   bnbx_linear_int8            Y = X . W^T, X quantized on the way
 *   bnbx_gemm_int8              the same from codes of X
 *   bnbx_gemm_int8_dx           dX = dY . W_hat, the input gradient
 *   bnbx_gemm_int8_dw           dW = dY^T . X_hat, the weight's gradient from
 *                               the activations' codes
 *
 * Source: the pomoai.com bitsandbytes overview, module list (Linear8bitLt
 * replaces torch.nn.Linear: int8 products with a scale for each row of both
 * operands).  All features stay in 8 bits here; there is no second part in 16
 * bits for outlying features.
 *
 * The format of a row x of K values (bf16 or binary16):
 *   a = max |x_k|,  scale = fl32(a / 127),
 *   code_k = 127 x_k / a rounded to the nearest integer, ties to even (of the
 *            exact quotient), -127 .. 127;
 *   a = 0: scale 0, codes 0.  A row with an infinity or a NaN: scale NaN, codes
 *   0, so that what is computed from it is NaN.
 * The value of a code is v = rnd16(fl32(code * scale)), rnd16 the rounding to
 * nearest even into the rows' 16-bit type (as W_hat of the 4-bit format).
 * A row of codes starts at a multiple of 16 bytes, and the bytes behind its
 * last code up to the next multiple of 16 are zero (the quantizer writes them;
 * the products read them).
 *
 * Conventions and status codes are those of bnbx.h: the caller owns every
 * buffer and the stream, nothing is allocated or synchronised, every argument
 * is checked on the host before anything is enqueued, calls keep no state
 * between them, what a call writes (its workspace too) overlaps nothing else that it is
 * given, and calls that share an output or a workspace must be ordered
 * by the caller.  The same call on the same inputs repeats bit for bit.
 */
#ifndef BNBX_INT8_H
#define BNBX_INT8_H

#include "bnbx.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Only the entry points below are exported from libbnbx_int8.so. */
#define BNBX_INT8_API __attribute__((visibility("default")))

/* Output type of bnbx_gemm_int8_dw beside BNBX_DTYPE_BF16 and BNBX_DTYPE_F16. */
enum { BNBX_DTYPE_F32 = 2 };

/* Most columns of a row in the products: 128^2 * K stays below 2^31. */
#define BNBX_INT8_MAX_COLS 131071

/* Rows of codes (host descriptor of device buffers). */
typedef struct {
  int8_t* codes;  /* device, row r at codes + r * ld, 16-byte aligned            */
  float* scale;   /* device float[rows], 4-byte aligned                          */
  int64_t ld;     /* bytes from row to row, a multiple of 16, at least cols
                     rounded up to one, below 2^23                              */
  int32_t rows;   /* >= 0                                                        */
  int32_t cols;   /* >= 1                                                        */
  int32_t dtype;  /* BNBX_DTYPE_BF16 or BNBX_DTYPE_F16: type of the values       */
} bnbx_int8_rows;

/* Codes and scales of x [q->rows, q->cols] (16-bit of q->dtype), row r at x +
 * r * ldx; ldx >= cols (ldx a multiple of 8 and x 16-byte aligned is the fast
 * path; any ldx and 2-byte alignment work).  Writes q->codes, the zeros behind
 * each row, and q->scale.  Errors: BNBX_E_INVAL, BNBX_E_ALIGN,
 * BNBX_E_UNSUPPORTED (ld of 2^23 or more). */
BNBX_INT8_API int bnbx_quantize_rows_int8(const uint16_t* x, int64_t ldx,
                                          const bnbx_int8_rows* q, void* stream);

/* The values of q's codes, row r at out + r * ldo (written; 16-bit of
 * q->dtype; ldo >= cols, alignment as x above). */
BNBX_INT8_API int bnbx_dequantize_rows_int8(const bnbx_int8_rows* q, uint16_t* out, int64_t ldo,
                                            void* stream);

/* Bytes of device workspace bnbx_gemm_int8 needs; 0 where it needs none, and
 * for invalid arguments. */
BNBX_INT8_API size_t bnbx_gemm_int8_workspace_bytes(int M, int N, int K);

/* Y[m, n] = rnd16(fl32(fl32(sum_k x_mk w_nk) * sx_m) * sw_n) over the codes x
 * [M, K] and w [N, K] of one dtype and equal cols K <= BNBX_INT8_MAX_COLS (more:
 * BNBX_E_UNSUPPORTED).  The sum is exact (int32); it is rounded to fp32, then by
 * each multiplication, then to 16 bits.
 *   y          device, row m at y + m * ldy; ldy >= N (written); 2-byte aligned
 *   workspace  device, >= bnbx_gemm_int8_workspace_bytes(...) bytes, 16-byte
 *              aligned (may be NULL when that is 0); scratch
 * M = 0 is a call that does nothing; w->rows must be positive.  y must not overlap
 * the operands.  Errors: BNBX_E_INVAL, BNBX_E_ALIGN, BNBX_E_UNSUPPORTED (K above
 * the limit, 2^31 - 511 rows or more of an operand, more output tiles than one launch
 * takes), BNBX_E_WORKSPACE. */
BNBX_INT8_API int bnbx_gemm_int8(const bnbx_int8_rows* x, const bnbx_int8_rows* w, uint16_t* y,
                                 int64_t ldy, void* workspace, size_t workspace_bytes,
                                 void* stream);

/* Bytes of device workspace bnbx_linear_int8 needs (X's codes among them
 * unless `saved`); 0 for invalid arguments. */
BNBX_INT8_API size_t bnbx_linear_int8_workspace_bytes(int M, int N, int K, int saved);

/* The layer: X's rows quantized as by bnbx_quantize_rows_int8, and
 * bnbx_gemm_int8 of their codes with w, to the same bits.
 *   x      device, 16-bit of w->dtype, M rows of w->cols at x + m * ldx (as in
 *          bnbx_quantize_rows_int8)
 *   saved  NULL, or where X's codes and scales are written for the backward
 *          pass: rows M, cols K, dtype of w
 * The rest as bnbx_gemm_int8. */
BNBX_INT8_API int bnbx_linear_int8(const uint16_t* x, int64_t ldx, int M,
                                   const bnbx_int8_rows* w, const bnbx_int8_rows* saved,
                                   uint16_t* y, int64_t ldy, void* workspace,
                                   size_t workspace_bytes, void* stream);

/* Bytes of device workspace bnbx_gemm_int8_dx needs; 0 where it needs none,
 * and for invalid arguments. */
BNBX_INT8_API size_t bnbx_gemm_int8_dx_workspace_bytes(int M, int N, int K);

/* Input gradient: dX[m, k] = rnd16(sum_n dY[m, n] v_nk) with the values v of w's
 * codes [N, K], products of 16-bit values accumulated in fp32.
 *   dy  device, 16-bit of w->dtype, row m at dy + m * lddy; lddy >= N, lddy a
 *       multiple of 8 below 2^22, 16-byte aligned; rows are read in pieces of
 *       eight: up to N rounded up to 8 they must be readable, and finite behind N
 *   dx  device, row m at dx + m * lddx; lddx >= K (written); 2-byte aligned
 * M = 0 is a call that does nothing.  Workspace and errors as bnbx_gemm_int8. */
BNBX_INT8_API int bnbx_gemm_int8_dx(const uint16_t* dy, int64_t lddy, int M,
                                    const bnbx_int8_rows* w, uint16_t* dx, int64_t lddx,
                                    void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of device workspace bnbx_gemm_int8_dw needs; 0 where it needs none,
 * and for invalid arguments. */
BNBX_INT8_API size_t bnbx_gemm_int8_dw_workspace_bytes(int M, int N, int K);

/* Weight's gradient from saved activations: dW[n, k] = rnd(sum_m dY[m, n] v_mk)
 * with the values v of x's codes [M, K], accumulated in fp32.
 *   dy         device, 16-bit of x->dtype, M = x->rows rows of N at dy + m * lddy;
 *              lddy >= N, lddy a multiple of 8 below 2^22, 16-byte aligned; rows
 *              are read in pieces of eight: the last one too must be readable up
 *              to N rounded up to 8 (what lies there has no effect)
 *   dw         device, row n at dw + n * lddw values; lddw >= K (written, zero
 *              for M = 0); aligned to its type
 *   out_dtype  x->dtype or BNBX_DTYPE_F32
 * Workspace and errors as bnbx_gemm_int8. */
BNBX_INT8_API int bnbx_gemm_int8_dw(const uint16_t* dy, int64_t lddy, int N,
                                    const bnbx_int8_rows* x, void* dw, int64_t lddw,
                                    int out_dtype, void* workspace, size_t workspace_bytes,
                                    void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BNBX_INT8_H */
