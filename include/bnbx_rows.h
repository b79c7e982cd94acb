/*
 * bnbx_rows.h -- C ABI of libbnbx_rows.so: 4-bit linear layers whose rows
 * belong to groups, for MI355X (gfx950).
 *
 * A row's group is the expert that a router sent it to, or the adapter of the
 * request it came with.  bnbx_group_rows makes a plan (the rows in group
 * order and every group's bounds) on the device, with no host round trip;
 * the products take the plan:
 *   bnbx_gemm_nf4_experts     Y_i = X_i . W_hat_g^T, one 4-bit weight a group
 *   bnbx_gemm_nf4_experts_dx  dX_i = dY_i . W_hat_g, its input gradient
 *   bnbx_gemm_nf4_adapters    Y = X . W_hat^T + s_g . (X . A_g^T) . B_g^T, one
 *                             shared 4-bit weight, one low-rank adapter a group
 *
 * Conventions, status codes, the quant state and the stored format are those
 * of bnbx.h: the caller owns every buffer and the stream, nothing is
 * allocated or synchronised, every argument the host can see is checked before
 * anything is enqueued.  Index arrays live on the device, where the host
 * cannot check them: the kernels clamp offsets to the plan's rows and skip a
 * row whose index lies outside X or Y, so a wrong plan gives wrong or missing
 * rows of Y, never an access outside the buffers.  Calls keep no state between
 * them; calls that share an output or a workspace must be ordered by the
 * caller.  Results do not depend on timing: the same call on the same
 * inputs repeats bit for bit.
 */
#ifndef BNBX_ROWS_H
#define BNBX_ROWS_H

#include "bnbx.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Only the entry points below are exported from libbnbx_rows.so. */
#define BNBX_ROWS_API __attribute__((visibility("default")))

/* Most groups a plan holds. */
#define BNBX_ROWS_MAX_GROUPS 1024

/* A plan: the rows 0 .. rows-1 in group order.  Group g holds the plan's
 * places offsets[g] .. offsets[g+1]-1; places offsets[groups] .. rows-1 are
 * rows of no group. */
typedef struct {
  const int32_t* offsets; /* device int32[groups + 1], 0 <= ascending <= rows  */
  const int32_t* order;   /* device int32[rows]: the row at each place         */
  int32_t groups;         /* 1 .. BNBX_ROWS_MAX_GROUPS                         */
  int32_t rows;           /* >= 0; products take rows <= 2^31 - 512 and
                             (rows / 16 + 1) * groups < 2^31 (else
                             BNBX_E_UNSUPPORTED)                               */
} bnbx_row_groups;

/* Bytes of device workspace bnbx_group_rows needs; 0 for few rows (one
 * launch does it all) and for invalid arguments. */
BNBX_ROWS_API size_t bnbx_group_rows_workspace_bytes(int rows, int groups);

/* The plan of ids[0 .. rows-1]: rows sorted by group, rows of one group in
 * ascending order, rows whose id is outside 0 .. groups-1 (-1: none) behind
 * the last group, ascending too.
 *   ids        device, int32[rows], 4-byte aligned (may be NULL for rows = 0)
 *   rows       >= 0
 *   groups     1 .. BNBX_ROWS_MAX_GROUPS (more: BNBX_E_UNSUPPORTED)
 *   offsets    device, int32[groups + 1] (written)
 *   order      device, int32[rows] (written; may be NULL for rows = 0)
 *   workspace  device, >= bnbx_group_rows_workspace_bytes(...) bytes, 4-byte
 *              aligned (may be NULL when that is 0); scratch
 * Errors: BNBX_E_INVAL, BNBX_E_ALIGN, BNBX_E_UNSUPPORTED, BNBX_E_WORKSPACE. */
BNBX_ROWS_API int bnbx_group_rows(const int32_t* ids, int rows, int groups, int32_t* offsets,
                                  int32_t* order, void* workspace, size_t workspace_bytes,
                                  void* stream);

/* Products grouped by expert (the 4-bit linear layers of a mixture of
 * experts; W_hat as in bnbx_dequantize_nf4): place i of the plan, in group g,
 *   Y[row_y(i)] = X[row_x(i)] . W_hat_g^T,   W_hat_g [N, K] the g-th of the
 * `groups` weights of one stack [groups, N, K], quantized as one tensor
 * (st->n = groups * N * K).
 *   row_x(i) = order[i] / gather for gather >= 1 (1: the rows themselves; top_k:
 *              order numbers the top_k slots of each token), i for gather 0
 *   row_y(i) = order[i] for scatter 1, i for scatter 0
 * Rows of Y that no place of a group writes keep what they held (places of no
 * group among them).  A place whose row lies outside X or Y is left out.  With
 * scatter 0 or 1 and a plan of bnbx_group_rows no two places share a row of Y.
 *   x       device, 16-bit of st->compute_dtype, x_rows rows at x + row*ldx;
 *           ldx >= K, ldx % 8 == 0, 16-byte aligned (may be NULL if x_rows = 0)
 *   packed  device, the packed stack, 16-byte aligned
 *   plan    host descriptor; plan->rows = 0 is a call that does nothing
 *   N, K    of one weight; K a multiple of 64; N * K below 2^32
 *   y       device, y_rows rows at y + row*ldy; ldy >= N (written)
 * Any number of rows a group, none included.  X of 2 GiB and more (x_rows * ldx * 2
 * bytes) with gather >= 1 takes a form of about half the rate where many rows a
 * group would take the fastest one; split the rows over calls there.  y must not
 * overlap x.  Errors: BNBX_E_INVAL,
 * BNBX_E_ALIGN, BNBX_E_UNSUPPORTED (a weight too large for 32-bit offsets, more
 * than BNBX_ROWS_MAX_GROUPS groups, more output tiles than one launch takes). */
BNBX_ROWS_API int bnbx_gemm_nf4_experts(const uint16_t* x, int64_t ldx, int x_rows,
                                        const uint8_t* packed, const bnbx_nf4_state* st,
                                        const bnbx_row_groups* plan, int N, int K, int gather,
                                        int scatter, uint16_t* y, int64_t ldy, int y_rows,
                                        void* stream);

/* Input gradient of bnbx_gemm_nf4_experts (frozen weights): for place i of
 * group g,   dX[row_x(i)] = dY[row_y(i)] . W_hat_g,   dY [dy_rows, N], dX
 * [dx_rows, K], with row_y(i) = order[i] / gather or i and row_x(i) = order[i] or
 * i as above.  Where the forward gathered with top_k, call with scatter 1: dX
 * then has a row per slot, rounded to 16 bits, and a token's gradient is the sum
 * of its slots' rows.
 * The other arguments, what is left untouched and the errors as above (lddy for
 * ldx, lddx for ldy), except: N a multiple of 64 (else BNBX_E_UNSUPPORTED). */
BNBX_ROWS_API int bnbx_gemm_nf4_experts_dx(const uint16_t* dy, int64_t lddy, int dy_rows,
                                           const uint8_t* packed, const bnbx_nf4_state* st,
                                           const bnbx_row_groups* plan, int N, int K, int gather,
                                           int scatter, uint16_t* dx, int64_t lddx, int dx_rows,
                                           void* stream);

/* The adapters of a call, one per group of its plan (host descriptor; device
 * pointers).  A lower rank than r is held as r with zero rows of A or zero
 * columns of B. */
typedef struct {
  const uint16_t* lora_a; /* adapter g's A [r, K], row j at lora_a + g*stride_a + j*lda;
                             lda >= K, lda and stride_a % 8 == 0, 16-byte aligned     */
  const uint16_t* lora_b; /* adapter g's B [N, r], row n at lora_b + g*stride_b + n*ldb;
                             ldb >= r, ldb and stride_b % 8 == 0, 16-byte aligned     */
  const float* scale;     /* s_g, float[groups]                                       */
  int64_t lda, stride_a, ldb, stride_b;
  int32_t r;              /* a multiple of 16, 16 <= r <= 256                         */
} bnbx_adapters;

/* Bytes of device workspace bnbx_gemm_nf4_adapters needs for `rows` rows and
 * rank r; 0 for invalid arguments. */
BNBX_ROWS_API size_t bnbx_gemm_nf4_adapters_workspace_bytes(int rows, int r);

/* One shared 4-bit linear layer beside the adapters of many requests:
 *   Y_m = X_m . W_hat^T + s_g . (X_m . A_g^T) . B_g^T   for row m of group g,
 *   Y_m = X_m . W_hat^T                                 for a row of no group.
 * X [rows, K] and Y [rows, N] in the requests' own order, rows = plan->rows; the
 * plan (bnbx_group_rows of the rows' adapter ids) gives each adapter its rows,
 * any number of them, and must list every row in `order`: a row it does not
 * list is not written.  Values are of st->compute_dtype; both products
 * accumulate in fp32, X . A_g^T keeps 16 significant bits, and Y is rounded
 * once.  X of 2 GiB and more runs at about half the rate (as with gather above).
 * An adapter with infinities or NaN reaches its own rows only, and gives
 * them what the formula gives: a signed infinity, or NaN for 0 . inf and
 * inf - inf.
 *   x, packed, st, N, K  as bnbx_gemm_nf4 (st->n = N * K)
 *   y          device, row m at y + m*ldy; ldy >= N (written); must not overlap x
 *   workspace  device, >= bnbx_gemm_nf4_adapters_workspace_bytes(...) bytes,
 *              16-byte aligned; scratch
 * Errors: as bnbx_gemm_nf4_experts, and BNBX_E_WORKSPACE. */
BNBX_ROWS_API int bnbx_gemm_nf4_adapters(const uint16_t* x, int64_t ldx, const uint8_t* packed,
                                         const bnbx_nf4_state* st, const bnbx_row_groups* plan,
                                         int N, int K, const bnbx_adapters* adapters, uint16_t* y,
                                         int64_t ldy, void* workspace, size_t workspace_bytes,
                                         void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BNBX_ROWS_H */
