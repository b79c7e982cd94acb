// C entry points of libbnbx_rows (declared in include/bnbx_rows.h): argument
// checks on the host and kernel launches.
#include "../../include/bnbx_rows.h"
#include "bnbx_checks.hpp"
#include "bnbx_rows.hpp"

namespace bnbx {
static_assert(kMaxGroups == BNBX_ROWS_MAX_GROUPS, "groups of a plan");
namespace {

int check_plan(const bnbx_row_groups* p) {
  if (p == nullptr || p->offsets == nullptr || p->groups < 1 || p->rows < 0) return BNBX_E_INVAL;
  if (p->rows > 0 && p->order == nullptr) return BNBX_E_INVAL;
  if (p->groups > BNBX_ROWS_MAX_GROUPS) return BNBX_E_UNSUPPORTED;
  if (!aligned(p->offsets, 4) || !aligned(p->order, 4)) return BNBX_E_ALIGN;
  return BNBX_OK;
}

// x [x_rows, kx] -> y [y_rows, ny] over a stack of `stack` weights [N, K].
int check_rows(const uint16_t* x, int64_t ldx, int x_rows, int64_t kx, const uint8_t* packed,
               const bnbx_nf4_state* st, int64_t stack, int N, int K, int gather, int scatter,
               const uint16_t* y, int64_t ldy, int y_rows, int64_t ny) {
  if (packed == nullptr || x_rows < 0 || y_rows < 0) return BNBX_E_INVAL;
  if ((x_rows > 0 && x == nullptr) || (y_rows > 0 && y == nullptr)) return BNBX_E_INVAL;
  const int s = check_state(st);
  if (s != BNBX_OK) return s;
  if (N < 1 || K < kBlock || K % kBlock != 0) return BNBX_E_INVAL;
  if ((__int128)stack * N * K != st->n) return BNBX_E_INVAL;
  if (gather < 0 || (scatter != 0 && scatter != 1)) return BNBX_E_INVAL;
  if (ldx < kx || ldy < ny) return BNBX_E_INVAL;
  if (ldx % 8 != 0) return BNBX_E_ALIGN;
  if (!aligned(x, 16) || !aligned(packed, 16) || !aligned(y, 2)) return BNBX_E_ALIGN;
  if (st->double_quant == kDqNone && !aligned(st->absmax, 4)) return BNBX_E_ALIGN;
  if ((int64_t)N * (K / 2) >= ((int64_t)1 << 31)) return BNBX_E_UNSUPPORTED;
  return BNBX_OK;
}

RowsGemm rows_gemm(const uint16_t* x, int64_t ldx, int x_rows, const uint8_t* packed,
                   const bnbx_nf4_state* st, const bnbx_row_groups* p, int N, int K, int gather,
                   int scatter, uint16_t* y, int64_t ldy, int y_rows) {
  RowsGemm a{};
  a.x = x;
  a.ldx = ldx;
  a.x_rows = x_rows;
  a.packed = packed;
  a.absmax = st->absmax;
  a.absmax2 = st->absmax2;
  a.mean = st->absmax_mean;
  a.double_quant = st->double_quant;
  a.offsets = p->offsets;
  a.order = p->order;
  a.groups = p->groups;
  a.rows = p->rows;
  a.gather = gather;
  a.scatter = scatter;
  a.N = N;
  a.K = K;
  a.y = y;
  a.ldy = ldy;
  a.y_rows = y_rows;
  return a;
}

int rows_status(hipError_t e) {
  return e == hipErrorNotSupported ? BNBX_E_UNSUPPORTED : hip_status(e);
}

}  // namespace
}  // namespace bnbx

using namespace bnbx;

extern "C" {

size_t bnbx_group_rows_workspace_bytes(int rows, int groups) {
  if (rows < 0 || groups < 1 || groups > BNBX_ROWS_MAX_GROUPS) return 0;
  return group_rows_workspace_bytes(rows, groups);
}

int bnbx_group_rows(const int32_t* ids, int rows, int groups, int32_t* offsets, int32_t* order,
                    void* workspace, size_t workspace_bytes, void* stream) {
  if (rows < 0 || groups < 1 || offsets == nullptr) return BNBX_E_INVAL;
  if (rows > 0 && (ids == nullptr || order == nullptr)) return BNBX_E_INVAL;
  if (groups > BNBX_ROWS_MAX_GROUPS) return BNBX_E_UNSUPPORTED;
  if (!aligned(ids, 4) || !aligned(offsets, 4) || !aligned(order, 4)) return BNBX_E_ALIGN;
  const size_t need = group_rows_workspace_bytes(rows, groups);
  if (need > 0) {
    if (workspace == nullptr || workspace_bytes < need) return BNBX_E_WORKSPACE;
    if (!aligned(workspace, 4)) return BNBX_E_ALIGN;
  }
  return hip_status(launch_group_rows(ids, rows, groups, offsets, order, (int32_t*)workspace,
                                      (hipStream_t)stream));
}

int bnbx_gemm_nf4_experts(const uint16_t* x, int64_t ldx, int x_rows, const uint8_t* packed,
                          const bnbx_nf4_state* st, const bnbx_row_groups* plan, int N, int K,
                          int gather, int scatter, uint16_t* y, int64_t ldy, int y_rows,
                          void* stream) {
  int s = check_plan(plan);
  if (s != BNBX_OK) return s;
  s = check_rows(x, ldx, x_rows, K, packed, st, plan->groups, N, K, gather, scatter, y, ldy,
                 y_rows, N);
  if (s != BNBX_OK) return s;
  if (plan->rows == 0 || x_rows == 0 || y_rows == 0) return BNBX_OK;
  const RowsGemm a = rows_gemm(x, ldx, x_rows, packed, st, plan, N, K, gather, scatter, y, ldy,
                               y_rows);
  return rows_status(launch_rows_stream(a, st->quant_type, st->compute_dtype == BNBX_DTYPE_F16,
                                        device_cus(), (hipStream_t)stream));
}

}  // extern "C"
