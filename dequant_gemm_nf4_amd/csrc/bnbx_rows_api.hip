// C entry points of libbnbx_rows (declared in include/bnbx_rows.h): argument
// checks on the host and kernel launches.
#include "../../include/bnbx_rows.h"
#include "bnbx_checks.hpp"
#include "bnbx_rows.hpp"
#include "bnbx_rows_form.hpp"

namespace bnbx {
static_assert(kMaxGroups == BNBX_ROWS_MAX_GROUPS, "groups of a plan");
namespace {

int check_plan(const bnbx_row_groups* p) {
  if (p == nullptr || p->offsets == nullptr || p->groups < 1 || p->rows < 0) return BNBX_E_INVAL;
  if (p->rows > 0 && p->order == nullptr) return BNBX_E_INVAL;
  if (p->groups > BNBX_ROWS_MAX_GROUPS) return BNBX_E_UNSUPPORTED;
  if (!aligned(p->offsets, 4) || !aligned(p->order, 4)) return BNBX_E_ALIGN;
  // the kernels count places to the end of a last tile and tiles of 16 places or
  // more in 32 bits, and groups of a wrong plan may overlap
  if (p->rows > kMaxRows) return BNBX_E_UNSUPPORTED;
  if (((int64_t)p->rows / 16 + 1) * p->groups >= ((int64_t)1 << 31)) return BNBX_E_UNSUPPORTED;
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
  if (st->double_quant == kDqNone ? !aligned(st->absmax, 4)
                                  : !aligned(st->absmax2, 4) || !aligned(st->absmax_mean, 4))
    return BNBX_E_ALIGN;
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

// The groups of a product as the choice of form counts them.
int groups_of(const RowsGemm& a) { return a.offsets == nullptr ? 0 : a.groups; }

// The products of both operators: the tiled form, or the streaming form (also
// for an X past 32-bit offsets).
hipError_t launch_rows(const RowsGemm& a, int quant_type, bool f16, int cus, hipStream_t hs,
                       bool launch) {
  const bool low_rank = a.lora.offsets != nullptr;
  if (prefer_tiles(a.rows, groups_of(a), a.N, a.K, a.lora.adapters, low_rank ? a.lora.r : 0,
                   cus)) {
    const hipError_t e = low_rank ? launch_rows_gemm_lora(a, quant_type, f16, hs, launch)
                                  : launch_rows_gemm(a, quant_type, f16, hs, launch);
    if (e != hipErrorNotSupported) return e;
  }
  return launch_rows_stream(a, quant_type, f16, cus, hs, launch);
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
  return rows_status(launch_rows(a, st->quant_type, st->compute_dtype == BNBX_DTYPE_F16,
                                 rows_cus(), (hipStream_t)stream, true));
}

int bnbx_gemm_nf4_experts_dx(const uint16_t* dy, int64_t lddy, int dy_rows,
                             const uint8_t* packed, const bnbx_nf4_state* st,
                             const bnbx_row_groups* plan, int N, int K, int gather, int scatter,
                             uint16_t* dx, int64_t lddx, int dx_rows, void* stream) {
  int s = check_plan(plan);
  if (s != BNBX_OK) return s;
  s = check_rows(dy, lddy, dy_rows, N, packed, st, plan->groups, N, K, gather, scatter, dx, lddx,
                 dx_rows, K);
  if (s != BNBX_OK) return s;
  if (N % 64 != 0) return BNBX_E_UNSUPPORTED;
  if (plan->rows == 0 || dy_rows == 0 || dx_rows == 0) return BNBX_OK;
  const RowsGemm a = rows_gemm(dy, lddy, dy_rows, packed, st, plan, N, K, gather, scatter, dx,
                               lddx, dx_rows);
  const bool f16 = st->compute_dtype == BNBX_DTYPE_F16;
  hipError_t e = hipErrorNotSupported;
  if (prefer_dx_tiles(a.rows, groups_of(a), a.K, rows_cus()))
    e = launch_rows_dx(a, st->quant_type, f16, (hipStream_t)stream);
  if (e == hipErrorNotSupported)
    e = launch_rows_dx_stream(a, st->quant_type, f16, (hipStream_t)stream);
  return rows_status(e);
}

size_t bnbx_gemm_nf4_adapters_workspace_bytes(int rows, int r) {
  if (rows < 0 || r < 16 || r > 256 || r % 16 != 0) return 0;
  return (size_t)rows * 2 * (size_t)r * sizeof(uint16_t);
}

int bnbx_gemm_nf4_adapters(const uint16_t* x, int64_t ldx, const uint8_t* packed,
                           const bnbx_nf4_state* st, const bnbx_row_groups* plan, int N, int K,
                           const bnbx_adapters* ad, uint16_t* y, int64_t ldy, void* workspace,
                           size_t workspace_bytes, void* stream) {
  int s = check_plan(plan);
  if (s != BNBX_OK) return s;
  s = check_rows(x, ldx, plan->rows, K, packed, st, 1, N, K, 1, 1, y, ldy, plan->rows, N);
  if (s != BNBX_OK) return s;
  if (ad == nullptr || ad->lora_a == nullptr || ad->lora_b == nullptr || ad->scale == nullptr)
    return BNBX_E_INVAL;
  if (ad->r < 16 || ad->r > 256 || ad->r % 16 != 0) return BNBX_E_INVAL;
  if (ad->lda < K || ad->ldb < ad->r || ad->stride_a < 0 || ad->stride_b < 0) return BNBX_E_INVAL;
  if (ad->lda % 8 != 0 || ad->ldb % 8 != 0 || ad->stride_a % 8 != 0 || ad->stride_b % 8 != 0)
    return BNBX_E_ALIGN;
  if (!aligned(ad->lora_a, 16) || !aligned(ad->lora_b, 16) || !aligned(ad->scale, 4))
    return BNBX_E_ALIGN;
  if (plan->rows == 0) return BNBX_OK;
  const size_t need = bnbx_gemm_nf4_adapters_workspace_bytes(plan->rows, ad->r);
  if (workspace == nullptr || workspace_bytes < need) return BNBX_E_WORKSPACE;
  if (!aligned(workspace, 16)) return BNBX_E_ALIGN;
  const bool f16 = st->compute_dtype == BNBX_DTYPE_F16;
  const int cus = rows_cus();
  hipStream_t hs = (hipStream_t)stream;
  const RowsGemm a =
      rows_gemm(x, ldx, plan->rows, packed, st, plan, N, K, 1, 1, y, ldy, plan->rows);
  const LoraDown d{plan->offsets, plan->groups, ad->r, ad->lora_a, ad->lda, ad->stride_a,
                   ad->scale};
  RowsGemm b = a;
  b.offsets = nullptr;   // the shared weight: one group of all rows
  b.groups = 1;
  b.lora = LoraRows{plan->offsets, plan->groups, ad->r, (const uint16_t*)workspace, ad->lora_b,
                    ad->ldb, ad->stride_b};
  // nothing is enqueued unless both launches fit
  for (const bool launch : {false, true}) {
    hipError_t e = launch_rows_lora_down(a, d, f16, cus, (uint16_t*)workspace, hs, launch);
    if (e == hipSuccess) e = launch_rows(b, st->quant_type, f16, cus, hs, launch);
    if (e != hipSuccess) return rows_status(e);
  }
  return BNBX_OK;
}

}  // extern "C"
