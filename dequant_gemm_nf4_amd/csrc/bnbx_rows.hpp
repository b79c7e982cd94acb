// Internal declarations of libbnbx_rows (include/bnbx_rows.h).
#pragma once

#include "bnbx_internal.hpp"

namespace bnbx {

constexpr int kMaxGroups = 1024;   // BNBX_ROWS_MAX_GROUPS

// bnbx_group_rows: workspace bytes and launch.
size_t group_rows_workspace_bytes(int rows, int groups);
hipError_t launch_group_rows(const int32_t* ids, int rows, int groups, int32_t* offsets,
                             int32_t* order, int32_t* workspace, hipStream_t stream);

// Low-rank term of the adapters product, Y_i += XA_i . B_g^T for the places
// i of adapter g.  XA is held as two bf16 planes (hi + lo, together 16
// significant bits of the fp32 sum; bnbx_rows_lora.hip says how infinities are
// held) per place: place i's hi plane at xa + 2 i r, its lo plane r further.
struct LoraRows {
  const int32_t* offsets;   // the adapters' bounds, null: no low-rank term
  int adapters;
  int r;
  const uint16_t* xa;       // [rows][2][r] bf16
  const uint16_t* b;        // adapter g's B [N, r], row n at b + g stride + n ld
  int64_t ldb, stride_b;
};

// One product over grouped rows.  Place i of the plan reads row
//   gather ? order[i] / gather : i     of X (x_rows rows), and writes row
//   scatter ? order[i] : i             of Y (y_rows rows);
// a place whose row lies outside X or Y is left out.
struct RowsGemm {
  const uint16_t* x;
  int64_t ldx;
  int x_rows;
  const uint8_t* packed;     // [groups][N][K / 2]
  const void* absmax;        // scales of the whole stack, as one tensor
  const float* absmax2;
  const float* mean;
  int double_quant;          // kDqNone, kDqLinear, kDqDynamic
  const int32_t* offsets;    // null: one group of all rows
  const int32_t* order;
  int groups, rows;
  int gather, scatter;
  int N, K;
  uint16_t* y;
  int64_t ldy;
  int y_rows;
  LoraRows lora;
};

// The adapters' down-projections into xa's planes (bnbx_rows_lora.hip).
struct LoraDown {
  const int32_t* offsets;
  int adapters;
  int r;
  const uint16_t* a;        // adapter g's A [r, K], row j at a + g stride + j ld
  int64_t lda, stride_a;
  const float* scale;       // [adapters]
};
hipError_t launch_rows_lora_down(const RowsGemm& a, const LoraDown& d, bool f16, int cus,
                                 uint16_t* xa, hipStream_t stream);

// Streaming form: row tiles of 16, 32 or 64 places (bnbx_rows_stream.hip).
hipError_t launch_rows_stream(const RowsGemm& a, int quant_type, bool f16, int cus,
                              hipStream_t stream);

// Tiled form: row tiles of 256 places (bnbx_rows_gemm.hip), and with a
// low-rank term (bnbx_rows_gemm_lora.hip).  hipErrorNotSupported where X does
// not fit 32-bit offsets.
hipError_t launch_rows_gemm(const RowsGemm& a, int quant_type, bool f16, hipStream_t stream);
hipError_t launch_rows_gemm_lora(const RowsGemm& a, int quant_type, bool f16,
                                 hipStream_t stream);

// dX_i = dY_i . W_hat_g: x is dY [x_rows, N], y is dX [y_rows, K]; N a
// multiple of 64 (bnbx_rows_dx.hip).
hipError_t launch_rows_dx(const RowsGemm& a, int quant_type, bool f16, hipStream_t stream);

// The same over few rows a group (bnbx_rows_dx_stream.hip).
hipError_t launch_rows_dx_stream(const RowsGemm& a, int quant_type, bool f16, hipStream_t stream);

// Compute units of the current device.
int rows_cus();

}  // namespace bnbx
