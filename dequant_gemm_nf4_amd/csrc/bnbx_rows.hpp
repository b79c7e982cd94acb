// Internal declarations of libbnbx_rows (include/bnbx_rows.h).
#pragma once

#include "bnbx_internal.hpp"

namespace bnbx {

constexpr int kMaxGroups = 1024;   // BNBX_ROWS_MAX_GROUPS
constexpr int kMaxRows = INT32_MAX - 511;   // place numbers of a last tile stay in 31 bits
constexpr int kXcds = 8;

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

// Workgroups of a launch over tiles of tm places, `across` to a row tile (the most
// tiles there can be, a multiple of kXcds); 0: more than one launch takes, which
// counts threads in 32 bits.
inline unsigned rows_grid(int rows, int groups, int tm, int across, int threads) {
  const int64_t tiles = (int64_t)rows / tm + (groups < rows ? groups : rows);
  const int64_t grid = (tiles * across + kXcds - 1) / kXcds * kXcds;
  return grid * threads < ((int64_t)1 << 32) ? (unsigned)grid : 0;
}

// The launches below return hipErrorNotSupported, before anything is enqueued,
// for a call that they do not take; without `launch` that is all they do.

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
                                 uint16_t* xa, hipStream_t stream, bool launch);

// Streaming form: row tiles of 16, 32 or 64 places (bnbx_rows_stream.hip).
hipError_t launch_rows_stream(const RowsGemm& a, int quant_type, bool f16, int cus,
                              hipStream_t stream, bool launch);

// Tiled form: row tiles of 256 places (bnbx_rows_gemm.hip), and with a
// low-rank term (bnbx_rows_gemm_lora.hip).  Not for an X past 32-bit offsets.
hipError_t launch_rows_gemm(const RowsGemm& a, int quant_type, bool f16, hipStream_t stream,
                            bool launch);
hipError_t launch_rows_gemm_lora(const RowsGemm& a, int quant_type, bool f16, hipStream_t stream,
                                 bool launch);

// dX_i = dY_i . W_hat_g: x is dY [x_rows, N], y is dX [y_rows, K]; N a
// multiple of 64 (bnbx_rows_dx.hip).
hipError_t launch_rows_dx(const RowsGemm& a, int quant_type, bool f16, hipStream_t stream);

// The same over few rows a group (bnbx_rows_dx_stream.hip).
hipError_t launch_rows_dx_stream(const RowsGemm& a, int quant_type, bool f16, hipStream_t stream);

// Compute units of the current device.
int rows_cus();

}  // namespace bnbx
