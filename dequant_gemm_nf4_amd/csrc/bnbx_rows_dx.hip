// Input gradient of the expert-grouped 4-bit product for gfx950:
// dX_i = dY_i . W_hat_g, i a place of group g (the weights stay frozen).
//
// Many rows a group: the tiles of bnbx_gemm_dx_core.hpp, a tile's 256 rows the
// places of one group.  Bound: as the ungrouped form's (the barrier of a step
// with its LDS and dequant work in between), and the last round of tiles: 8192
// rows in 8 uneven groups of 11008 x 4096 take 1110 us, 667 TFLOP/s.  A form
// whose waves dequantize their operands straight into registers (no LDS tile of
// weights) took 1250 us: its table reads double.
#include "bnbx_gemm_dx_core.hpp"

namespace bnbx {

hipError_t launch_rows_dx(const RowsGemm& a, int quant_type, bool f16, hipStream_t stream) {
  const int64_t kLimit = (int64_t)1 << 31;
  if (a.N % TN != 0 || (int64_t)a.N * (a.K / 2) >= kLimit) return hipErrorNotSupported;
  // 32-bit offsets into dY: all of it where rows are looked up, one tile else
  const int64_t reach = a.gather > 0 ? a.x_rows : TM;
  if (reach * a.ldx * 2 >= kLimit) return hipErrorNotSupported;
  const int tiles_k = (a.K - 1) / TK + 1;
  const unsigned grid = rows_grid(a.rows, a.groups, TM, tiles_k, kThreads);
  if (grid == 0) return hipErrorNotSupported;
  const LevelTable& lv = level_table(quant_type);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(kThreads), 0, stream, a.x, a.ldx,
                       a.packed, a.absmax, a.absmax2, a.mean, a.rows, a.N, a.K, a.y, a.ldy, 0,
                       tiles_k, lv, a);
  };
  if (a.double_quant == kDqDynamic) {
    if (f16) go(gemm_dx_kernel<kDqDynamic, true, true>);
    else go(gemm_dx_kernel<kDqDynamic, false, true>);
  } else if (a.double_quant) {
    if (f16) go(gemm_dx_kernel<kDqLinear, true, true>);
    else go(gemm_dx_kernel<kDqLinear, false, true>);
  } else {
    if (f16) go(gemm_dx_kernel<kDqNone, true, true>);
    else go(gemm_dx_kernel<kDqNone, false, true>);
  }
  return hipGetLastError();
}

}  // namespace bnbx
