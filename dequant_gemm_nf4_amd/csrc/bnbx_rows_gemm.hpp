// Launch of the tiled form over grouped rows: the tiles of bnbx_gemm_core.hpp, a
// tile's 256 rows the places of one group, with a low-rank term (LORA) or none.
#pragma once

#include "bnbx_gemm_core.hpp"

namespace bnbx {
namespace {

template <bool LORA>
hipError_t launch_rows_tiles(const RowsGemm& a, int quant_type, bool f16, hipStream_t stream,
                             bool launch) {
  const int64_t kLimit = (int64_t)1 << 31;
  if ((int64_t)a.N * (a.K / 2) >= kLimit) return hipErrorNotSupported;
  // 32-bit offsets into X: all of it where rows are looked up, one tile else
  const int64_t reach = a.gather > 0 ? a.x_rows : BM;
  if (reach * a.ldx * 2 >= kLimit) return hipErrorNotSupported;
  if (LORA && (int64_t)a.N * a.lora.ldb * 2 >= kLimit) return hipErrorNotSupported;
  const int tiles_n = (a.N - 1) / BN + 1;
  const unsigned grid = rows_grid(a.rows, a.groups, BM, tiles_n, kThreads);
  if (grid == 0) return hipErrorNotSupported;
  if (!launch) return hipSuccess;
  const LevelTable& lv = level_table(quant_type);
  // Four block codes per dword load, as in the ungrouped GEMM.
  const bool q4 = a.double_quant && (a.K / 64) % 4 == 0 && ((uintptr_t)a.absmax & 3) == 0;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(kThreads), 0, stream, a.x, a.ldx,
                       a.packed, a.absmax, a.absmax2, a.mean, a.rows, a.N, a.K, a.y, a.ldy, 0,
                       tiles_n, lv, LoraArgs{}, SplitArgs{}, a);
  };
  auto pick = [&](auto half) {
    constexpr bool F16 = decltype(half)::value;
    if (!a.double_quant) go(gemm_kernel<kDqNone, false, false, F16, LORA, false, true>);
    else if (a.double_quant == kDqDynamic && q4)
      go(gemm_kernel<kDqDynamic, true, false, F16, LORA, false, true>);
    else if (a.double_quant == kDqDynamic)
      go(gemm_kernel<kDqDynamic, false, false, F16, LORA, false, true>);
    else if (q4) go(gemm_kernel<kDqLinear, true, false, F16, LORA, false, true>);
    else go(gemm_kernel<kDqLinear, false, false, F16, LORA, false, true>);
  };
  if (f16) pick(std::true_type{});
  else pick(std::false_type{});
  return hipGetLastError();
}

}  // namespace
}  // namespace bnbx
