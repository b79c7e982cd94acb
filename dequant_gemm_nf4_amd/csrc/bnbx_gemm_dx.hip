// Input gradient of the 4-bit linear layer, dX[M, K] = dY[M, N] . W_hat[N, K]
// (the kernel: bnbx_gemm_dx_core.hpp).
#include "bnbx_gemm_dx_core.hpp"

namespace bnbx {

hipError_t launch_gemm_dx(const uint16_t* dy, int64_t lddy, const uint8_t* packed,
                          const void* absmax, const float* absmax2, const float* mean,
                          int double_quant, int quant_type, bool f16, int M, int N, int K,
                          uint16_t* dx, int64_t lddx, hipStream_t stream) {
  const int64_t kLimit = (int64_t)1 << 31;
  if (N % TN != 0 || K % 64 != 0) return hipErrorNotSupported;
  if ((int64_t)N * (K / 2) >= kLimit) return hipErrorNotSupported;
  // dY offsets are 32-bit: walk M in slabs whose rows fit.
  int64_t slab = (kLimit - (int64_t)N * 2) / (lddy * 2);
  slab = slab / TM * TM;
  if (slab < TM) return hipErrorNotSupported;
  const LevelTable& lv = level_table(quant_type);
  for (int64_t r0 = 0; r0 < M; r0 += slab) {
    const int m = (int)(M - r0 < slab ? M - r0 : slab);
    const int tm = (m + TM - 1) / TM, tk = (K + TK - 1) / TK;
    const int per_xcd = (tm * tk + kXcds - 1) / kXcds;
    const uint16_t* dys = dy + r0 * lddy;
    uint16_t* dxs = dx + r0 * lddx;
    auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, dim3((unsigned)(per_xcd * kXcds)), dim3(kThreads), 0, stream,
                         dys, lddy, packed, absmax, absmax2, mean, m, N, K, dxs, lddx, tm, tk,
                         lv, NoRows{});
    };
    if (double_quant == kDqDynamic) {
      if (f16) go(gemm_dx_kernel<kDqDynamic, true>);
      else go(gemm_dx_kernel<kDqDynamic, false>);
    } else if (double_quant) {
      if (f16) go(gemm_dx_kernel<kDqLinear, true>);
      else go(gemm_dx_kernel<kDqLinear, false>);
    } else {
      if (f16) go(gemm_dx_kernel<kDqNone, true>);
      else go(gemm_dx_kernel<kDqNone, false>);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace bnbx
