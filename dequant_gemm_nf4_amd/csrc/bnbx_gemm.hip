// Prefill GEMM with NF4 weights (the kernel: bnbx_gemm_core.hpp): the
// split-K reduction, the plans and the launches.
#include "bnbx_gemm_core.hpp"

namespace bnbx {
namespace {

// Split K: the fp32 partial tiles of the tail tiles, added in split order
// and rounded once; four columns per thread, only rows and columns inside
// Y are stored.
template <bool F16>
__global__ __launch_bounds__(256) void split_reduce_kernel(const float* __restrict__ part,
                                                           int nsplit, int ntail, int tile0,
                                                           int tiles_n, int M, int N,
                                                           uint16_t* __restrict__ y,
                                                           int64_t ldy) {
  constexpr int kQuads = BM * BN / 4;   // per tile
  const int64_t idx = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int t = (int)(idx / kQuads);
  if (t >= ntail) return;
  const int e = (int)(idx - (int64_t)t * kQuads) * 4;
  const int tile = tile0 + t;
  const int r = (tile / tiles_n) * BM + e / BN;
  const int c = (tile % tiles_n) * BN + e % BN;
  if (r >= M) return;
  float4 a = *(const float4*)(part + (int64_t)t * BM * BN + e);
  for (int s = 1; s < nsplit; ++s) {
    const float4 b4 = *(const float4*)(part + ((int64_t)s * ntail + t) * BM * BN + e);
    a.x += b4.x;
    a.y += b4.y;
    a.z += b4.z;
    a.w += b4.w;
  }
  const float v[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (c + k < N) y[(int64_t)r * ldy + c + k] = f32_to_16<F16>(v[k]);
}

int device_cus() {
  static int n = 0;
  if (n == 0) {
    int dev = 0, v = 0;
    if (hipGetDevice(&dev) == hipSuccess &&
        hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) == hipSuccess &&
        v > 0)
      n = v;
    else
      n = 256;
  }
  return n;
}

// Split-K plan (K of at least 32 blocks).  Tiles that fill at most half of
// the CUs all split, into up to four ranges; more tiles than CUs but fewer
// than twice as many run the first round whole (tile0 = the CUs, rounded
// down to a multiple of 8) and split the tail tiles, whose round would
// otherwise leave most CUs idle.  Ranges are multiples of 4 steps, at least
// 16.  Returns the partial tiles' bytes, 0 without a split.
struct SplitPlan {
  int nsplit, kb_per, tile0, ntail, per_xcd;
};
size_t split_plan(int M, int N, int K, SplitPlan& sp) {
  sp = SplitPlan{1, 0, 0, 0, 0};
  const int64_t tiles = (int64_t)((M + BM - 1) / BM) * ((N + BN - 1) / BN);
  const int nkb = K / 64;
  const int cus = device_cus();
  if (nkb < 32) return 0;
  int64_t tile0 = 0;
  if (tiles * 2 > cus) {
    if (tiles <= cus || tiles >= 2 * (int64_t)cus) return 0;
    tile0 = cus / kXcds * kXcds;
  }
  const int64_t ntail = tiles - tile0;
  if (ntail < 1 || ntail * 2 > cus) return 0;
  int s = (int)(cus / ntail);
  s = s < 4 ? s : 4;
  s = s < nkb / 16 ? s : nkb / 16;
  if (s < 2) return 0;
  const int kb_per = ((nkb + s - 1) / s + 3) / 4 * 4;
  const int n = (nkb + kb_per - 1) / kb_per;
  if (n < 2) return 0;
  sp.nsplit = n;
  sp.kb_per = kb_per;
  sp.tile0 = (int)tile0;
  sp.ntail = (int)ntail;
  sp.per_xcd = (int)((ntail + kXcds - 1) / kXcds);
  return (size_t)n * (size_t)ntail * BM * BN * sizeof(float);
}

template <int DQ, bool Q4, bool LORA>
void launch_one(const uint16_t* x, int64_t ldx, const uint8_t* packed, const void* absmax,
                const float* absmax2, const float* mean, int M, int N, int K, uint16_t* y,
                int64_t ldy, int quant_type, bool f16, const LoraArgs& la, const SplitPlan& plan,
                float* part, hipStream_t stream) {
  const int tm = (M + BM - 1) / BM, tn = (N + BN - 1) / BN;
  const int per_xcd = (tm * tn + kXcds - 1) / kXcds;
  const LevelTable& lv = level_table(quant_type);
  if constexpr (!LORA) {
    if (plan.nsplit > 1) {
      const SplitArgs sa{plan.kb_per, plan.tile0, plan.per_xcd, plan.ntail, part};
      const unsigned grid = (unsigned)(plan.tile0 + plan.nsplit * plan.per_xcd * kXcds);
      auto go = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(grid), dim3(kThreads), 0, stream, x, ldx, packed,
                           absmax, absmax2, mean, M, N, K, y, ldy, tm, tn, lv, la, sa, NoRows{});
      };
      if (quant_type == kQuantFP4) {
        if (f16) go(gemm_kernel<DQ, Q4, true, true, false, true>);
        else go(gemm_kernel<DQ, Q4, true, false, false, true>);
      } else {
        if (f16) go(gemm_kernel<DQ, Q4, false, true, false, true>);
        else go(gemm_kernel<DQ, Q4, false, false, false, true>);
      }
      const int64_t quads = (int64_t)plan.ntail * (BM * BN / 4);
      const unsigned rgrid = (unsigned)((quads + 255) / 256);
      if (f16)
        hipLaunchKernelGGL(split_reduce_kernel<true>, dim3(rgrid), dim3(256), 0, stream, part,
                           plan.nsplit, plan.ntail, plan.tile0, tn, M, N, y, ldy);
      else
        hipLaunchKernelGGL(split_reduce_kernel<false>, dim3(rgrid), dim3(256), 0, stream, part,
                           plan.nsplit, plan.ntail, plan.tile0, tn, M, N, y, ldy);
      return;
    }
  }
  const SplitArgs none{0, 0, 0, 0, nullptr};
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)(per_xcd * kXcds)), dim3(kThreads), 0, stream, x,
                       ldx, packed, absmax, absmax2, mean, M, N, K, y, ldy, tm, tn, lv, la, none, NoRows{});
  };
  if (quant_type == kQuantFP4) {
    if (f16) go(gemm_kernel<DQ, Q4, true, true, LORA, false>);
    else go(gemm_kernel<DQ, Q4, true, false, LORA, false>);
  } else {
    if (f16) go(gemm_kernel<DQ, Q4, false, true, LORA, false>);
    else go(gemm_kernel<DQ, Q4, false, false, LORA, false>);
  }
}

// The M-slab loop of both entry points.  Split K (no LoRA term) needs one
// slab and a workspace of split_plan's size; otherwise the tiles run whole.
template <bool LORA>
hipError_t launch_gemm_any(const uint16_t* x, int64_t ldx, const uint8_t* packed,
                           const void* absmax, const float* absmax2, const float* mean,
                           int double_quant, int quant_type, bool f16, int M, int N, int K,
                           uint16_t* y, int64_t ldy, LoraArgs la, void* workspace,
                           size_t workspace_bytes, hipStream_t stream) {
  // Buffer offsets are 32-bit: the weights and their scales must fit, and M
  // is walked in slabs whose X (and XA) rows do.
  const int64_t kLimit = (int64_t)1 << 31;
  if ((int64_t)N * (K / 2) >= kLimit) return hipErrorNotSupported;
  if (LORA && (int64_t)N * la.ldb * 2 >= kLimit) return hipErrorNotSupported;
  int64_t slab = (kLimit - (int64_t)K * 2) / (ldx * 2);
  if (LORA) {
    const int64_t s2 = (kLimit - (int64_t)la.r * 2) / (la.ldxa * 2);
    slab = s2 < slab ? s2 : slab;
  }
  slab = slab / BM * BM;
  if (slab < BM) return hipErrorNotSupported;
  SplitPlan plan;
  const size_t need = LORA ? 0 : split_plan(M, N, K, plan);
  if (need == 0 || M > slab || workspace == nullptr || workspace_bytes < need ||
      ((uintptr_t)workspace & 15) != 0)
    plan = SplitPlan{1, 0, 0, 0, 0};
  const int nkb = K / 64;
  // Four block codes per dword load: needs whole groups of four blocks per
  // row (then four blocks never straddle a group of 256) and an aligned
  // code array.
  const bool q4 = double_quant && nkb % 4 == 0 && ((uintptr_t)absmax & 3) == 0;
  float* part = (float*)workspace;
  for (int64_t r0 = 0; r0 < M; r0 += slab) {
    const int m = (int)(M - r0 < slab ? M - r0 : slab);
    const uint16_t* xs = x + r0 * ldx;
    uint16_t* ys = y + r0 * ldy;
    LoraArgs ls = la;
    if (LORA) ls.xa = la.xa + r0 * la.ldxa;
    if (!double_quant)
      launch_one<kDqNone, false, LORA>(xs, ldx, packed, absmax, absmax2, mean, m, N, K, ys, ldy,
                                       quant_type, f16, ls, plan, part, stream);
    else if (double_quant == kDqDynamic && q4)
      launch_one<kDqDynamic, true, LORA>(xs, ldx, packed, absmax, absmax2, mean, m, N, K, ys,
                                         ldy, quant_type, f16, ls, plan, part, stream);
    else if (double_quant == kDqDynamic)
      launch_one<kDqDynamic, false, LORA>(xs, ldx, packed, absmax, absmax2, mean, m, N, K, ys,
                                          ldy, quant_type, f16, ls, plan, part, stream);
    else if (q4)
      launch_one<kDqLinear, true, LORA>(xs, ldx, packed, absmax, absmax2, mean, m, N, K, ys, ldy,
                                        quant_type, f16, ls, plan, part, stream);
    else
      launch_one<kDqLinear, false, LORA>(xs, ldx, packed, absmax, absmax2, mean, m, N, K, ys,
                                         ldy, quant_type, f16, ls, plan, part, stream);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

size_t gemm_workspace_bytes(int M, int N, int K) {
  SplitPlan plan;
  return split_plan(M, N, K, plan);
}

hipError_t launch_gemm(const uint16_t* x, int64_t ldx, const uint8_t* packed, const void* absmax,
                       const float* absmax2, const float* mean, int double_quant, int quant_type,
                       bool f16, int M, int N, int K, uint16_t* y, int64_t ldy, void* workspace,
                       size_t workspace_bytes, hipStream_t stream) {
  return launch_gemm_any<false>(x, ldx, packed, absmax, absmax2, mean, double_quant, quant_type,
                                f16, M, N, K, y, ldy, LoraArgs{nullptr, 0, nullptr, 0, 0},
                                workspace, workspace_bytes, stream);
}

hipError_t launch_gemm_lora(const uint16_t* x, int64_t ldx, const uint8_t* packed,
                            const void* absmax, const float* absmax2, const float* mean,
                            int double_quant, int quant_type, bool f16, int M, int N, int K,
                            const uint16_t* xa, int64_t ldxa, const uint16_t* lora_b,
                            int64_t ldb, int r, uint16_t* y, int64_t ldy, hipStream_t stream) {
  return launch_gemm_any<true>(x, ldx, packed, absmax, absmax2, mean, double_quant, quant_type,
                               f16, M, N, K, y, ldy, LoraArgs{xa, ldxa, lora_b, ldb, r}, nullptr,
                               0, stream);
}

}  // namespace bnbx
