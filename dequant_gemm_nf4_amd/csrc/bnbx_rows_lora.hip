// Down-projections of many adapters for gfx950: for place i of adapter g,
//   XA_i = s_g (X_i . A_g^T)   (A_g [r, K], fp32 accumulation),
// stored as two bf16 planes, hi = bf16(XA) and lo = bf16(XA - hi): together 16
// significant bits, in bf16's range, so that neither compute type costs the
// low-rank term accuracy or range before it joins the 4-bit product.  An
// infinity or NaN is held in lo, beside hi = +-2^-126: of the up-projection's
// products hi . B, lo . B and (fp16, B's own low part) hi . B_lo, the last must
// not see it (B_lo may be zero), and the first gives an infinite B its sign.
//
// Bound: reading the adapters' A (a decode batch reads a new A for nearly every
// row) or X (a prefill), and at one token the latency of one dependent load
// chain.  A workgroup of 16 waves takes 16 places of one adapter and 16 RT
// ranks; wave w takes the w-th of 16 parts of K, in steps of 32 k: one
// v_mfma_f32_16x16x32 per 16 ranks, A rows as its first operand and X rows as
// its second, so that lane (q, r) ends with ranks 4 q .. 4 q + 3 of place r.
// Loads are quad-coalesced and turned into the MFMA layout through a 1 KB
// stage per wave (as in the single adapter's down-projection).  Partial sums
// meet in LDS in wave order.  Measured: 1 row, K = 4096, rank 16, 6 us; 16 rows
// of 32 adapters of rank 64 7 us; 2048 rows, K = 8192, 8 adapters of rank 64 27 us.
#include "bnbx_rows_device.hpp"

namespace bnbx {
namespace {

constexpr int kWaves = 16, kThreads = kWaves * 64;
constexpr int kTile = 16;

template <bool F16, int RT>
__global__ __launch_bounds__(kThreads) void rows_lora_down_kernel(RowsGemm a, LoraDown d,
                                                                  int rank_tiles,
                                                                  uint16_t* __restrict__ xa) {
  constexpr int U = RT == 1 ? 4 : 1;   // steps loaded at once
  __shared__ f32x4_t red[kWaves][RT][64];
  __shared__ __attribute__((aligned(16))) unsigned char stages[kWaves][1024];
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  RowTiles<kTile> tiles{d.offsets, d.adapters, a.rows};
  const int nt = tiles.count();
  const int id = xcd_item(nt * rank_tiles);
  if (id < 0) return;
  // the rank tiles of one row tile are neighbours: they share X
  const RowTile tile = tiles.find(__builtin_amdgcn_readfirstlane(id / rank_tiles));
  const int c0 = __builtin_amdgcn_readfirstlane(id % rank_tiles) * 16 * RT;

  unsigned char* const stage = stages[wave];
  const int lr = lane >> 2, lp = lane & 3;   // load layout: row, piece
  const int r = lane & 15, q = lane >> 4;    // MFMA layout
  const uint32_t wslot = 16u * (uint32_t)(16 * lp + ((lr + 4 * lp) & 15));
  const uint32_t rslot = 16u * (uint32_t)(16 * q + ((r + 4 * q) & 15));
  auto relayout = [&](u32x4_t v) {
    *(u32x4_t*)(stage + wslot) = v;
    return *(const u32x4_t*)(stage + rslot);
  };

  // Rows past the tile repeat its first row (never stored), ranks past r
  // repeat rank 0 of the tile (never stored either).
  const int place = tile.r0 + lr < tile.r1 ? tile.r0 + lr : tile.r0;
  int xr = x_row_of(a, place);
  xr = xr < 0 ? 0 : xr;
  const uint16_t* const xp = a.x + (int64_t)xr * a.ldx + 8 * lp;
  const uint16_t* ap[RT];
#pragma unroll
  for (int c = 0; c < RT; ++c) {
    const int rank = c0 + 16 * c + lr < d.r ? c0 + 16 * c + lr : 0;
    ap[c] = d.a + (int64_t)tile.g * d.stride_a + (int64_t)rank * d.lda + 8 * lp;
  }

  f32x4_t acc[RT];
#pragma unroll
  for (int c = 0; c < RT; ++c) acc[c] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  const int kq = ((a.K + kWaves - 1) / kWaves + 31) / 32 * 32;
  const int k0 = wave * kq < a.K ? wave * kq : a.K;
  const int k1 = k0 + kq < a.K ? k0 + kq : a.K;
  struct Grp {
    u32x4_t x[U];
    u32x4_t w[U][RT];
  };
  auto load = [&](Grp& g, int k) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k + 32 * u >= k1) break;   // uniform in the wave
      g.x[u] = *(const u32x4_t*)(xp + k + 32 * u);
#pragma unroll
      for (int c = 0; c < RT; ++c) g.w[u][c] = *(const u32x4_t*)(ap[c] + k + 32 * u);
    }
  };
  auto mul = [&](const Grp& g, int k) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (k + 32 * u >= k1) break;
      const u32x4_t xv = relayout(g.x[u]);
#pragma unroll
      for (int c = 0; c < RT; ++c) acc[c] = mfma_16x16x32<F16>(relayout(g.w[u][c]), xv, acc[c]);
    }
  };
  Grp g0, g1;
  load(g0, k0);
  for (int k = k0; k < k1; k += 64 * U) {
    load(g1, k + 32 * U);
    mul(g0, k);
    load(g0, k + 64 * U);
    mul(g1, k + 32 * U);
  }

#pragma unroll
  for (int c = 0; c < RT; ++c) red[wave][c][lane] = acc[c];
  __syncthreads();
  const float s = d.scale[tile.g];
  // Output e: ranks tile e / 256, lane (e / 4) % 64, value e % 4.
  for (int e = t; e < RT * 256; e += kThreads) {
    const int c = e >> 8, l = (e >> 2) & 63, v = e & 3;
    const int p = tile.r0 + (l & 15), rank = c0 + 16 * c + 4 * (l >> 4) + v;
    if (p < tile.r1 && rank < d.r) {
      float sum = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) sum += red[w][c][l][v];
      const float o = s * sum;
      uint16_t hi = f32_to_bf16(o);
      uint16_t lo = f32_to_bf16(o - bf16lo_to_f32(hi));
      if ((hi & 0x7f80) == 0x7f80) {   // infinite or NaN: in the lo plane
        lo = hi;
        hi = (uint16_t)((hi & 0x8000) | 0x0080);
      }
      uint16_t* const out = xa + (int64_t)p * 2 * d.r + rank;
      out[0] = hi;
      out[d.r] = lo;
    }
  }
}

}  // namespace

hipError_t launch_rows_lora_down(const RowsGemm& a, const LoraDown& d, bool f16, int cus,
                                 uint16_t* xa, hipStream_t stream, bool launch) {
  const int64_t most = a.rows / kTile + (d.adapters < a.rows ? d.adapters : a.rows);
  // Four rank tiles a workgroup read X once for 64 ranks; one a workgroup
  // while the row tiles alone leave CUs idle.
  const bool wide = most >= cus;
  const int rt = wide ? 4 : 1;
  const int rank_tiles = (d.r + 16 * rt - 1) / (16 * rt);
  const unsigned grid = rows_grid(a.rows, d.adapters, kTile, rank_tiles, kThreads);
  if (grid == 0) return hipErrorNotSupported;
  if (!launch) return hipSuccess;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(kThreads), 0, stream, a, d, rank_tiles,
                       xa);
  };
  if (f16) {
    if (wide) go(rows_lora_down_kernel<true, 4>);
    else go(rows_lora_down_kernel<true, 1>);
  } else {
    if (wide) go(rows_lora_down_kernel<false, 4>);
    else go(rows_lora_down_kernel<false, 1>);
  }
  return hipGetLastError();
}

}  // namespace bnbx
