// Input gradient of the expert-grouped product over few rows a group, for
// gfx950: dX_i = dY_i . W_hat_g, i a place of group g, the weight streamed once
// per row tile of 32 places.
//
// Bound: the vector and LDS work of the dequant (2.4 vector instructions and
// half a b64 table read a weight).  Measured, 8 groups of 4096 x 4096: 8 rows a
// group 26 us (2.7 TB/s), 50 rows 49 us.
//
// The contraction runs over the weight rows n, so an operand holds eight
// consecutive n of one column k.  A lane loads the same 8 columns (one dword)
// of 8 consecutive rows; the byte -> level pair table gives two columns of one
// row, two products scale them, and the conversion that packs two 16-bit values
// packs those of two neighbouring rows: the transpose costs nothing.  Lane (q,
// r) (q = lane / 16, r = lane % 16) holds rows 8 q .. 8 q + 7 and columns 8 r ..
// 8 r + 7 of a unit of 32 rows x 128 columns; v_mfma_f32_16x16x32 number j takes
// column 8 r + j of every lane, so its D has columns 8 (4 q + v) + j down the
// values and the places across the lanes, and the 8 accumulators of one v are 8
// neighbouring columns of dX.
//
// Waves share nothing but the table: the WS waves of a workgroup own the same
// 128 columns and take every WS-th unit of 32 rows.  dY is loaded quad-coalesced
// (lane x: 16 bytes of place x / 4: 22 cycles of the CU's address path a load,
// against 67 with every lane on a line of its own, which bound the kernel) and
// turned to lane (q, r): place r, 16 bytes, through a 1 KB stage per wave.  The
// unit's 64 block scales are formed one a lane and turned through 256 bytes of
// LDS.  At the end the
// accumulators meet in LDS, pairwise in a fixed tree.
#include "bnbx_rows_device.hpp"

namespace bnbx {
namespace {

constexpr int kCols = 128, kUnit = 32;
constexpr int kAhead = 2;   // units loaded ahead
// 32 places a tile and 8 waves a workgroup at every size.  Measured on 8 experts
// of 4096 x 4096 in us, 8 / 50 / 128 rows a group: 16 places 27.9 / 81.9 / 176,
// 32 places 29.1 / 53.3 / 126, 64 places 43.7 / 88.6 / 142 (its accumulators
// spill); 16 waves spill, 4 waves 39.0 / 51.0 / 121.  (With the block scale
// formed without a branch, this form now takes 26 / 49 / 116.)
constexpr int RB = 2, TM = 16 * RB, WS = 8;

template <int DQ, bool F16>
__global__ __launch_bounds__(WS * 64) void rows_dx_stream_kernel(RowsGemm a, int tiles_k,
                                                                 LevelTable lv) {
  constexpr bool DYN = DQ == kDqDynamic;
  constexpr int kAcc = 8 * RB;                      // f32x4 a lane
  // LDS: the byte table (at offset 0), two scale sets and a stage a wave, the
  // dynamic map; the tree of sums reuses all of it.
  constexpr int kScl = kLutBytes, kStage = kScl + WS * 512, kMap = kStage + WS * 1024;
  constexpr int kUsed = kMap + (DYN ? 1024 : 0), kRed = WS / 2 * kAcc * 1024;
  __shared__ __attribute__((aligned(256))) unsigned char smem[kUsed > kRed ? kUsed : kRed];
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int r = lane & 15, q = lane >> 4;      // MFMA layout
  const int lr = lane >> 2, lp = lane & 3;     // load layout: row, piece

  RowTiles<TM> tiles{a.offsets, a.groups, a.rows};
  const int nt = tiles.count();
  const int id = xcd_item(nt * tiles_k);
  if (id < 0) return;
  // row tiles of one group and the same columns are neighbours
  const int tk = __builtin_amdgcn_readfirstlane((int)((uint32_t)id / (uint32_t)nt));
  const RowTile tile = tiles.find(id - tk * nt);
  const int k0 = tk * kCols;

  const float mu = DQ ? *a.mean : 0.0f;
  const uint32_t rowK2 = (uint32_t)a.K >> 1, nkb = (uint32_t)a.K >> 6;
  const uint32_t nblocks = (uint32_t)a.N * nkb;
  const int64_t blk0 = (int64_t)tile.g * nblocks;
  const rsrc_t rw = make_rsrc(a.packed + (int64_t)tile.g * a.N * rowK2, (uint32_t)a.N * rowK2);
  const rsrc_t rq = make_rsrc((const char*)a.absmax + blk0 * (DQ ? 1 : 4),
                              DQ ? nblocks : nblocks * 4u);
  const uint32_t grem = (uint32_t)(blk0 & 255);
  const rsrc_t rg = make_rsrc(DQ ? a.absmax2 + (blk0 >> 8) : nullptr,
                              DQ ? (grem + nblocks + 255u) / 256u * 4u : 0u);

  // Unit u: rows 32 u ..; columns past K read zeros and have scale zero.
  const int nunits = a.N / kUnit;
  const bool kin = k0 + 8 * r < a.K;
  const uint32_t wlane =
      kin ? (uint32_t)(8 * q) * rowK2 + (uint32_t)(k0 + 8 * r) / 2u : kFar;
  // the lane's own scale: row lane / 2, block lane % 2 of the unit
  const uint32_t sblk = (uint32_t)k0 / 64u + (uint32_t)(lane & 1);
  const bool sin = sblk < nkb;
  const uint32_t slane = (uint32_t)(lane >> 1) * nkb + sblk;
  struct Unit {
    uint32_t w[8];
    uint32_t q;
    float s;
    u32x4_t y[RB];
  };
  const uint16_t* yp[RB];
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    // places past the tile repeat its first row (never stored)
    const int place = tile.r0 + 16 * i + lr < tile.r1 ? tile.r0 + 16 * i + lr : tile.r0;
    int yr = x_row_of(a, place);
    yr = yr < 0 ? 0 : yr;
    yp[i] = a.x + (int64_t)yr * a.ldx + 8 * lp;
  }
  auto load = [&](Unit& u, int at) {
    at = at < nunits ? at : nunits - 1;   // past the end: never used
    const uint32_t so = (uint32_t)at * kUnit * rowK2;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      u.w[i] = __builtin_amdgcn_raw_buffer_load_b32(rw, wlane + (uint32_t)i * rowK2, so, 0);
    const uint32_t blk = slane + (uint32_t)at * kUnit * nkb;
    if (DQ) {
      u.q = __builtin_amdgcn_raw_buffer_load_b8(rq, sin ? blk : kFar, 0, 0);
      u.s = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(
                                          rg, sin ? ((grem + blk) >> 8) * 4u : kFar, 0, 0));
    } else {
      u.q = __builtin_amdgcn_raw_buffer_load_b32(rq, sin ? blk * 4u : kFar, 0, 0);
      u.s = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < RB; ++i) u.y[i] = *(const u32x4_t*)(yp[i] + at * kUnit);
  };
  float* const dmap = (float*)(smem + kMap);
  auto scale_of = [&](const Unit& u) {
    float sc;
    if (DYN) {
      const float prod = dmap[u.q & 0xffu] * u.s;
      sc = prod + mu;
    } else if (DQ) {
      sc = rows_dq_scale((float)(int8_t)(uint8_t)u.q, u.s, mu);
    } else {
      sc = __builtin_bit_cast(float, u.q);
    }
    return sin ? sc : 0.0f;
  };

  Unit un[kAhead];
#pragma unroll
  for (int p = 0; p < kAhead; ++p) load(un[p], wave + p * WS);
  lut_build(smem, lv, WS * 64);
  if (DYN)
    for (int e = t; e < 256; e += WS * 64) dmap[e] = kDynMapDev.v[e];
  __syncthreads();

  f32x4_t acc[8][RB];
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int i = 0; i < RB; ++i) acc[j][i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  const uint32_t lcol = 8u * (uint32_t)(lane & 31);
  float* const scl = (float*)(smem + kScl + wave * 512);   // two sets of [block][row]
  unsigned char* const stage = smem + kStage + wave * 1024;
  const uint32_t wslot = 16u * (uint32_t)(16 * lp + ((lr + 4 * lp) & 15));
  const uint32_t rslot = 16u * (uint32_t)(16 * q + ((r + 4 * q) & 15));
  auto mul = [&](Unit& u, int at, int set) {
    scl[64 * set + 32 * (lane & 1) + (lane >> 1)] = scale_of(u);
    const float4 s0 = *(const float4*)&scl[64 * set + 32 * (r >> 3) + 8 * q];
    const float4 s1 = *(const float4*)&scl[64 * set + 32 * (r >> 3) + 8 * q + 4];
    const float sc[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
    uint32_t w[8];
    u32x4_t y[RB];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = u.w[i];
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      *(u32x4_t*)(stage + wslot) = u.y[i];
      y[i] = *(const u32x4_t*)(stage + rslot);
    }
    load(u, at + kAhead * WS);
    float2 l2[2][8];
    auto look = [&](int e) {
#pragma unroll
      for (int i = 0; i < 8; ++i) l2[e & 1][i] = lut_pair(smem, w[i], lcol, e);
    };
    look(0);
#pragma unroll
    for (int e = 0; e < 4; ++e) {   // byte e: columns 2 e and 2 e + 1
      if (e < 3) look(e + 1);
      __builtin_amdgcn_sched_barrier(0);
      u32x4_t w0, w1;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const float2 la = l2[e & 1][2 * p], lb = l2[e & 1][2 * p + 1];
        w0[p] = pack16x2<F16>(la.x * sc[2 * p], lb.x * sc[2 * p + 1]);
        w1[p] = pack16x2<F16>(la.y * sc[2 * p], lb.y * sc[2 * p + 1]);
      }
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        acc[2 * e][i] = mfma_16x16x32<F16>(w0, y[i], acc[2 * e][i]);
        acc[2 * e + 1][i] = mfma_16x16x32<F16>(w1, y[i], acc[2 * e + 1][i]);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // No branch around a load, only out of the loop: the compiler's waits count
  // the loads issued since.
  for (int at = wave; at < nunits;) {
#pragma unroll
    for (int p = 0; p < kAhead; ++p) {
      mul(un[p], at, p & 1);
      at += WS;
      if (at >= nunits) break;
    }
  }

  // The tree: the upper half of the waves hands over, the lower half adds.
  f32x4_t* const red = (f32x4_t*)smem;
#pragma unroll
  for (int half = WS / 2; half >= 1; half /= 2) {
    __syncthreads();
    if (wave >= half && wave < 2 * half) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 0; i < RB; ++i)
          red[((wave - half) * kAcc + j * RB + i) * 64 + lane] = acc[j][i];
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int i = 0; i < RB; ++i) {
          const f32x4_t o = red[(wave * kAcc + j * RB + i) * 64 + lane];
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[j][i][v] += o[v];
        }
    }
  }
  if (wave != 0) return;

  // Lane (q, r): place r of each 16; value v of the 8 accumulators: columns
  // 8 (4 q + v) .. + 7.
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    const int place = tile.r0 + 16 * i + r;
    if (place >= tile.r1 || x_row_of(a, place) < 0) continue;
    const int row = y_row_of(a, place);
    if (row < 0) continue;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int k = k0 + 8 * (4 * q + v);
      if (k >= a.K) continue;   // K is a multiple of 64: all 8 or none
      uint16_t* const o = a.y + (int64_t)row * a.ldy + k;
      u32x4_t p;
#pragma unroll
      for (int e = 0; e < 4; ++e) p[e] = pack16x2<F16>(acc[2 * e][i][v], acc[2 * e + 1][i][v]);
      if (((uintptr_t)o & 15) == 0) {
        *(u32x4_t*)o = p;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          o[2 * e] = (uint16_t)p[e];
          o[2 * e + 1] = (uint16_t)(p[e] >> 16);
        }
      }
    }
  }
}

}  // namespace

hipError_t launch_rows_dx_stream(const RowsGemm& a, int quant_type, bool f16,
                                 hipStream_t stream) {
  const int tiles_k = (a.K - 1) / kCols + 1;
  const unsigned grid = rows_grid(a.rows, a.groups, TM, tiles_k, WS * 64);
  if (grid == 0) return hipErrorNotSupported;
  const LevelTable& lv = level_table(quant_type);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(WS * 64), 0, stream, a, tiles_k, lv);
  };
  if (a.double_quant == kDqNone) {
    if (f16) go(rows_dx_stream_kernel<kDqNone, true>);
    else go(rows_dx_stream_kernel<kDqNone, false>);
  } else if (a.double_quant == kDqLinear) {
    if (f16) go(rows_dx_stream_kernel<kDqLinear, true>);
    else go(rows_dx_stream_kernel<kDqLinear, false>);
  } else {
    if (f16) go(rows_dx_stream_kernel<kDqDynamic, true>);
    else go(rows_dx_stream_kernel<kDqDynamic, false>);
  }
  return hipGetLastError();
}

}  // namespace bnbx
