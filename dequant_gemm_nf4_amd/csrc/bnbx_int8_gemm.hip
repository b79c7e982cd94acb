// Y[M, N] = X . W^T over int8 codes with a scale for each row of both (the
// 8-bit linear layer), for gfx950.
//
// Tiling.  A workgroup of WN x WM waves owns TN rows of W by TM rows of X; a wave
// 32 FN by 32 FM, as FN x FM tiles of v_mfma_i32_32x32x32_i8 with W as the
// A operand: a lane then holds four consecutive n of one token.  K is walked in
// steps of 128 bytes (whole cache lines), four substeps of 32.
//
// Both operands go from global memory straight into LDS (buffer_load ... lds, 16
// bytes a lane), ND buffers.  A row is 128 bytes, its eight 16-byte chunks
// permuted by (row / 2) % 8, so that 16 lanes reading one chunk of 16 consecutive
// rows meet all 64 banks once.  Rows past the end and chunks past K read as zeros
// through the buffer range check.
//
// Pipeline of step t: substep s multiplies while the operands of substep s + 1
// are read; before substep 3 one wait and barrier (step t+1 has landed, every
// wave has read its last operands of step t), and under substep 3's products the
// first operands of step t+1 are read and the copies of step t+ND begin, into the
// buffer that step t has left.  The wait leaves the copies of later steps in flight:
// every memory operation of the loop is a copy into LDS, and these land in order.
//
// What bounds it: the large tiles the matrix units under the power limit (2048 x 8192
// x 8192 107-115 us by the card's state, 2.4-2.6 POP/s; the library's int8 product 118;
// copies and reads alone 96 us, products and reads alone 80-100), the small ones the
// copies (301 x 4096 x 11008 27-29 us; where the whole took 31, the copies alone took 31
// too and the rest alone 17): bytes come from behind L2 at 28-47 B/ns a CU (64 to 128 KB a CU under
// way), from L2 at 130, in this product's mixture of both at 73.
#include <type_traits>

#include "bnbx_int8_device.hpp"
#include "bnbx_int8_form.hpp"

namespace bnbx {
namespace {

constexpr int kThreads = 256;   // of the reduction
constexpr int BK = kInt8GemmStep;

// Scheduling-group masks (AMDGPU sched_group_barrier).
constexpr int kSgMfma = 0x008, kSgValu = 0x002, kSgSalu = 0x004, kSgVmem = 0x010,
              kSgDsRead = 0x100;

struct GemmArgs {
  const int8_t* x;
  const int8_t* w;
  const float* sx;
  const float* sw;
  int64_t ldx, ldw;
  int M, N, K;
  uint16_t* y;
  int64_t ldy;
  int tiles_m, tiles_n;
  int splits, steps_per;   // splits of K, steps of each
  int* part;               // [splits][M][ldp] (splits > 1)
  int64_t ldp;
};

// 16-bit results of four consecutive n.
template <bool F16>
__device__ __forceinline__ u32x2_t scaled4(const int* v, float sx, f32x4_t sw) {
  float f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = ((float)v[i] * sx) * sw[i];
  u32x2_t r = {pack16x2<F16>(f[0], f[1]), pack16x2<F16>(f[2], f[3])};
  return r;
}

// Eight results at y, `left` of them inside the row.
__device__ __forceinline__ void store8(uint16_t* y, u32x4_t v, int left, bool vec) {
  if (vec && left >= 8) {
    *(u32x4_t*)y = v;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) y[i] = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
  }
}

// ND: buffers, 2 to 4.
template <int FM, int FN, int WM, int WN, int ND, bool F16, bool SPLIT>
__global__ __launch_bounds__(64 * WM * WN) void int8_gemm_kernel(GemmArgs a) {
  constexpr int TM = 32 * FM * WM, TN = 32 * FN * WN, WV = WM * WN;
  constexpr int SUB = BK / 32, RCH = BK / 16, RI = 64 / RCH;   // RI: rows an instruction copies
  constexpr int CW = TN / RI / WV, CX = TM / RI / WV;          // copies a wave and step
  static_assert(CW * RI * WV == TN && CX * RI * WV == TM, "whole copies a wave");
  constexpr int kBuf = (TM + TN) * BK;
  __shared__ __attribute__((aligned(16))) uint8_t buf0[kBuf];
  __shared__ __attribute__((aligned(16))) uint8_t buf1[kBuf];
  __shared__ __attribute__((aligned(16))) uint8_t buf2[ND > 2 ? kBuf : 16];
  __shared__ __attribute__((aligned(16))) uint8_t buf3[ND > 3 ? kBuf : 16];
  // buffer k mod ND, known at compile time
  auto buf = [&](auto k) -> uint8_t* {
    constexpr int i = decltype(k)::value % ND;
    if constexpr (i == 0) return buf0;
    if constexpr (i == 1) return buf1;
    if constexpr (i == 2) return buf2;
    return buf3;
  };
  int tm, tn;
  if (!tile_of(blockIdx.x, a.tiles_m, a.tiles_n, tm, tn)) return;
  const int m0 = tm * TM, n0 = tn * TN;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 31, half = lane >> 5;
  const int wn = wave % WN * 32 * FN, wm = wave / WN * 32 * FM;   // the wave's corner
  const int steps = (a.K + BK - 1) / BK;
  const int t0 = SPLIT ? (int)blockIdx.y * a.steps_per : 0;
  const int t1 = SPLIT ? (t0 + a.steps_per < steps ? t0 + a.steps_per : steps) : steps;
  const int kp = (a.K + 15) / 16 * 16;

  // Copies: instruction i of a wave fills RI rows, lane l chunk slot l % RCH of row
  // l / RCH of them.  A row's chunks are permuted by turn(row).
  auto turn = [](int row) { return (row >> 1) & 7; };
  const rsrc8_t rw = rsrc8(a.w + (int64_t)n0 * a.ldw, (int64_t)kFar8);
  const rsrc8_t rx = rsrc8(a.x + (int64_t)m0 * a.ldx, (int64_t)kFar8);
  uint32_t off[CW + CX];
#pragma unroll
  for (int i = 0; i < CW + CX; ++i) {
    const bool isw = i < CW;
    const int r = (isw ? wave * CW + i : wave * CX + i - CW) * RI + lane / RCH;
    const int chunk = (lane % RCH) ^ turn(r);
    const bool in = isw ? n0 + r < a.N : m0 + r < a.M;
    off[i] = in ? (uint32_t)r * (uint32_t)(isw ? a.ldw : a.ldx) + 16u * chunk : kFar8;
  }
  // this lane's chunk in the even instructions, and in the odd ones (eight rows on)
  const int c0 = (lane % RCH) ^ turn(lane / RCH), c1 = c0 ^ 4;
  auto copies = [&](uint8_t* buf, int t, int i0, int i1) {
    const int left = kp - t * BK;
    const bool ok0 = 16 * c0 < left, ok1 = 16 * c1 < left;
#pragma unroll
    for (int i = i0; i < i1; ++i) {
      const int ri = i < CW ? wave * CW + i : wave * CX + i - CW;
      const uint32_t o = ((ri & 1) ? ok1 : ok0) ? off[i] : kFar8;
      copy16_lds(i < CW ? rw : rx, buf + ((i < CW ? 0 : TN) + ri * RI) * BK, o, (uint32_t)t * BK);
    }
  };

  // Operand reads: lane (col, half) takes chunk 2 s + half of row col of a tile.
  uint32_t rd[SUB];
#pragma unroll
  for (int s = 0; s < SUB; ++s) rd[s] = col * BK + 16 * ((2 * s + half) ^ turn(col));
  u32x4_t ow[2][FN], ox[2][FM];
  auto reads = [&](const uint8_t* buf, int s, int set) {
#pragma unroll
    for (int f = 0; f < FN; ++f) ow[set][f] = *(const u32x4_t*)(buf + (wn + 32 * f) * BK + rd[s]);
#pragma unroll
    for (int f = 0; f < FM; ++f)
      ox[set][f] = *(const u32x4_t*)(buf + (TN + wm + 32 * f) * BK + rd[s]);
  };
  i32x16_t acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0;
  auto products = [&](int set) {
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < FM; ++j) acc[i][j] = mfma_i8_32x32x32(ow[set][i], ox[set][j], acc[i][j]);
  };
  // all but the last `out` of this wave's copies have landed, and every wave is here
  auto land = [&](auto out) {
    constexpr int n = decltype(out)::value;
    static_assert(n < 64, "the memory counter");
    __builtin_amdgcn_s_waitcnt(0x0F70 | (n & 15) | (n >> 4) << 14);   // vmcnt(n)
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  };
  using All = std::integral_constant<int, 0>;

  // One substep's products with the operand reads of the next one and `nc` copies
  // laid between them.
  auto interleave = [&](int nc) {
    constexpr int N = FM * FN;
#pragma unroll
    for (int q = 0; q < N; ++q) {
      __builtin_amdgcn_sched_group_barrier(kSgMfma, 1, 0);
      if (q < FM + FN) __builtin_amdgcn_sched_group_barrier(kSgDsRead, 1, 0);
      if (q * nc / N != (q + 1) * nc / N) {
        __builtin_amdgcn_sched_group_barrier(kSgSalu, 1, 0);
        __builtin_amdgcn_sched_group_barrier(kSgValu, 1, 0);
        __builtin_amdgcn_sched_group_barrier(kSgVmem, 1, 0);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };

  constexpr int C = CW + CX;
  constexpr int CL = C / 2;   // copies of a step that go out in the last substep, as its
                              // buffer is left; the others in the next substep
  using Ahead = std::integral_constant<int, (ND - 2) * C>;   // copies of later steps
  in_turn<ND>([&](auto k) {
    copies(buf(k), t0 + k, 0, decltype(k)::value + 1 < ND ? C : CL);
  });
  land(std::integral_constant<int, (ND - 2) * C + CL>{});
  reads(buf0, 0, 0);
  // step t, in buffer k of ND
  auto step = [&](int t, auto at) {
    constexpr int k = decltype(at)::value;
    uint8_t* const last = buf(std::integral_constant<int, k + ND - 1>{});
    uint8_t* const cur = buf(at);
    uint8_t* const next = buf(std::integral_constant<int, k + 1>{});
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s < SUB; ++s) {
      const bool end = s == SUB - 1;
      if (s == 0) copies(last, t + ND - 1, CL, C);
      if (end) {
        land(Ahead{});
        copies(cur, t + ND, 0, CL);
      }
      reads(end ? next : cur, end ? 0 : s + 1, (s & 1) ^ 1);
      products(s & 1);
      interleave(end ? CL : s == 0 ? C - CL : 0);
    }
  };
  int t = t0;
  for (; t + ND <= t1; t += ND) in_turn<ND>([&](auto k) { step(t + k, k); });
  in_turn<ND - 1>([&](auto k) {
    if (t + k < t1) step(t + k, k);
  });

  land(All{});   // every wave has read its operands, and no copy is in flight
  if constexpr (SPLIT) {
    int* part = a.part + (int64_t)blockIdx.y * a.M * a.ldp;
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      const int m = m0 + wm + 32 * j + col;
      if (m >= a.M) continue;
#pragma unroll
      for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int n = n0 + wn + 32 * i + 8 * g + 4 * half;
          if (n < a.N) {
            const i32x4_t v = {acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2],
                               acc[i][j][4 * g + 3]};
            *(i32x4_t*)(part + (int64_t)m * a.ldp + n) = v;
          }
        }
    }
    return;
  }

  // Results through LDS, 32 tokens at a time in a wave's own part of a buffer: rows
  // of 32 FN values, 16-byte chunks permuted by the row, so that a row is written by
  // neighbouring lanes.
  constexpr int CH = 4 * FN;
  constexpr int PER = ND > 2 ? (WV + 1) / 2 : WV;   // waves a buffer serves
  static_assert(PER * 32 * CH * 16 <= kBuf && WV * 256 <= kBuf && TN <= 64 * WV,
                "results and scales fit a buffer");
  uint8_t* const mine = (wave < PER ? buf0 : buf2) + wave % PER * 32 * CH * 16;
  // the tile's scales of W (64 a wave, TN of them wanted), from the tile's first on: N
  // of them may be more than a resource's 2^31 bytes
  copy4_lds(rsrc8(a.sw + n0, (int64_t)(a.N - n0) * 4), buf1 + wave * 256,
            4u * (uint32_t)(64 * wave + lane), 0);
  land(All{});
  const bool vec = ((uintptr_t)a.y % 16 == 0) && a.ldy % 8 == 0;
#pragma unroll
  for (int j = 0; j < FM; ++j) {
    __builtin_amdgcn_sched_barrier(0);   // one tile's values in registers at a time
    const int mj = m0 + wm + 32 * j;
    const float sx = mj + col < a.M ? a.sx[mj + col] : 0.0f;
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        int v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = acc[i][j][4 * g + e];
        *(u32x2_t*)(mine + 16 * (col * CH + ((4 * i + g) ^ (col & (CH - 1)))) + 8 * half) =
            scaled4<F16>(v, sx, *(const f32x4_t*)(buf1 + 4 * (wn + 32 * i + 8 * g + 4 * half)));
      }
#pragma unroll 2
    for (int k = 0; k < 32 * CH / 64; ++k) {
      const int r = (k * 64 + lane) / CH, ch = lane % CH;
      const int m = mj + r, n = n0 + wn + 8 * ch;
      const u32x4_t v = *(const u32x4_t*)(mine + 16 * (r * CH + (ch ^ (r & (CH - 1)))));
      if (m < a.M && n < a.N) store8(a.y + (int64_t)m * a.ldy + n, v, a.N - n, vec);
    }
  }
}

// The splits of K added, scaled and rounded: a thread takes four n, eight splits'
// loads under way at a time.
constexpr int kAtOnce = 8;
template <bool F16>
__global__ __launch_bounds__(kThreads) void int8_reduce_kernel(GemmArgs a) {
  const int quads = (a.N + 3) / 4;
  const int64_t total = (int64_t)a.M * quads;
  for (int64_t q = (int64_t)blockIdx.x * kThreads + threadIdx.x; q < total;
       q += (int64_t)gridDim.x * kThreads) {
    const int m = (int)(q / quads), n = 4 * (int)(q - (int64_t)m * quads);
    const int* p = a.part + (int64_t)m * a.ldp + n;
    const int64_t pitch = (int64_t)a.M * a.ldp;
    i32x4_t s = {0, 0, 0, 0};
    for (int k = 0; k < a.splits; k += kAtOnce) {
      i32x4_t v[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i)
        v[i] = k + i < a.splits ? *(const i32x4_t*)(p + (k + i) * pitch) : i32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) s += v[i];
    }
    const float sx = a.sx[m];
    uint16_t* y = a.y + (int64_t)m * a.ldy + n;
    f32x4_t sw;
#pragma unroll
    for (int e = 0; e < 4; ++e) sw[e] = n + e < a.N ? a.sw[n + e] : 0.0f;
    const int v[4] = {s[0], s[1], s[2], s[3]};
    const u32x2_t r = scaled4<F16>(v, sx, sw);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < a.N) y[e] = (uint16_t)(r[e / 2] >> (16 * (e & 1)));
  }
}

Int8Form form_of(int M, int N, int K) { return int8_gemm_form(M, N, K, int8_cus()); }

void tiles_of(const Int8Form& f, int M, int N, int64_t& tm, int64_t& tn) {
  const Int8Shape& tile = kInt8GemmShapes[f.shape];
  tm = ((int64_t)M + tile.rows - 1) / tile.rows;
  tn = ((int64_t)N + tile.cols - 1) / tile.cols;
}

template <bool F16, bool SPLIT>
hipError_t launch(const GemmArgs& a, int shape, hipStream_t s) {
  const int total = a.tiles_m * a.tiles_n;
  const dim3 grid((total + kXcds - 1) / kXcds * kXcds, a.splits);
  switch (shape) {
    case 0: int8_gemm_kernel<4, 2, 2, 4, 2, F16, SPLIT><<<grid, 512, 0, s>>>(a); break;
    case 1: int8_gemm_kernel<2, 2, 4, 2, 3, F16, SPLIT><<<grid, 512, 0, s>>>(a); break;
    case 2: int8_gemm_kernel<2, 1, 2, 4, 4, F16, SPLIT><<<grid, 512, 0, s>>>(a); break;
    case 3: int8_gemm_kernel<2, 1, 2, 2, 4, F16, SPLIT><<<grid, 256, 0, s>>>(a); break;
    default: int8_gemm_kernel<1, 1, 2, 2, 4, F16, SPLIT><<<grid, 256, 0, s>>>(a);
  }
  return hipGetLastError();
}

}  // namespace

bool int8_gemm_fits(int M, int N, int K) {
  if (int8_rows16_takes(M)) return int8_rows16_fits(N);
  const Int8Form f = form_of(M, N, K);
  int64_t tm, tn;
  tiles_of(f, M, N, tm, tn);
  return launch_fits((tm * tn + kXcds) * f.splits, 512);
}

size_t int8_gemm_workspace(int M, int N, int K) {
  if (int8_rows16_takes(M)) return 0;
  const Int8Form f = form_of(M, N, K);
  return f.splits > 1 ? (size_t)f.splits * M * ((N + 3) / 4 * 4) * sizeof(int) : 0;
}

hipError_t launch_int8_gemm(const Int8Rows& x, const Int8Rows& w, uint16_t* y, int64_t ldy,
                            bool f16, void* workspace, hipStream_t s) {
  if (int8_rows16_takes(x.rows)) return launch_int8_rows16(x, w, y, ldy, f16, s);
  const Int8Form f = form_of(x.rows, w.rows, x.cols);
  GemmArgs a{};
  a.x = x.codes;
  a.w = w.codes;
  a.sx = x.scale;
  a.sw = w.scale;
  a.ldx = x.ld;
  a.ldw = w.ld;
  a.M = x.rows;
  a.N = w.rows;
  a.K = x.cols;
  a.y = y;
  a.ldy = ldy;
  int64_t tm, tn;
  tiles_of(f, a.M, a.N, tm, tn);
  a.tiles_m = (int)tm;
  a.tiles_n = (int)tn;
  a.splits = f.splits;
  a.steps_per = f.steps_per;
  a.part = (int*)workspace;
  a.ldp = (a.N + 3) / 4 * 4;
  if (f.splits == 1) return f16 ? launch<true, false>(a, f.shape, s) : launch<false, false>(a, f.shape, s);
  const hipError_t e = f16 ? launch<true, true>(a, f.shape, s) : launch<false, true>(a, f.shape, s);
  if (e != hipSuccess) return e;
  const int64_t quads = (int64_t)a.M * ((a.N + 3) / 4), groups = (quads + kThreads - 1) / kThreads;
  const int grid = (int)(groups < 65536 ? groups : 65536);
  if (f16)
    int8_reduce_kernel<true><<<grid, kThreads, 0, s>>>(a);
  else
    int8_reduce_kernel<false><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace bnbx
