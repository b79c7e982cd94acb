// Products of 16-bit gradients with the values of int8 codes, for gfx950:
//   out[r, c] = sum_t A(r, t) v(t, c),   v(t, c) = rnd16(fl32(code_tc * scale_t)),
// the input gradient of the 8-bit layer (A = dY, the codes its weight's) and the
// weight's gradient from saved activations (A = dY^T, `TURNED`, the codes X's).
//
// The sum runs over the rows of the codes, so a matrix instruction wants eight
// rows of one column in a lane: both operands that lie row by row are read from
// LDS by the transposing reads (ds_read_b64_tr_b8 / _b16).
//
// Tiling.  A workgroup owns 32 FR rows r by 128 FC columns c.  Four of its waves
// multiply (in all but the largest tile four more copy for them), each all the rows
// and 32 FC columns, so every code is read, converted and scaled by one wave only,
// straight into operand registers, and A's operands are shared by all four.  The codes are the A operand of v_mfma_f32_32x32x16: a lane
// then holds four consecutive columns of one row.  t is walked in steps of 64,
// four substeps of 16.
//
// All operands go from global memory straight into LDS, three or four buffers;
// 16-byte chunks are permuted by their row so that the reads below meet every bank
// evenly (which rows a read meets is said at each).  Rows t past the end read as zero
// codes, scales and gradients.  The pipeline is that of the forward product: the
// operands of a substep are read and the codes converted during the products of the
// one before, with one wait and barrier a step before the last substep.
//
// What bounds it (4096 x 11008 x 4096, timed in copies with a part taken out): the
// products with their reads 230 us, the copies 200, the conversion 30, which overlap
// to 295-310 us by the card's state, 1.19-1.25 PFLOP/s; a large bf16 library product of
// that shape runs at 0.92.
#include <type_traits>

#include "bnbx_int8_device.hpp"
#include "bnbx_int8_form.hpp"

namespace bnbx {
namespace {

constexpr int kThreads = 256;   // of the reduction
constexpr int BT = kInt8GradStep;
typedef __attribute__((ext_vector_type(4))) short s16x4_t;
typedef __attribute__((ext_vector_type(2))) int i32x2_t;

struct GradArgs {
  const uint16_t* dy;
  int64_t ldy;
  const int8_t* codes;
  const float* scale;
  int64_t ldv;
  int R, C, T;
  void* out;
  int64_t ldo;
  int tiles_r, tiles_c;
  int splits, steps_per;
  float* part;   // [splits][R][ldp] (splits > 1)
  int64_t ldp;
};

__device__ __forceinline__ u32x2_t read_tr8(const uint8_t* p) {
  return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                                         (__attribute__((address_space(3))) i32x2_t*)p));
}
__device__ __forceinline__ u32x2_t read_tr16(const uint8_t* p) {
  return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                                         (__attribute__((address_space(3))) s16x4_t*)p));
}

// Four values of a row, `left` of them inside it.
template <int OUT>
__device__ __forceinline__ void store4(void* out, int64_t at, f32x4_t v, int left, bool vec) {
  if constexpr (OUT == kOutF32) {
    float* o = (float*)out + at;
    if (vec && left >= 4) {
      *(f32x4_t*)o = v;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < left) o[e] = v[e];
    }
  } else {
    uint16_t* o = (uint16_t*)out + at;
    const u32x2_t p = {pack16x2<OUT == kOutF16>(v[0], v[1]), pack16x2<OUT == kOutF16>(v[2], v[3])};
    if (vec && left >= 4) {
      *(u32x2_t*)o = p;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < left) o[e] = (uint16_t)(p[e / 2] >> (16 * (e & 1)));
    }
  }
}
template <int OUT>
__device__ __forceinline__ bool whole4(const void* out, int64_t ldo) {
  return (uintptr_t)out % (OUT == kOutF32 ? 16 : 8) == 0 && ldo % 4 == 0;
}

// ND: buffers, 3 or 4.  LOAD: four more waves make all the copies, so that a wave
// that multiplies never waits to hand one over (with the largest tile a wave's
// registers leave no room for them).  OUT: kOutBf16 / kOutF16 / kOutF32; SPLIT: fp32
// partial sums instead.
template <int FR, int FC, int ND, bool LOAD, bool TURNED, bool F16, int OUT, bool SPLIT>
__global__ __launch_bounds__(LOAD ? 512 : 256) void int8_grad_kernel(GradArgs a) {
  constexpr int TR = 32 * FR, TC = 128 * FC;
  constexpr int CW = 4;   // waves that copy: those that multiply, or the four behind them
  constexpr int kA = TR * BT * 2, kV = BT * TC, kBuf = kA + kV + CW * BT * 4;
  constexpr int CA = FR, CV = 2 * FC;   // copies of such a wave and step
  __shared__ __attribute__((aligned(16))) uint8_t buf0[kBuf];
  __shared__ __attribute__((aligned(16))) uint8_t buf1[kBuf];
  __shared__ __attribute__((aligned(16))) uint8_t buf2[ND > 2 ? kBuf : 16];
  __shared__ __attribute__((aligned(16))) uint8_t buf3[ND > 3 ? kBuf : 16];
  int tr, tc;
  if (!tile_of(blockIdx.x, a.tiles_r, a.tiles_c, tr, tc)) return;
  const int r0 = tr * TR, c0 = tc * TC;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cw = wave & 3;   // its number among those that multiply, or copy
  const int col = lane & 31, half = lane >> 5;
  const int steps = (a.T + BT - 1) / BT;
  const int t0 = SPLIT ? (int)blockIdx.y * a.steps_per : 0;
  const int t1 = SPLIT ? (t0 + a.steps_per < steps ? t0 + a.steps_per : steps) : steps;

  // ---- copies -------------------------------------------------------------
  // Codes: rows t of TC bytes, chunk permuted by turn_v.
  constexpr int VCH = TC / 16, VR = 64 / VCH;   // chunks a row, rows an instruction
  auto turn_v = [](int t) { return FC == 2 ? 2 * (t & 7) : 2 * ((t >> 1) & 3); };
  const int cp = (a.C + 15) / 16 * 16;
  uint32_t voff[CV];
#pragma unroll
  for (int i = 0; i < CV; ++i) {
    const int t = (cw * CV + i) * VR + lane / VCH;
    const int ch = (lane % VCH) ^ turn_v(t);
    voff[i] = c0 + 16 * ch < cp ? (uint32_t)t * (uint32_t)a.ldv + 16u * ch : kFar8;
  }
  // Gradients.  Rows r of 64 t (128 bytes, chunk permuted by the row pair), or
  // rows t of TR values.
  constexpr int ACH = TURNED ? TR / 8 : 8, AR = 64 / ACH;
  auto turn_a = [](int row) {
    if (!TURNED) return (row >> 1) & 7;
    return FR >= 4 ? 4 * (row & 3) : FR == 2 ? 4 * ((row >> 1) & 1) : 0;
  };
  uint32_t aoff[CA];
#pragma unroll
  for (int i = 0; i < CA; ++i) {
    const int row = (cw * CA + i) * AR + lane / ACH;
    const int ch = (lane % ACH) ^ turn_a(row);
    const bool in = TURNED ? r0 + 8 * ch < a.R : r0 + row < a.R;
    aoff[i] = in ? (uint32_t)row * (uint32_t)a.ldy * 2u + 16u * ch : kFar8;
  }
  // !TURNED: the first t of this lane's chunk; odd instructions permute by 4 more
  const int ach0 = 8 * ((lane & 7) ^ ((lane >> 4) & 3));
  const rsrc8_t ra = rsrc8(a.dy + (int64_t)r0 * a.ldy, (int64_t)kFar8);
  const uint32_t ldv = (uint32_t)a.ldv, ldy2 = (uint32_t)a.ldy * 2u;
  // A step's source: rows t past the end are past the resources.
  struct Source {
    rsrc8_t v, s, y;
    uint32_t soff;
    bool ok0, ok1;
  };
  auto source = [&](int t) {
    int rows = a.T - t * BT;
    Source f;
    f.soff = (uint32_t)t * (BT * 2);
    f.ok0 = ach0 < rows;
    f.ok1 = (ach0 ^ 32) < rows;
    rows = rows < 0 ? 0 : rows < BT ? rows : BT;
    f.v = rsrc8_near(a.codes + c0 + (int64_t)t * BT * a.ldv, rows * ldv);
    f.s = rsrc8_near(a.scale + (int64_t)t * BT, rows * 4u);
    f.y = TURNED ? rsrc8_near(a.dy + r0 + (int64_t)t * BT * a.ldy, rows * ldy2) : ra;
    return f;
  };
  constexpr int C = CV + 1 + CA;
  auto copy = [&](uint8_t* to_buf, const Source& f, int i) {
    if (i < CV) {
      copy16_lds(f.v, to_buf + kA + (cw * CV + i) * 1024, voff[i], 0);
    } else if (i == CV) {
      copy4_lds(f.s, to_buf + kA + kV + cw * BT * 4, 4u * lane, 0);
    } else {
      i -= CV + 1;
      uint8_t* const to = to_buf + (cw * CA + i) * 1024;
      if constexpr (TURNED)
        copy16_lds(f.y, to, aoff[i], 0);
      else
        copy16_lds(f.y, to, (((cw * CA + i) & 1) ? f.ok1 : f.ok0) ? aoff[i] : kFar8, f.soff);
    }
  };

  // ---- operands -----------------------------------------------------------
  u32x4_t oa[2][FR];     // gradients
  u32x4_t ov[2][FC];     // values
  u32x2_t oc[FC];        // codes
  f32x4_t os[2];         // scales of the lane's eight t
  const int g = lane >> 4, l16 = lane & 15;
  // Codes: 16 lanes read eight rows t of 16 columns (two lanes a row), 32 lanes
  // eight rows of 32 bytes, each row in other banks.
  uint32_t vrd[FC];
  {
    const int t = 8 * (g >> 1) + (l16 >> 1);   // + 16 s, which leaves turn_v alone
#pragma unroll
    for (int f = 0; f < FC; ++f) {
      const int ch = ((cw * FC + f) * 2 + (g & 1)) ^ turn_v(t);
      vrd[f] = kA + t * TC + 16 * ch + 8 * (l16 & 1);
    }
  }
  const uint32_t srd = kA + kV + cw * BT * 4 + 32 * half;
  // Gradients: row col of a tile, chunk 2 s + half; or four rows t of 16 values in
  // 16 lanes (four lanes a row), twice, each row in other banks.  turn_a moves
  // whole groups of four chunks (two with FR = 2), so tiles four apart differ by a
  // constant.
  constexpr int SUB = 4;   // substeps of a step
  constexpr int NRD = TURNED ? (FR < 4 ? FR : 4) : SUB;
  uint32_t ard[NRD];
  if constexpr (TURNED) {
    const int t = 8 * (g >> 1) + (l16 >> 2);   // + 16 s + 4 j, the same turn_a for FR >= 4
#pragma unroll
    for (int f = 0; f < NRD; ++f)
      ard[f] = t * TR * 2 + 16 * ((4 * f + 2 * (g & 1) + ((l16 & 3) >> 1)) ^ turn_a(t)) +
               8 * (l16 & 1);
  } else {
#pragma unroll
    for (int s = 0; s < SUB; ++s)
      ard[s] = col * BT * 2 + 16 * ((2 * s + half) ^ turn_a(col));
  }
  // Read i of substep s: the codes, the scales, then the gradients.
  constexpr int NR = FC + 2 + FR;
  auto read = [&](const uint8_t* buf, int s, int set, int i) {
    if (i < FC) {
      oc[i] = read_tr8(buf + vrd[i] + 16 * s * TC);
    } else if (i < FC + 2) {
      os[i - FC] = *(const f32x4_t*)(buf + srd + 64 * s + 16 * (i - FC));
    } else {
      const int f = i - FC - 2;
      if constexpr (TURNED) {
        const uint8_t* p = buf + ard[f % NRD] + 16 * s * TR * 2 + f / NRD * 256;
        const u32x2_t lo = read_tr16(p), hi = read_tr16(p + 4 * TR * 2);
        oa[set][f] = u32x4_t{lo[0], lo[1], hi[0], hi[1]};
      } else {
        oa[set][f] = *(const u32x4_t*)(buf + 32 * f * BT * 2 + ard[s]);
      }
    }
  };
  // Pair i of the values.
  constexpr int NP = 4 * FC;
  auto convert = [&](int set, int i) {
    const int f = i / 4, p = i % 4;
    ov[set][f][p] =
        pack16x2<F16>(code_value(oc[f][p / 2], 2 * (p & 1), os[p / 2][2 * (p & 1)]),
                      code_value(oc[f][p / 2], 2 * (p & 1) + 1, os[p / 2][2 * (p & 1) + 1]));
  };
  f32x16_t acc[FC][FR];
#pragma unroll
  for (int i = 0; i < FC; ++i)
#pragma unroll
    for (int j = 0; j < FR; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
  // all but the last `out` of this wave's copies have landed, and every wave is here
  auto land = [&](auto out) {
    constexpr int n = decltype(out)::value;
    __builtin_amdgcn_s_waitcnt(0x0F70 | (n & 15) | (n >> 4) << 14);   // vmcnt(n)
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  };
  using All = std::integral_constant<int, 0>;

  // The copies of a step go out as its buffer is left: the first CL of them in the
  // last substep, the rest in the substeps after it.
  constexpr int CL = (C + 2) / 3, C0 = CL + (C - CL + 1) / 2;   // up to substep 0; then all
  using Ahead = std::integral_constant<int, LOAD ? 0 : (ND - 2) * C>;   // of later steps
  if constexpr (LOAD) {
    if (wave >= 4) {
      static_assert(ND == 4, "four buffers");
      auto step_of = [&](uint8_t* to, int t) {
        const Source f = source(t);
#pragma unroll
        for (int i = 0; i < C; ++i) copy(to, f, i);
      };
      step_of(buf0, t0);
      step_of(buf1, t0 + 1);
      step_of(buf2, t0 + 2);
      step_of(buf3, t0 + 3);
      land(std::integral_constant<int, 3 * C>{});
      auto turn = [&](int t, uint8_t* cur) {
        land(std::integral_constant<int, 2 * C>{});
        step_of(cur, t + 4);
      };
      int t = t0;
      for (; t + 3 < t1; t += 4) {
        turn(t, buf0);
        turn(t + 1, buf1);
        turn(t + 2, buf2);
        turn(t + 3, buf3);
      }
      if (t < t1) turn(t, buf0);
      if (t + 1 < t1) turn(t + 1, buf1);
      if (t + 2 < t1) turn(t + 2, buf2);
      land(All{});   // nothing is in flight
      return;
    }
  } else {
    static_assert(ND == 3, "three buffers");
    const Source f0 = source(t0), f1 = source(t0 + 1), f2 = source(t0 + 2);
#pragma unroll
    for (int i = 0; i < C; ++i) copy(buf0, f0, i);
#pragma unroll
    for (int i = 0; i < C; ++i) copy(buf1, f1, i);
#pragma unroll
    for (int i = 0; i < CL; ++i) copy(buf2, f2, i);
  }
  land(std::integral_constant<int, LOAD ? 0 : Ahead::value + CL>{});
#pragma unroll
  for (int i = 0; i < NR; ++i) read(buf0, 0, 0, i);
#pragma unroll
  for (int i = 0; i < NP; ++i) convert(0, i);

  auto step = [&](int t, uint8_t* last, uint8_t* cur, uint8_t* next) {
    Source f{};
    if constexpr (!LOAD) f = source(t + ND - 1);
#pragma unroll
    for (int s = 0; s < SUB; ++s) {
      const int set = s & 1;
      const bool end = s == SUB - 1;
      __builtin_amdgcn_sched_barrier(0);
      if (end) {
        land(Ahead{});
        if constexpr (!LOAD) f = source(t + ND);
      }
      uint8_t* const to = end ? cur : last;
      const int i0 = end ? 0 : s == 0 ? CL : s == 1 ? C0 : C;
      const int i1 = end ? CL : s == 0 ? C0 : C;
      // One product a slot, and between the products what the next substep needs:
      // its reads in the first half, the conversion in the second, and the copies.
      constexpr int N = FC * FR, H = N / 2;
#pragma unroll
      for (int q = 0; q < N; ++q) {
        const int j = q / FC, i = q % FC;
        acc[i][j] = mfma_32x32x16<F16>(ov[set][i], oa[set][j], acc[i][j]);
#pragma unroll
        for (int k = 0; k < NR; ++k)
          if (k * H / NR == q) read(end ? next : cur, end ? 0 : s + 1, set ^ 1, k);
#pragma unroll
        for (int k = 0; k < NP; ++k)
          if (H + k * (N - H) / NP == q) convert(set ^ 1, k);
#pragma unroll
        for (int k = i0; k < i1; ++k)
          if (!LOAD && (k - i0) * N / (i1 - i0) == q) copy(to, f, k);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  int t = t0;
  if constexpr (ND == 3) {
    for (; t + 2 < t1; t += 3) {
      step(t, buf2, buf0, buf1);
      step(t + 1, buf0, buf1, buf2);
      step(t + 2, buf1, buf2, buf0);
    }
    if (t < t1) step(t, buf2, buf0, buf1);
    if (t + 1 < t1) step(t + 1, buf0, buf1, buf2);
  } else {
    for (; t + 3 < t1; t += 4) {
      step(t, buf3, buf0, buf1);
      step(t + 1, buf0, buf1, buf2);
      step(t + 2, buf1, buf2, buf3);
      step(t + 3, buf2, buf3, buf0);
    }
    if (t < t1) step(t, buf3, buf0, buf1);
    if (t + 1 < t1) step(t + 1, buf0, buf1, buf2);
    if (t + 2 < t1) step(t + 2, buf1, buf2, buf3);
  }
  land(All{});   // every wave has read its operands, and no copy is in flight

  // ---- results: value 4 q + e of a tile is row col, column 8 q + 4 half + e ----
  // Through LDS, 32 rows at a time in a wave's own part of a buffer (16-byte chunks
  // permuted by the row), so that a row is written by neighbouring lanes.
  void* const out = SPLIT ? (void*)(a.part + (int64_t)blockIdx.y * a.R * a.ldp) : a.out;
  constexpr int KIND = SPLIT ? (int)kOutF32 : OUT;
  constexpr int OCH = 8 * FC, OR = 64 / OCH;   // chunks a row, rows an instruction
  static_assert(2 * 32 * OCH * 16 <= kBuf, "results of two waves fit a buffer");
  const int64_t ldo = SPLIT ? a.ldp : a.ldo;
  const int cend = SPLIT ? (int)a.ldp : a.C;
  const bool vec = SPLIT || whole4<KIND>(out, ldo);
  auto turn_o = [](int row) { return FC == 2 ? row & 15 : (row >> 1) & 7; };
  uint8_t* const mine = (wave < 2 ? buf0 : buf1) + (wave & 1) * 32 * OCH * 16;
#pragma unroll
  for (int j = 0; j < FR; ++j) {
#pragma unroll
    for (int i = 0; i < FC; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4_t v = {acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                           acc[i][j][4 * q + 3]};
        *(f32x4_t*)(mine + 16 * (col * OCH + ((8 * i + 2 * q + half) ^ turn_o(col)))) = v;
      }
#pragma unroll 2
    for (int k = 0; k < 32 / OR; ++k) {
      const int row = k * OR + lane / OCH, ch = lane % OCH;
      const f32x4_t v = *(const f32x4_t*)(mine + 16 * (row * OCH + (ch ^ turn_o(row))));
      const int r = r0 + 32 * j + row, c = c0 + 32 * FC * cw + 4 * ch;
      if (r < a.R && c < cend) store4<KIND>(out, (int64_t)r * ldo + c, v, cend - c, vec);
    }
  }
}

// The splits of t added in order and rounded: a thread takes four columns, eight
// splits' loads under way at a time.
constexpr int kAtOnce = 8;
template <int OUT>
__global__ __launch_bounds__(kThreads) void int8_grad_reduce_kernel(GradArgs a) {
  const int quads = (a.C + 3) / 4;
  const int64_t total = (int64_t)a.R * quads;
  const bool vec = whole4<OUT>(a.out, a.ldo);
  for (int64_t q = (int64_t)blockIdx.x * kThreads + threadIdx.x; q < total;
       q += (int64_t)gridDim.x * kThreads) {
    const int64_t r = q / quads;
    const int c = 4 * (int)(q - r * quads);
    const float* p = a.part + r * a.ldp + c;
    const int64_t pitch = (int64_t)a.R * a.ldp;
    f32x4_t s = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int k = 0; k < a.splits; k += kAtOnce) {
      f32x4_t v[kAtOnce];
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i)
        v[i] = k + i < a.splits ? *(const f32x4_t*)(p + (k + i) * pitch) : f32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < kAtOnce; ++i) s += v[i];
    }
    store4<OUT>(a.out, r * a.ldo + c, s, a.C - c, vec);
  }
}

Int8Form form_of(int R, int C, int T) { return int8_grad_form(R, C, T, int8_cus()); }

template <bool TURNED, bool F16, int OUT, bool SPLIT>
hipError_t launch(const GradArgs& a, int shape, hipStream_t s) {
  const dim3 grid((a.tiles_r * a.tiles_c + kXcds - 1) / kXcds * kXcds, a.splits);
  switch (shape) {
    case 0: int8_grad_kernel<8, 2, 3, false, TURNED, F16, OUT, SPLIT><<<grid, 256, 0, s>>>(a); break;
    case 1: int8_grad_kernel<4, 2, 4, true, TURNED, F16, OUT, SPLIT><<<grid, 512, 0, s>>>(a); break;
    case 2: int8_grad_kernel<4, 1, 4, true, TURNED, F16, OUT, SPLIT><<<grid, 512, 0, s>>>(a); break;
    case 3: int8_grad_kernel<2, 1, 4, true, TURNED, F16, OUT, SPLIT><<<grid, 512, 0, s>>>(a); break;
    default: int8_grad_kernel<1, 1, 4, true, TURNED, F16, OUT, SPLIT><<<grid, 512, 0, s>>>(a);
  }
  return hipGetLastError();
}

template <bool TURNED, bool F16, int OUT>
hipError_t launch(const GradArgs& a, const Int8Form& f, hipStream_t s) {
  if (f.splits == 1) return launch<TURNED, F16, OUT, false>(a, f.shape, s);
  const hipError_t e = launch<TURNED, F16, kOutF32, true>(a, f.shape, s);
  if (e != hipSuccess) return e;
  const int64_t groups = ((int64_t)a.R * ((a.C + 3) / 4) + kThreads - 1) / kThreads;
  int8_grad_reduce_kernel<OUT>
      <<<(int)(groups < 65536 ? groups : 65536), kThreads, 0, s>>>(a);
  return hipGetLastError();
}

template <bool TURNED>
hipError_t launch(const GradArgs& a, const Int8Form& f, bool f16, int out, hipStream_t s) {
  if (out == kOutF32)
    return f16 ? launch<TURNED, true, kOutF32>(a, f, s) : launch<TURNED, false, kOutF32>(a, f, s);
  return f16 ? launch<TURNED, true, kOutF16>(a, f, s) : launch<TURNED, false, kOutBf16>(a, f, s);
}

}  // namespace

size_t int8_grad_workspace(int R, int C, int T) {
  const Int8Form f = form_of(R, C, T);
  return f.splits > 1 ? (size_t)f.splits * R * ((C + 3) / 4 * 4) * sizeof(float) : 0;
}

hipError_t launch_int8_grad(const GradGemm& g, bool turned, bool f16, void* workspace,
                            hipStream_t s) {
  const Int8Form f = form_of(g.R, g.v.cols, g.v.rows);
  GradArgs a{};
  a.dy = g.dy;
  a.ldy = g.ldy;
  a.codes = g.v.codes;
  a.scale = g.v.scale;
  a.ldv = g.v.ld;
  a.R = g.R;
  a.C = g.v.cols;
  a.T = g.v.rows;
  a.out = g.out;
  a.ldo = g.ldo;
  const int wide_r = kInt8GradShapes[f.shape].rows, wide_c = kInt8GradShapes[f.shape].cols;
  const int64_t tr = ((int64_t)a.R + wide_r - 1) / wide_r,
                tc = ((int64_t)a.C + wide_c - 1) / wide_c;
  if (!launch_fits((tr * tc + kXcds) * f.splits, 512)) return hipErrorNotSupported;
  a.tiles_r = (int)tr;
  a.tiles_c = (int)tc;
  a.splits = f.splits;
  a.steps_per = f.steps_per;
  a.part = (float*)workspace;
  a.ldp = (a.C + 3) / 4 * 4;
  return turned ? launch<true>(a, f, f16, g.out_type, s) : launch<false>(a, f, f16, g.out_type, s);
}

}  // namespace bnbx
