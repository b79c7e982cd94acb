// Products of 16-bit gradients with the values of int8 codes, for gfx950:
//   out[r, c] = sum_t A(r, t) v(t, c),   v(t, c) = rnd16(fl32(code_tc * scale_t)),
// the input gradient of the 8-bit layer (A = dY, the codes its weight's) and the
// weight's gradient from saved activations (A = dY^T, `TURNED`, the codes X's).
//
// The sum runs over the rows of the codes, so a matrix instruction wants eight
// rows of one column in a lane: both operands that lie row by row are read from
// LDS by the transposing reads (ds_read_b64_tr_b8 / _b16).
//
// Tiling.  A workgroup of four waves owns 32 FR rows r by 128 FC columns c; a
// wave all its rows and 32 FC columns, so every code is read, converted and
// scaled by one wave only, straight into operand registers, and A's operands are
// shared by all four.  The codes are the A operand of v_mfma_f32_32x32x16: a lane
// then holds four consecutive columns of one row.  t is walked in steps of 64,
// four substeps of 16.
//
// All operands go from global memory straight into LDS, two buffers; 16-byte
// chunks are permuted by their row so that the reads below meet every bank evenly
// (which rows a read meets is said at each).  Rows t past the end read as zero
// codes, scales and gradients.  The pipeline is that of the forward product: the
// operands of a substep are read during the products of the one before, with one
// wait and barrier a step before the last substep.
#include <type_traits>

#include "bnbx_int8_device.hpp"

namespace bnbx {
namespace {

constexpr int kThreads = 256;
constexpr int BT = 64;
constexpr int kXcds = 8;

// Scheduling-group masks (AMDGPU sched_group_barrier).
constexpr int kSgMfma = 0x008, kSgValu = 0x002, kSgSalu = 0x004, kSgVmem = 0x010,
              kSgDsRead = 0x100;

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

// ND: buffers, 2 or 4.  OUT: kOutBf16 / kOutF16 / kOutF32; SPLIT: fp32 partial sums
// instead.
template <int FR, int FC, int ND, bool TURNED, bool F16, int OUT, bool SPLIT>
__global__ __launch_bounds__(kThreads) void int8_grad_kernel(GradArgs a) {
  constexpr int TR = 32 * FR, TC = 128 * FC;
  constexpr int kA = TR * BT * 2, kV = BT * TC, kBuf = kA + kV + 4 * BT * 4;
  constexpr int CA = FR, CV = 2 * FC;   // copies a wave and step
  __shared__ __attribute__((aligned(16))) uint8_t buf0[kBuf];
  __shared__ __attribute__((aligned(16))) uint8_t buf1[kBuf];
  __shared__ __attribute__((aligned(16))) uint8_t buf2[ND > 2 ? kBuf : 16];
  __shared__ __attribute__((aligned(16))) uint8_t buf3[ND > 2 ? kBuf : 16];
  // consecutive tiles (one band of rows r) on one XCD
  const int total = a.tiles_r * a.tiles_c, per = (total + kXcds - 1) / kXcds;
  const int id = (int)(blockIdx.x % kXcds) * per + (int)(blockIdx.x / kXcds);
  if ((int)(blockIdx.x / kXcds) >= per || id >= total) return;
  const int r0 = id / a.tiles_c * TR, c0 = id % a.tiles_c * TC;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 31, half = lane >> 5;
  const int steps = (a.T + BT - 1) / BT;
  const int t0 = SPLIT ? (int)blockIdx.y * a.steps_per : 0;
  const int t1 = SPLIT ? (t0 + a.steps_per < steps ? t0 + a.steps_per : steps) : steps;

  // ---- copies -------------------------------------------------------------
  // Codes: rows t of TC bytes, chunk permuted by kTurnV.
  constexpr int VCH = TC / 16, VR = 64 / VCH;   // chunks a row, rows an instruction
  auto turn_v = [](int t) { return FC == 2 ? 2 * (t & 7) : 2 * ((t >> 1) & 3); };
  const int cp = (a.C + 15) / 16 * 16;
  uint32_t voff[CV];
#pragma unroll
  for (int i = 0; i < CV; ++i) {
    const int t = (wave * CV + i) * VR + lane / VCH;
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
    const int row = (wave * CA + i) * AR + lane / ACH;
    const int ch = (lane % ACH) ^ turn_a(row);
    const bool in = TURNED ? r0 + 8 * ch < a.R : r0 + row < a.R;
    aoff[i] = in ? (uint32_t)row * (uint32_t)a.ldy * 2u + 16u * ch : kFar8;
  }
  // !TURNED: the first t of this lane's chunk; instructions 4 rows pairs apart
  // permute it by 4
  const int ach0 = 8 * ((lane & 7) ^ ((lane >> 4) & 3));
  const rsrc8_t ra = rsrc8(a.dy + (int64_t)r0 * a.ldy, (int64_t)kFar8);
  auto rows_left = [&](int t) {
    const int left = a.T - t * BT;
    return left < 0 ? 0 : left < BT ? left : BT;
  };
  auto copy_codes = [&](uint8_t* buf, int t) {
    const int rows = rows_left(t);
    const rsrc8_t rv = rsrc8(a.codes + c0 + (int64_t)t * BT * a.ldv, rows * a.ldv);
#pragma unroll
    for (int i = 0; i < CV; ++i) copy16_lds(rv, buf + kA + (wave * CV + i) * 1024, voff[i], 0);
    const rsrc8_t rs = rsrc8(a.scale + (int64_t)t * BT, rows * 4);
    copy4_lds(rs, buf + kA + kV + wave * BT * 4, 4u * lane, 0);
  };
  auto copy_dy = [&](uint8_t* buf, int t, int i0, int i1) {
    if constexpr (TURNED) {
      const rsrc8_t rt = rsrc8(a.dy + r0 + (int64_t)t * BT * a.ldy, rows_left(t) * a.ldy * 2);
#pragma unroll
      for (int i = i0; i < i1; ++i) copy16_lds(rt, buf + (wave * CA + i) * 1024, aoff[i], 0);
    } else {
      const int left = a.T - t * BT;
      const bool ok0 = ach0 < left, ok1 = (ach0 ^ 32) < left;
#pragma unroll
      for (int i = i0; i < i1; ++i)
        copy16_lds(ra, buf + (wave * CA + i) * 1024,
                   (((wave * CA + i) & 1) ? ok1 : ok0) ? aoff[i] : kFar8, (uint32_t)t * (BT * 2));
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
      const int ch = ((wave * FC + f) * 2 + (g & 1)) ^ turn_v(t);
      vrd[f] = kA + t * TC + 16 * ch + 8 * (l16 & 1);
    }
  }
  const uint32_t srd = kA + kV + wave * BT * 4 + 32 * half;
  // Gradients: row col of a tile, chunk 2 s + half; or four rows t of 16 values in
  // 16 lanes (four lanes a row), twice, each row in other banks.  turn_a moves
  // whole groups of four chunks (two with FR = 2), so tiles four apart differ by a
  // constant.
  constexpr int NRD = TURNED ? (FR < 4 ? FR : 4) : 4;
  uint32_t ard[NRD];
  if constexpr (TURNED) {
    const int t = 8 * (g >> 1) + (l16 >> 2);   // + 16 s + 4 j, the same turn_a for FR >= 4
#pragma unroll
    for (int f = 0; f < NRD; ++f)
      ard[f] = t * TR * 2 + 16 * ((4 * f + 2 * (g & 1) + ((l16 & 3) >> 1)) ^ turn_a(t)) +
               8 * (l16 & 1);
  } else {
#pragma unroll
    for (int s = 0; s < 4; ++s) ard[s] = col * BT * 2 + 16 * ((2 * s + half) ^ turn_a(col));
  }
  auto read_codes = [&](const uint8_t* buf, int s) {
#pragma unroll
    for (int f = 0; f < FC; ++f) oc[f] = read_tr8(buf + vrd[f] + 16 * s * TC);
#pragma unroll
    for (int j = 0; j < 2; ++j) os[j] = *(const f32x4_t*)(buf + srd + 64 * s + 16 * j);
  };
  auto read_dy = [&](const uint8_t* buf, int s, int set) {
#pragma unroll
    for (int f = 0; f < FR; ++f) {
      if constexpr (TURNED) {
        const uint8_t* p = buf + ard[f % NRD] + 16 * s * TR * 2 + f / NRD * 256;
        const u32x2_t lo = read_tr16(p), hi = read_tr16(p + 4 * TR * 2);
        oa[set][f] = u32x4_t{lo[0], lo[1], hi[0], hi[1]};
      } else {
        oa[set][f] = *(const u32x4_t*)(buf + 32 * f * BT * 2 + ard[s]);
      }
    }
  };
  auto convert = [&](int set) {
#pragma unroll
    for (int i = 0; i < FC; ++i)
#pragma unroll
      for (int p = 0; p < 4; ++p)
        ov[set][i][p] =
            pack16x2<F16>(code_value(oc[i][p / 2], 2 * (p & 1), os[p / 2][2 * (p & 1)]),
                          code_value(oc[i][p / 2], 2 * (p & 1) + 1, os[p / 2][2 * (p & 1) + 1]));
  };
  f32x16_t acc[FC][FR];
#pragma unroll
  for (int i = 0; i < FC; ++i)
#pragma unroll
    for (int j = 0; j < FR; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
  auto products = [&](int set) {
#pragma unroll
    for (int j = 0; j < FR; ++j)
#pragma unroll
      for (int i = 0; i < FC; ++i)
        acc[i][j] = mfma_32x32x16<F16>(ov[set][i], oa[set][j], acc[i][j]);
  };
  // One substep's products with the reads and the conversion of the next one laid
  // between them, and `nc` copies.
  auto interleave = [&](int nc) {
    constexpr int N = FC * FR;
    __builtin_amdgcn_sched_group_barrier(kSgDsRead, FC + 2, 0);
#pragma unroll
    for (int q = 0; q < N; ++q) {
      __builtin_amdgcn_sched_group_barrier(kSgMfma, 1, 0);
      if (q < N / 2) {
        __builtin_amdgcn_sched_group_barrier(kSgDsRead, (TURNED ? 4 : 2) / FC, 0);
        __builtin_amdgcn_sched_group_barrier(kSgValu, 2, 0);
      } else {
        __builtin_amdgcn_sched_group_barrier(kSgValu, 44 / FR, 0);
      }
      if (q * nc / N != (q + 1) * nc / N) {
        __builtin_amdgcn_sched_group_barrier(kSgSalu, 2, 0);
        __builtin_amdgcn_sched_group_barrier(kSgVmem, 1, 0);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  // all but the last `out` of this wave's copies have landed, and every wave is here
  auto land = [&](auto out) {
    constexpr int n = decltype(out)::value;
    __builtin_amdgcn_s_waitcnt(0x0F70 | (n & 15) | (n >> 4) << 14);   // vmcnt(n)
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  };
  using All = std::integral_constant<int, 0>;
  using Ahead = std::integral_constant<int, (ND - 2) * (CA + CV + 1)>;   // of later steps

  auto copy_step = [&](uint8_t* buf, int t) {
    copy_codes(buf, t);
    copy_dy(buf, t, 0, CA);
  };
  copy_step(buf0, t0);
  if constexpr (ND > 2) {
    copy_step(buf1, t0 + 1);
    copy_step(buf2, t0 + 2);
  }
  copy_codes(ND > 2 ? buf3 : buf1, t0 + ND - 1);
  land(std::integral_constant<int, Ahead::value + CV + 1>{});
  read_codes(buf0, 0);
  read_dy(buf0, 0, 0);
  convert(0);
  auto step = [&](int t, uint8_t* last, uint8_t* cur, uint8_t* next) {
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int set = s & 1;
      if (s == 3) {
        land(Ahead{});
        copy_codes(cur, t + ND);
      }
      if (s == 0) copy_dy(last, t + ND - 1, 0, (CA + 1) / 2);
      if (s == 1) copy_dy(last, t + ND - 1, (CA + 1) / 2, CA);
      const uint8_t* from = s == 3 ? next : cur;
      read_codes(from, (s + 1) & 3);
      read_dy(from, (s + 1) & 3, set ^ 1);
      products(set);
      convert(set ^ 1);
      interleave(s == 3 ? CV + 1 : s == 0 ? (CA + 1) / 2 : s == 1 ? CA / 2 : 0);
    }
  };
  int t = t0;
  if constexpr (ND == 2) {
    for (; t + 1 < t1; t += 2) {
      step(t, buf1, buf0, buf1);
      step(t + 1, buf0, buf1, buf0);
    }
    if (t < t1) step(t, buf1, buf0, buf1);
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

  // ---- results: value 4 q + e of a tile is row col, column 8 q + 4 half + e ----
  // Through LDS, 32 rows at a time in a wave's own part of a buffer (16-byte chunks
  // permuted by the row), so that a row is written by neighbouring lanes.
  void* const out = SPLIT ? (void*)(a.part + (int64_t)blockIdx.y * a.R * a.ldp) : a.out;
  constexpr int KIND = SPLIT ? (int)kOutF32 : OUT;
  constexpr int OCH = 8 * FC, OR = 64 / OCH;   // chunks a row, rows an instruction
  static_assert(4 * 32 * OCH * 16 <= kBuf, "results fit a buffer");
  const int64_t ldo = SPLIT ? a.ldp : a.ldo;
  const int cend = SPLIT ? (int)a.ldp : a.C;
  const bool vec = SPLIT || whole4<KIND>(out, ldo);
  auto turn_o = [](int row) { return FC == 2 ? row & 15 : (row >> 1) & 7; };
  land(All{});   // every wave has read its operands, and no copy is in flight
  uint8_t* const mine = buf0 + wave * 32 * OCH * 16;
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
      const int r = r0 + 32 * j + row, c = c0 + 32 * FC * wave + 4 * ch;
      if (r < a.R && c < cend) store4<KIND>(out, (int64_t)r * ldo + c, v, cend - c, vec);
    }
  }
}

// The splits of t added in order and rounded: a thread takes four columns.
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
    f32x4_t s = *(const f32x4_t*)p;
    for (int k = 1; k < a.splits; ++k) s += *(const f32x4_t*)(p + (int64_t)k * a.R * a.ldp);
    store4<OUT>(a.out, r * a.ldo + c, s, a.C - c, vec);
  }
}

struct Form {
  int fr, fc;
  int splits, steps_per;
};
Form form_of(int R, int C, int T) {
  const int cus = int8_cus();
  auto tiles = [&](int fr, int fc) {
    return (int64_t)((R + 32 * fr - 1) / (32 * fr)) * ((C + 128 * fc - 1) / (128 * fc));
  };
  Form f{2, 1, 1, 1};
  if (tiles(8, 2) >= cus * 3 / 4) f = Form{8, 2, 1, 1};
  const int steps = (T + BT - 1) / BT;
  if (f.fr == 2) {
    const int64_t most = 2 * cus / tiles(2, 1);
    f.splits = (int)(most < steps / 4 ? most : steps / 4);
    f.splits = f.splits < 1 ? 1 : f.splits;
  }
  f.steps_per = (steps + f.splits - 1) / f.splits;
  if (f.steps_per < 1) f.steps_per = 1;
  f.splits = steps > 0 ? (steps + f.steps_per - 1) / f.steps_per : 1;
  return f;
}

template <bool TURNED, bool F16, int OUT, bool SPLIT>
hipError_t launch(const GradArgs& a, const Form& f, hipStream_t s) {
  const dim3 grid((a.tiles_r * a.tiles_c + kXcds - 1) / kXcds * kXcds, a.splits);
  if (f.fr == 8)
    int8_grad_kernel<8, 2, 2, TURNED, F16, OUT, SPLIT><<<grid, kThreads, 0, s>>>(a);
  else
    int8_grad_kernel<2, 1, 4, TURNED, F16, OUT, SPLIT><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}

template <bool TURNED, bool F16, int OUT>
hipError_t launch(const GradArgs& a, const Form& f, hipStream_t s) {
  if (f.splits == 1) return launch<TURNED, F16, OUT, false>(a, f, s);
  const hipError_t e = launch<TURNED, F16, kOutF32, true>(a, f, s);
  if (e != hipSuccess) return e;
  const int64_t groups = ((int64_t)a.R * ((a.C + 3) / 4) + kThreads - 1) / kThreads;
  int8_grad_reduce_kernel<OUT>
      <<<(int)(groups < 65536 ? groups : 65536), kThreads, 0, s>>>(a);
  return hipGetLastError();
}

template <bool TURNED>
hipError_t launch(const GradArgs& a, const Form& f, bool f16, int out, hipStream_t s) {
  if (out == kOutF32)
    return f16 ? launch<TURNED, true, kOutF32>(a, f, s) : launch<TURNED, false, kOutF32>(a, f, s);
  return f16 ? launch<TURNED, true, kOutF16>(a, f, s) : launch<TURNED, false, kOutBf16>(a, f, s);
}

}  // namespace

size_t int8_grad_workspace(int R, int C, int T) {
  const Form f = form_of(R, C, T);
  return f.splits > 1 ? (size_t)f.splits * R * ((C + 3) / 4 * 4) * sizeof(float) : 0;
}

hipError_t launch_int8_grad(const GradGemm& g, bool turned, bool f16, void* workspace,
                            hipStream_t s) {
  const Form f = form_of(g.R, g.v.cols, g.v.rows);
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
  const int64_t tr = ((int64_t)a.R + 32 * f.fr - 1) / (32 * f.fr),
                tc = ((int64_t)a.C + 128 * f.fc - 1) / (128 * f.fc);
  // a launch counts its threads in 32 bits
  if (tr * tc * f.splits >= ((int64_t)1 << 32) / kThreads - kXcds) return hipErrorNotSupported;
  a.tiles_r = (int)tr;
  a.tiles_c = (int)tc;
  a.splits = f.splits;
  a.steps_per = f.steps_per;
  a.part = (float*)workspace;
  a.ldp = (a.C + 3) / 4 * 4;
  return turned ? launch<true>(a, f, f16, g.out_type, s) : launch<false>(a, f, f16, g.out_type, s);
}

}  // namespace bnbx
