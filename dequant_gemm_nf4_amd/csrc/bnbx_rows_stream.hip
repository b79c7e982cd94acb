// 4-bit products over grouped rows, few rows a group, for gfx950:
//   Y_i = X_i . W_hat_g^T (+ XA_i . B_a^T),  i a place of group g,
// W_hat_g[n][k] = rnd16(L[code] * scale), the dequantized weight exactly as
// stored (the products run on the same 16-bit values bnbx_dequantize_nf4
// gives), fp32 accumulation, one rounding of Y.
//
// Bound: a wave's table reads, vector work and matrix instructions wait on each
// other (with 16 waves on a CU, over the time it has a workgroup: vector units 61
// % busy, LDS 66 %); then the start and end of a workgroup (6 - 7 us of a round).
// The packed weights stream once per row tile (RB x 16 places).  Measured: 32
// rows in 8 groups of 14336 x 4096 (241 MB) 70 us a call, 3.4 TB/s; 16 rows of
// one 11008 x 4096 weight 16 us; 566 rows in 16 groups of 4096 x 11008 225 us.
//
// A wave takes units of 16 weight rows x 256 k (2 KB packed).  Loads are
// quad-coalesced (lane x: 16 bytes of row x / 4, twice); a 2 KB LDS stage per
// wave turns them so that lane (q, r) (q = lane / 16, r = lane % 16) holds the
// 32 bytes of block q of row r: one block scale and one 16-entry table per
// lane and unit.  Dword m of them is the A operand of MFMA m (16x16x32: A row
// r, eight k); which eight k feed which MFMA is free as long as X agrees: lane
// q of X takes k = 64 q + 8 m.  So D has the weight rows down the values
// (n = 4 q + v) and the places across the lanes (i = lane % 16).
//
// Dequant.  Up to 32 places a tile (LUT): a byte -> fp32 level pair table in
// LDS, 32 copies side by side so that its b64 reads never conflict (with 16
// copies half of all LDS cycles were conflicts), 256 bytes an entry so that
// one v_perm forms an address; two products and one conversion a byte, 2.3
// vector instructions a weight in all.  64 places: the 16 products of a block
// as register byte tables (decode8, 3.7 a weight), because LDS then serves the
// operands of X and its table would leave one workgroup a CU.
//
// X goes through LDS, double-buffered, in slices of 256 k: 32 chunks of 16
// bytes a row, chunk c of row r in slot c ^ (r % 16), so that 16 lanes reading
// one chunk of 16 rows hit 64 banks.
//
// WN waves of a workgroup take different weight rows (and share X), WK waves
// split K slice by slice; their sums meet in LDS in wave order.  WK > 1 is for
// launches whose weight rows alone give the GPU too few waves.  With WN = 1 no
// wave shares X and each loads its operands straight from memory, only the
// lanes whose place exists (one token: 4 of 64).  16 waves over 16 places copy
// X for two steps at once: no row twice, and half the barriers (one round of
// 4096 deep workgroups 36.0 -> 32.8 us).
#include <algorithm>
#include <type_traits>

#include "bnbx_rows_device.hpp"
#include "bnbx_tab16.hpp"

namespace bnbx {
namespace {

constexpr int kSlice = 256;          // k per unit

template <int RB, int WN, int WK, bool LUT, int DQ, bool Q4, bool F16>
__global__ __launch_bounds__(WN* WK * 64) void rows_stream_kernel(RowsGemm a, int tiles_n,
                                                                  LevelTable lv) {
  constexpr int TM = 16 * RB, TN = 16 * WN, kThreads = WN * WK * 64;
  constexpr int kAhead = 2;   // units loaded ahead, per 16 weight rows
  constexpr bool DIRECT = WN == 1, DYN = DQ == kDqDynamic;
  constexpr int XS = WN > RB * 8 ? 2 : 1;                // steps per X buffer
  constexpr int kXPart = TM * kSlice;                    // 16-bit elements of one slice
  constexpr int kXBuf = DIRECT ? 0 : XS * WK * kXPart;
  constexpr int kXLoads = DIRECT ? 1 : XS * RB * 8 / WN;   // 1 KB loads a wave and buffer
  constexpr int kStages = WN * WK * 2048;
  constexpr int kRedBytes = (WK - 1) * WN * RB * 1024;
  // LDS: the byte table (at offset 0: its addresses are v_perm results), X,
  // the waves' stages, the dynamic map if there is room (else it is read from
  // memory); the partial sums reuse all of it.
  constexpr int kLut = LUT ? kLutBytes : 0;
  constexpr int kBufs = kLut + 2 * kXBuf * 2 + kStages;
  constexpr bool kMapLds = DYN && kBufs + 1024 <= 160 * 1024;
  constexpr int kUsed = kBufs + (kMapLds ? 1024 : 0);
  constexpr int kLds = kUsed > kRedBytes ? kUsed : kRedBytes;
  static_assert(DIRECT || XS * RB * 8 % WN == 0, "X loads split evenly");
  __shared__ __attribute__((aligned(256))) unsigned char smem[kLds];

  const float* const dmap = kMapLds ? (const float*)(smem + kBufs) : kDynMapDev.v;
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wn = wave % WN, wk = wave / WN;
  const int r = lane & 15, q = lane >> 4;      // MFMA layout
  const int lr = lane >> 2, lp = lane & 3;     // load layout: row, piece

  RowTiles<TM> tiles{a.offsets, a.groups, a.rows};
  const int nt = tiles.count();
  const int id = xcd_item(nt * tiles_n);   // fits: the grid covers it
  if (id < 0) return;
  // row tiles of one group and the same weight rows are neighbours: they
  // meet in one L2
  const int tn = __builtin_amdgcn_readfirstlane((int)((uint32_t)id / (uint32_t)nt));
  const RowTile tile = tiles.find(id - tn * nt);
  const int n0 = tn * TN + wn * 16;

  const float mu = DQ ? *a.mean : 0.0f;
  const uint32_t rowK2 = (uint32_t)a.K >> 1, nkb = (uint32_t)a.K >> 6;
  const int nslices = (a.K + kSlice - 1) / kSlice;
  const int nsteps = (nslices + WK - 1) / WK;

  // Resources of this group's weight: 64-bit bases, 32-bit offsets inside.
  const uint32_t nblocks = (uint32_t)a.N * nkb;
  const int64_t blk0 = (int64_t)tile.g * nblocks;
  const rsrc_t rw = make_rsrc(a.packed + (int64_t)tile.g * a.N * rowK2, (uint32_t)a.N * rowK2);
  const rsrc_t rq = make_rsrc((const char*)a.absmax + blk0 * (DQ ? 1 : 4),
                              DQ ? nblocks : nblocks * 4u);
  const uint32_t grem = (uint32_t)(blk0 & 255);   // the group's first block in its scale group
  const rsrc_t rg = make_rsrc(DQ ? a.absmax2 + (blk0 >> 8) : nullptr,
                              DQ ? (grem + nblocks + 255u) / 256u * 4u : 0u);

  // Slice of step s (none past the last step).
  auto slice_of = [&](int s) { return s < nsteps ? s * WK + wk : nslices; };

  struct Unit {
    u32x4_t w[2];
    uint32_t q;    // code byte, or the fp32 block maximum (not Q4)
    float s;       // group scale
  };
  const int nl = n0 + lr, nm = n0 + r;
  const uint32_t wrow = nl < a.N ? (uint32_t)nl * rowK2 + 16u * (uint32_t)lp : kFar;
  const uint32_t brow = nm < a.N ? (uint32_t)nm * nkb : kFar;   // row r's first block
  // Byte offset of a block's group scale.
  auto gidx = [&](uint32_t blk) { return ((grem + blk) >> 8) * 4u; };
  auto load_unit = [&](Unit& u, int slice) {
    const bool in = slice < nslices;
    const uint32_t wo = in ? wrow + (uint32_t)slice * (kSlice / 2) : kFar;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      u.w[h] = __builtin_amdgcn_raw_buffer_load_b128(rw, wo + 64u * h, 0, 2);
    if constexpr (!Q4) {
      // the lane's block; past the end of the row it has no scale and no value
      const uint32_t at = 4u * (uint32_t)slice + (uint32_t)q;
      const bool bin = in && brow != kFar && at < nkb;
      const uint32_t blk = brow + at;
      if (DQ) {
        u.q = __builtin_amdgcn_raw_buffer_load_b8(rq, bin ? blk : kFar, 0, 0);
        u.s = __builtin_bit_cast(
            float, __builtin_amdgcn_raw_buffer_load_b32(rg, bin ? gidx(blk) : kFar, 0, 0));
      } else {
        u.q = __builtin_amdgcn_raw_buffer_load_b32(rq, bin ? blk * 4u : kFar, 0, 0);
        u.s = 0.0f;
      }
    }
  };
  // Block scale from its code (or fp32 bits) and group scale.
  auto scale_of = [&](uint32_t code, float gs) {
    if (DYN) {
      const float prod = dmap[code & 0xffu] * gs;
      return prod + mu;
    }
    if (DQ) return rows_dq_scale((float)(int8_t)(uint8_t)code, gs, mu);
    return __builtin_bit_cast(float, code);
  };
  // Q4 (rows of a multiple of 4 blocks, codes 4-byte aligned, fp32 maxima 16):
  // the codes of four steps in one load.  A lane loads the four codes of row r
  // in the slice of step 4 t + q, all its bytes of that line at once (each such
  // request costs the address path a cycle, whatever its size); step 4 t + p
  // fetches lane (p, r)'s and takes block q's.
  struct Quad {
    u32x4_t q;     // code bytes (x), or four fp32 block maxima
    float s;       // their group scale
  };
  auto load_quad = [&](Quad& u, int s) {
    if constexpr (Q4) {
      const int slice = slice_of(s + q);
      const bool bin = brow != kFar && slice < nslices;
      const uint32_t blk = brow + 4u * (uint32_t)slice;
      if (DQ) {
        u.q[0] = __builtin_amdgcn_raw_buffer_load_b32(rq, bin ? blk : kFar, 0, 0);
        u.s = __builtin_bit_cast(
            float, __builtin_amdgcn_raw_buffer_load_b32(rg, bin ? gidx(blk) : kFar, 0, 0));
      } else {
        u.q = __builtin_amdgcn_raw_buffer_load_b128(rq, bin ? blk * 4u : kFar, 0, 0);
      }
    }
  };
  // Scale of the lane's block in step s (ph = s % 4).
  auto unit_scale = [&](const Unit& u, const Quad& c, int s, int ph) {
    const bool bin = brow != kFar && 4u * (uint32_t)slice_of(s) + (uint32_t)q < nkb;
    float sc;
    if constexpr (Q4) {
      const int from = (16 * ph + r) << 2;
      if (DQ) {
        const uint32_t codes = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)c.q[0]);
        const float gs = __int_as_float(__builtin_amdgcn_ds_bpermute(from, __float_as_int(c.s)));
        sc = scale_of(codes >> (8 * q), gs);
      } else {
        uint32_t v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = (uint32_t)__builtin_amdgcn_ds_bpermute(from, (int)c.q[e]);
        sc = __builtin_bit_cast(float, q < 2 ? (q == 0 ? v[0] : v[1]) : (q == 2 ? v[2] : v[3]));
      }
    } else {
      sc = scale_of(u.q, u.s);
    }
    return bin ? sc : 0.0f;
  };

  // Units of the first steps go out before the rows of X are looked up.
  Unit un[kAhead];
#pragma unroll
  for (int p = 0; p < kAhead; ++p)
    load_unit(un[p], slice_of(p));
  Quad quad, quad_next;   // of steps 4 t .. 4 t + 3, and of the next four
  load_quad(quad_next, 0);

  if (LUT) lut_build(smem, lv, kThreads);
  if (kMapLds)
    for (int e = t; e < 256; e += kThreads) ((float*)(smem + kBufs))[e] = kDynMapDev.v[e];

  unsigned char* const stage = smem + kLut + 2 * kXBuf * 2 + wave * 2048;
  auto barrier = [] { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); };

  // X through LDS: the WN waves of one K part copy its slices of XS steps, 2
  // rows an instruction (lane l: row l / 32, slot l % 32).  Rows past the tile
  // repeat its first row (their results are never stored); chunks past K are
  // zeros.
  uint16_t* const xs = (uint16_t*)(smem + kLut);
  const uint16_t* xp[kXLoads];
  int xk[kXLoads];
  uint32_t xslot[kXLoads];
  u32x4_t xv[kXLoads];
  auto x_sub = [&](int i) { return XS == 1 ? 0 : (WN * i + wn) / (RB * 8); };   // step
  if (!DIRECT) {
#pragma unroll
    for (int i = 0; i < kXLoads; ++i) {
      const int row = 2 * ((XS == 1 ? wn * kXLoads + i : WN * i + wn) % (RB * 8)) + (lane >> 5);
      const int place = tile.r0 + row < tile.r1 ? tile.r0 + row : tile.r0;
      int xr = x_row_of(a, place);
      xr = xr < 0 ? 0 : xr;
      xp[i] = a.x + (int64_t)xr * a.ldx;
      xk[i] = 8 * ((lane & 31) ^ (row & 15));
      xslot[i] = (uint32_t)((x_sub(i) * WK + wk) * kXPart + row * kSlice + 8 * (lane & 31));
    }
  }
  auto load_x = [&](int s) {   // of steps s .. s + XS - 1
    if (DIRECT) return;
#pragma unroll
    for (int i = 0; i < kXLoads; ++i) {
      const int k = slice_of(s + x_sub(i)) * kSlice + xk[i];
      xv[i] = *(const u32x4_t*)(xp[i] + (k < a.K ? k : 0));
    }
  };
  auto put_x = [&](int buf, int s) {
    if (DIRECT) return;
#pragma unroll
    for (int i = 0; i < kXLoads; ++i) {
      const int slice = slice_of(s + x_sub(i));
      const bool tail = (slice + 1) * kSlice > a.K;   // uniform
      if (tail && slice * kSlice + xk[i] >= a.K) xv[i] = u32x4_t{0u, 0u, 0u, 0u};
      *(u32x4_t*)(xs + buf * kXBuf + xslot[i]) = xv[i];
    }
  };
  // X straight into operands (DIRECT): lane (q, r) reads its chunks of place
  // r's row, if there is one; zeros past K and for places past the tile.
  const uint16_t* dp[DIRECT ? RB : 1];
  u32x4_t dx[DIRECT ? RB : 1][8];
  if (DIRECT) {
#pragma unroll
    for (int i = 0; i < RB; ++i) {
      const int place = tile.r0 + 16 * i + r;
      const int xr = place < tile.r1 ? x_row_of(a, place) : -1;
      dp[i] = xr >= 0 ? a.x + (int64_t)xr * a.ldx + 64 * q : nullptr;
    }
  }
  auto load_direct = [&](int slice) {
    if (!DIRECT) return;
    const bool kin = 4u * (uint32_t)slice + (uint32_t)q < nkb;
#pragma unroll
    for (int i = 0; i < RB; ++i)
#pragma unroll
      for (int m = 0; m < 8; ++m) {
        dx[i][m] = u32x4_t{0u, 0u, 0u, 0u};
        if (dp[i] != nullptr && kin) dx[i][m] = *(const u32x4_t*)(dp[i] + slice * kSlice + 8 * m);
      }
  };

  // Stage slots: piece p (16 bytes) of row w at slot 8 w + (p ^ f(w)), free of
  // bank conflicts both ways.
  auto fold = [](int w) { return ((w >> 1) & 1) * 4 + ((w >> 2) & 3); };
  const uint32_t ws0 = 16u * (uint32_t)(8 * lr + (lp ^ fold(lr)));
  const uint32_t rs0 = 16u * (uint32_t)(8 * r + ((2 * q) ^ fold(r)));

  // Rows of Y of the lane's places, looked up while the first loads are in
  // flight (-1: not written).
  int yrow[RB];
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    const int place = tile.r0 + 16 * i + r;
    yrow[i] = place < tile.r1 && x_row_of(a, place) >= 0 ? y_row_of(a, place) : -1;
  }

  f32x4_t acc[RB];
#pragma unroll
  for (int i = 0; i < RB; ++i) acc[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  const uint32_t lcol = 8u * (uint32_t)(lane & 31);
  // A unit in the MFMA layout: block q of row r, with its scale (or, for 64
  // places, its table).
  struct Op {
    u32x4_t w[2];
    float sc;
  };
  auto turn = [&](Op& o, Unit& u, int s, int ph) {   // ph = s % 4
    if (Q4 && ph == 0) {
      quad = quad_next;
      load_quad(quad_next, s + 4);
    }
    o.sc = unit_scale(u, quad, s, ph);
    *(u32x4_t*)(stage + ws0) = u.w[0];
    *(u32x4_t*)(stage + (ws0 ^ 64u)) = u.w[1];
    o.w[0] = *(const u32x4_t*)(stage + rs0);
    o.w[1] = *(const u32x4_t*)(stage + (rs0 ^ 16u));
    load_unit(u, slice_of(s + kAhead));
  };
  Op op;
  // Step s: `u` holds step s + 1's unit, turned while step s multiplies.
  // (With register tables, step s's own: the turned ones would cost registers
  // that the accumulators need.)
  auto step = [&](Unit& u, int s, auto phase) {
    constexpr int PH = decltype(phase)::value;
    if constexpr (!LUT) turn(op, u, s, PH);
    Tab16 tab;
    if constexpr (!LUT) tab = make_tab16_any<F16>(lv, op.sc);
    const float sc = op.sc;
    const u32x4_t w[2] = {op.w[0], op.w[1]};
    const uint16_t* xb = xs + (PH / XS & 1) * kXBuf + ((PH % XS) * WK + wk) * kXPart;
    if constexpr (LUT) {
      // Table reads (and X) of MFMA m + 1 go out before the products of m.
      float2 l2[2][4];
      u32x4_t xo[2][RB];
      auto look = [&](int m) {
        const uint32_t d = w[m >> 2][m & 3];
#pragma unroll
        for (int e = 0; e < 4; ++e) l2[m & 1][e] = lut_pair(smem, d, lcol, e);
        if (!DIRECT)
#pragma unroll
          for (int i = 0; i < RB; ++i)
            xo[m & 1][i] =
                *(const u32x4_t*)(xb + (16 * i + r) * kSlice + 8 * ((8 * q + m) ^ r));
      };
      look(0);
      turn(op, u, s + 1, (PH + 1) & 3);
#pragma unroll
      for (int m = 0; m < 8; ++m) {
        if (m < 7) look(m + 1);
        __builtin_amdgcn_sched_barrier(0);
        u32x4_t wo;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          wo[e] = pack16x2<F16>(l2[m & 1][e].x * sc, l2[m & 1][e].y * sc);
#pragma unroll
        for (int i = 0; i < RB; ++i)
          acc[i] = mfma_16x16x32<F16>(wo, DIRECT ? dx[DIRECT ? i : 0][m] : xo[m & 1][i], acc[i]);
        __builtin_amdgcn_sched_barrier(0);
      }
    } else {
      static_assert(LUT || !DIRECT, "operands of X from memory go with the byte table");
#pragma unroll
      for (int m = 0; m < 8; ++m) {
        u32x4_t xo[RB];
#pragma unroll
        for (int i = 0; i < RB; ++i)
          xo[i] = *(const u32x4_t*)(xb + (16 * i + r) * kSlice + 8 * ((8 * q + m) ^ r));
        uint32_t o[4];
        decode8(w[m >> 2][m & 3], tab, o);
        const u32x4_t wo = {o[0], o[1], o[2], o[3]};
#pragma unroll
        for (int i = 0; i < RB; ++i) acc[i] = mfma_16x16x32<F16>(wo, xo[i], acc[i]);
      }
    }
  };

  load_x(0);
  load_direct(slice_of(0));
  put_x(0, 0);
  barrier();
  if (LUT) turn(op, un[0], 0, 0);
  // No branch around a load, only out of the loop: the compiler's waits count
  // the loads issued since, and would wait for all of them where it cannot tell
  // how many.
  auto advance = [&](Unit& u, int s, auto phase) {
    constexpr int PH = decltype(phase)::value;
    if (PH % XS == 0) load_x(s + XS);
    step(u, s, phase);
    load_direct(slice_of(s + 1));
    if (PH % XS == XS - 1) {
      put_x(((PH + 1) / XS) & 1, s + 1);
      if (!DIRECT) barrier();
    }
  };
  for (int s = 0;;) {
    advance(un[LUT ? 1 : 0], s, std::integral_constant<int, 0>{});
    if (++s >= nsteps) break;
    advance(un[LUT ? 0 : 1], s, std::integral_constant<int, 1>{});
    if (++s >= nsteps) break;
    advance(un[LUT ? 1 : 0], s, std::integral_constant<int, 2>{});
    if (++s >= nsteps) break;
    advance(un[LUT ? 0 : 1], s, std::integral_constant<int, 3>{});
    if (++s >= nsteps) break;
  }
  if (DIRECT || XS > 1) barrier();

  // Low-rank term: the adapters whose places meet the tile, each in steps of
  // 32 ranks, shared out over the WK waves.  XA's two planes and, for fp16, B
  // split into two bf16 parts (11 bits: exact) keep the term's error at 2^-16
  // of it; products run in bf16 for the range.  Each adapter's term is summed
  // apart and added to its own places only, so one adapter's infinities never
  // reach another request's row.  An infinite or NaN B meets XA's high part as
  // it is, and the low part, which may be zero or of the other sign, as
  // +-2^-126.
  if (a.lora.offsets != nullptr) {
    const LoraRows& lo = a.lora;
    int seg = 0;
    for (int c = 0; c < lo.adapters; c += 64) {
      int b0 = 0, b1 = 0;
      const int gl = c + lane;
      if (gl < lo.adapters) {
        b0 = lo.offsets[gl];
        b1 = lo.offsets[gl + 1];
      }
      uint64_t hit = __ballot(b0 < b1 && b0 < tile.r1 && b1 > tile.r0);
      while (hit != 0) {
        const int l = __builtin_ctzll(hit);
        hit &= hit - 1;
        const int s0 = __builtin_amdgcn_readlane(b0, l), s1 = __builtin_amdgcn_readlane(b1, l);
        const uint16_t* bb = lo.b + (int64_t)(c + l) * lo.stride_b;
        f32x4_t term[RB];
#pragma unroll
        for (int i = 0; i < RB; ++i) term[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        for (int k = 0; k < lo.r; k += 32, ++seg) {
          if (seg % WK != wk) continue;   // uniform in the wave
          const int k8 = k + 8 * q;
          // XA's loads go out before the first use of B, for two row blocks at
          // most: all four of 64 places at once would cost the registers of the
          // second workgroup of a CU, none 5 % (22 sizes of up to 64 adapters)
          constexpr int kEarly = RB <= 2 ? RB : 2;
          u32x4_t xh[RB], xl[RB];
          auto load_xa = [&](int i) {
            const int place = tile.r0 + 16 * i + r;
            xh[i] = xl[i] = u32x4_t{0u, 0u, 0u, 0u};
            if (k8 < lo.r && place < tile.r1 && place >= s0 && place < s1) {
              const uint16_t* xa = lo.xa + (int64_t)place * 2 * lo.r + k8;
              xh[i] = *(const u32x4_t*)xa;
              xl[i] = *(const u32x4_t*)(xa + lo.r);
            }
          };
          const int n = n0 + r;
          u32x4_t bh = {0u, 0u, 0u, 0u}, bl;
          if (k8 < lo.r && n < a.N) bh = *(const u32x4_t*)(bb + (int64_t)n * lo.ldb + k8);
#pragma unroll
          for (int i = 0; i < kEarly; ++i) load_xa(i);
          if (F16) split_f16(bh, bh, bl);
          u32x4_t bt = bh;   // bh for xl
          uint32_t odd = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) odd |= odd_halves(bh[e]);
          if (__builtin_expect(__ballot(odd != 0) != 0, false)) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              bt[e] = tame_halves(bh[e], odd_halves(bh[e]));
              // (a low part is NaN where the value is not finite)
              if (F16) bl[e] = tame_halves(bl[e], odd_halves(bl[e]));
            }
          }
#pragma unroll
          for (int i = 0; i < RB; ++i) {
            if (i >= kEarly) load_xa(i);
            term[i] = mfma_16x16x32<false>(bh, xh[i], term[i]);
            term[i] = mfma_16x16x32<false>(bt, xl[i], term[i]);
            if (F16) term[i] = mfma_16x16x32<false>(bl, xh[i], term[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < RB; ++i) {
          const int place = tile.r0 + 16 * i + r;
          const bool own = place >= s0 && place < s1;
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[i][v] = own ? acc[i][v] + term[i][v] : acc[i][v];
        }
      }
    }
  }

  // The K parts' sums, in wave order (all of smem is free: every wave has
  // passed the last barrier).
  if (WK > 1) {
    f32x4_t* const red = (f32x4_t*)smem;
    if (wk > 0) {
#pragma unroll
      for (int i = 0; i < RB; ++i)
        red[(((wk - 1) * WN + wn) * RB + i) * 64 + lane] = acc[i];
    }
    __syncthreads();
    if (wk > 0) return;
#pragma unroll
    for (int p = 0; p < WK - 1; ++p)
#pragma unroll
      for (int i = 0; i < RB; ++i) {
        const f32x4_t v = red[((p * WN + wn) * RB + i) * 64 + lane];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][e] += v[e];
        }
  }

  // Lane (q, r): place r of each 16, weight rows 4 q .. 4 q + 3 of each 16.
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    const int row = yrow[i];
    if (row < 0) continue;
    uint16_t* const yr = a.y + (int64_t)row * a.ldy;
    const int n = n0 + 4 * q;
    const uint32_t p0 = pack16x2<F16>(acc[i][0], acc[i][1]);
    const uint32_t p1 = pack16x2<F16>(acc[i][2], acc[i][3]);
    if (n + 3 < a.N && ((uintptr_t)(yr + n) & 7) == 0) {
      *(uint2*)(yr + n) = make_uint2(p0, p1);
    } else {
      if (n < a.N) yr[n] = (uint16_t)p0;
      if (n + 1 < a.N) yr[n + 1] = (uint16_t)(p0 >> 16);
      if (n + 2 < a.N) yr[n + 2] = (uint16_t)p1;
      if (n + 3 < a.N) yr[n + 3] = (uint16_t)(p1 >> 16);
    }
  }
}

template <int RB, int WN, int WK, bool LUT>
hipError_t launch_one(const RowsGemm& a, int quant_type, bool f16, hipStream_t stream,
                      bool launch) {
  constexpr int TM = 16 * RB, TN = 16 * WN;
  const int tiles_n = (a.N - 1) / TN + 1;
  const unsigned grid = rows_grid(a.rows, a.groups, TM, tiles_n, WN * WK * 64);
  if (grid == 0) return hipErrorNotSupported;
  if (!launch) return hipSuccess;
  const LevelTable& lv = level_table(quant_type);
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(WN * WK * 64), 0, stream, a, tiles_n,
                       lv);
  };
  const int nkb = a.K / 64;
  const bool q4 =
      nkb % 4 == 0 && ((uintptr_t)a.absmax & (a.double_quant == kDqNone ? 15 : 3)) == 0;
  auto pick = [&](auto dq, auto quads) {
    constexpr int DQ = decltype(dq)::value;
    constexpr bool Q4 = decltype(quads)::value;
    if (f16) go(rows_stream_kernel<RB, WN, WK, LUT, DQ, Q4, true>);
    else go(rows_stream_kernel<RB, WN, WK, LUT, DQ, Q4, false>);
  };
  auto with = [&](auto dq) {
    if (q4) pick(dq, std::true_type{});
    else pick(dq, std::false_type{});
  };
  if (a.double_quant == kDqNone) with(std::integral_constant<int, kDqNone>{});
  else if (a.double_quant == kDqLinear) with(std::integral_constant<int, kDqLinear>{});
  else with(std::integral_constant<int, kDqDynamic>{});
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rows_stream(const RowsGemm& a, int quant_type, bool f16, int cus,
                              hipStream_t stream, bool launch) {
  const int groups = a.offsets == nullptr ? 1 : (a.groups < a.rows ? a.groups : a.rows);
  const int mean_rows = (a.rows + groups - 1) / groups;
  const int rb = mean_rows <= 16 ? 1 : mean_rows <= 32 ? 2 : 4;
  const int nslices = (a.K + kSlice - 1) / kSlice;
  // Row tiles the launch is likely to have, times 16-row weight slabs.
  const int64_t tm = 16 * rb;
  const int64_t slabs = (int64_t)groups * ((mean_rows + tm - 1) / tm) * ((a.N + 15) / 16);
  // Waves split K where the slabs alone do not fill the GPU: the more of them
  // share a workgroup's rows (WN), the better they use it, the more of them
  // split K (WK), the fewer steps it takes.  Each form's time is its rounds of
  // workgroups (one a CU) times one workgroup's: `ends` for its start and end
  // and `step` a step, in us, fitted to kernel times over N = 512 .. 32768 and
  // K = 1024 .. 14336 (within 10 %).  For instance 16 places, K = 4096, forms
  // (WN, WK) = (2, 4), (4, 4), (8, 2), (16, 1): N = 8192 13.1 / 15.8 / 21.8 /
  // 32.6; N = 16384 23.4 / 17.3 / 22.4 / 33.2; N = 24576 34.0 / 30.1 / 23.4 /
  // 33.8.
  auto cost = [&](int wn, int wk, double ends, double step) {
    const int64_t wgs = (slabs + wn - 1) / wn;
    const int steps = (nslices + wk - 1) / wk;
    return (double)((wgs + cus - 1) / cus) * (ends + step * steps);
  };
  if (rb == 1) {
    // Up to 4 places: operands of X straight from memory, K in eight.  One
    // place, 4096 x 4096: 8.4, against 11.9 with (2, 4); with 16 places 14.5
    // against 12.1.
    if (mean_rows <= 4 && slabs <= 2 * (int64_t)cus)
      return launch_one<1, 1, 8, true>(a, quant_type, f16, stream, launch);
    const double t2 = cost(2, 4, 6.5, 1.4), t4 = cost(4, 4, 6.5, 2.2),
                 t8 = cost(8, 2, 6.5, 1.85), t16 = cost(16, 1, 6.5, 1.65);
    const double least = std::min(std::min(t2, t4), std::min(t8, t16));
    if (t2 <= least) return launch_one<1, 2, 4, true>(a, quant_type, f16, stream, launch);
    if (t4 <= least) return launch_one<1, 4, 4, true>(a, quant_type, f16, stream, launch);
    if (t8 <= least) return launch_one<1, 8, 2, true>(a, quant_type, f16, stream, launch);
    return launch_one<1, 16, 1, true>(a, quant_type, f16, stream, launch);
  }
  if (rb == 2) {
    const double t2 = cost(2, 2, 7.0, 1.15), t4 = cost(4, 2, 6.5, 1.5),
                 t8 = cost(8, 1, 6.5, 1.35), t16 = cost(16, 1, 7.5, 2.15);
    const double least = std::min(std::min(t2, t4), std::min(t8, t16));
    if (t2 <= least) return launch_one<2, 2, 2, true>(a, quant_type, f16, stream, launch);
    if (t4 <= least) return launch_one<2, 4, 2, true>(a, quant_type, f16, stream, launch);
    if (t8 <= least) return launch_one<2, 8, 1, true>(a, quant_type, f16, stream, launch);
    return launch_one<2, 16, 1, true>(a, quant_type, f16, stream, launch);
  }
  // 64 places, K = 4096, forms (2, 2), (4, 2), (8, 1): N = 8192 23.7 / 25.4 /
  // 35.9; N = 16384 45.0 / 27.5 / 37.2; N = 24576 66.8 / 50.0 / 38.7.
  if (slabs <= 2 * (int64_t)cus) return launch_one<4, 2, 2, false>(a, quant_type, f16, stream, launch);
  if (slabs <= 4 * (int64_t)cus) return launch_one<4, 4, 2, false>(a, quant_type, f16, stream, launch);
  return launch_one<4, 8, 1, false>(a, quant_type, f16, stream, launch);
}

int rows_cus() {
  static const int n = [] {
    int dev = 0, v = 0;
    const bool ok = hipGetDevice(&dev) == hipSuccess &&
                    hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) ==
                        hipSuccess;
    return ok && v > 0 ? v : 256;
  }();
  return n;
}

}  // namespace bnbx
