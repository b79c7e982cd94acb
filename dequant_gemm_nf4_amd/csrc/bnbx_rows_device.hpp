// Device helpers of the kernels over grouped rows.
#pragma once

#include "bnbx_device.hpp"
#include "bnbx_rows.hpp"

namespace bnbx {

typedef __amdgpu_buffer_rsrc_t rsrc_t;
constexpr uint32_t kFar = 0x80000000u;   // an offset past every buffer resource

__device__ __forceinline__ rsrc_t make_rsrc(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes,
                                           0x00020000);
}

// Double-quant block scale exactly as stored, fl32(fl32(q * fl32(s / 127)) +
// mean), without a branch (one would cut the kernels' scheduling regions in
// two).  fl32(s / 127) is the binary64 product with 1/127 rounded once more:
// s / 127 lies at least 1/254 of a binary32 step from any midpoint of two
// binary32 values (s is a whole number of steps, 127 odd), the product's error
// is below 2^-28 of a step, so the second rounding is that of the quotient, for
// subnormals too.
__device__ __forceinline__ float rows_dq_scale(float q, float s, float mean) {
  const float step = (float)((double)s * (1.0 / 127.0));
  const float prod = q * step;
  return prod + mean;
}

// Range of a resource over `bytes` bytes (at most what 32-bit offsets that
// stay below kFar can reach).
__device__ __forceinline__ uint32_t rsrc_bytes(int64_t bytes) {
  return bytes <= 0 ? 0u : bytes < (int64_t)kFar ? (uint32_t)bytes : kFar;
}

// Inclusive prefix sum over the wave, on the DPP paths (no LDS round trips):
// within rows of 16 lanes, then lane 15 of each row into the next one, then
// lane 31 into the upper half.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);   // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);   // row_shr:2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);   // row_shr:4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);   // row_shr:8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);   // row_bcast:15
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);   // row_bcast:31
  return v;
}

// A row tile: places [r0, r1) of group g.
struct RowTile {
  int g, r0, r1;
};

// Row tiles of TM places, group by group (a tile never spans groups).  Every
// wave finds its workgroup's tile by itself from the bounds on the device:
// lane l takes group 64 c + l, a prefix over the lanes numbers the tiles.
// Bounds are clamped to the plan's rows.
template <int TM>
struct RowTiles {
  const int32_t* offsets;
  int groups, rows;

  __device__ __forceinline__ void bounds(int g, int& a, int& b) const {
    a = b = 0;
    if (g < groups) {
      a = offsets[g];
      b = offsets[g + 1];
      a = a < 0 ? 0 : a > rows ? rows : a;
      b = b < a ? a : b > rows ? rows : b;
    }
  }
  // The tiles of all groups; keeps the first 64 groups' part for find().
  int a0, b0, incl0;
  __device__ __forceinline__ int count() {
    if (offsets == nullptr) return (rows + TM - 1) / TM;
    bounds((int)(threadIdx.x & 63), a0, b0);
    incl0 = wave_scan((b0 - a0 + TM - 1) / TM);
    int n = __builtin_amdgcn_readlane(incl0, 63);
    for (int c = 64; c < groups; c += 64) {
      int a, b;
      bounds(c + (int)(threadIdx.x & 63), a, b);
      n += __builtin_amdgcn_readlane(wave_scan((b - a + TM - 1) / TM), 63);
    }
    return n;
  }
  // Tile t < count(), after count().
  __device__ __forceinline__ RowTile find(int t) const {
    RowTile r{0, 0, 0};
    if (offsets == nullptr) {
      r.r0 = t * TM;
      r.r1 = r.r0 + TM < rows ? r.r0 + TM : rows;
      return r;
    }
    int base = 0, a = a0, b = b0, incl = incl0;
    for (int c = 0;;) {
      const uint64_t past = __ballot(incl > t);
      if (past != 0) {
        const int l = __builtin_ctzll(past);
        const int n = (b - a + TM - 1) / TM;
        const int first = __builtin_amdgcn_readlane(incl - n, l);
        const int ga = __builtin_amdgcn_readlane(a, l), gb = __builtin_amdgcn_readlane(b, l);
        r.g = c + l;
        r.r0 = ga + (t - first) * TM;
        r.r1 = r.r0 + TM < gb ? r.r0 + TM : gb;
        return r;
      }
      base = __builtin_amdgcn_readlane(incl, 63);
      c += 64;
      if (c >= groups) return r;
      bounds(c + (int)(threadIdx.x & 63), a, b);
      incl = base + wave_scan((b - a + TM - 1) / TM);
    }
  }
};

// This workgroup's number among `total` items (no more than the grid has
// workgroups), XCD-aware: workgroup b runs on
// XCD b % 8, and consecutive items go to one XCD (they share weights or rows
// in its L2).  -1: nothing to do.
__device__ __forceinline__ int xcd_item(int total) {
  const int per = (total + kXcds - 1) / kXcds;
  const int slot = (int)(blockIdx.x / kXcds), xcd = (int)(blockIdx.x % kXcds);
  const int id = xcd * per + slot;
  return slot < per && id < total ? id : -1;
}

// Rows of X and Y of a place (-1: outside, the place is left out).
__device__ __forceinline__ int x_row_of(const RowsGemm& a, int place) {
  int row = place;
  if (a.gather > 0) {
    row = a.order[place];
    if (a.gather > 1 && row >= 0) row = (int)((uint32_t)row / (uint32_t)a.gather);
  }
  return row >= 0 && row < a.x_rows ? row : -1;
}
__device__ __forceinline__ int y_row_of(const RowsGemm& a, int place) {
  const int row = a.scatter ? a.order[place] : place;
  return row >= 0 && row < a.y_rows ? row : -1;
}

// In place of a RowsGemm in kernels that serve both kinds of rows: X's rows are
// the places, m of them.
struct NoRows {};
__device__ __forceinline__ int gather_of(const RowsGemm& a) { return a.gather; }
__device__ __forceinline__ int gather_of(const NoRows&) { return 0; }
__device__ __forceinline__ int x_rows_of(const RowsGemm& a, int) { return a.x_rows; }
__device__ __forceinline__ int x_rows_of(const NoRows&, int m) { return m; }

// The byte -> fp32 level pair table in LDS (64 KB at LDS offset 0): entry e,
// (level of the high nibble, level of the low one), in 32 copies side by side,
// 256 bytes an entry, so that one v_perm forms a read's address and b64 reads
// never conflict.
constexpr int kLutBytes = 256 * 256;
__device__ __forceinline__ void lut_build(unsigned char* lds, const LevelTable& lv, int threads) {
  const int lvl = level_lanes(lv);
  for (int e = threadIdx.x; e < kLutBytes / 16; e += threads) {
    const uint32_t b = (uint32_t)e / 16u;
    const float hi = level_lookup(lvl, b >> 4), lo = level_lookup(lvl, b & 15u);
    *(float4*)(lds + 16 * e) = make_float4(hi, lo, hi, lo);
  }
}
// The pair of byte `e` of d; lcol = 8 (lane % 32).
__device__ __forceinline__ float2 lut_pair(const unsigned char* lds, uint32_t d, uint32_t lcol,
                                           int e) {
  return *(const float2*)(lds + perm(d, lcol, 0x0c0c0000u | ((4u + e) << 8)));
}

// Eight binary16 values as two bf16 operands, hi + lo, exactly: binary16 has
// 11 significant bits, bf16 8, and the rest fits lo (bf16 reaches far below
// binary16's subnormals).  An infinity or NaN leaves NaN in lo, which the
// caller replaces.
__device__ __forceinline__ void split_f16(u32x4_t v, u32x4_t& hi, u32x4_t& lo) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const f16x2_t p = __builtin_bit_cast(f16x2_t, (uint32_t)v[k]);
    const float a = (float)p[0], b = (float)p[1];
    const uint32_t h = pack_bf16x2(a, b);
    hi[k] = h;
    const float ra = a - bf16lo_to_f32(h), rb = b - bf16hi_to_f32(h);
    lo[k] = pack_bf16x2(ra, rb);
  }
}

// The top bits of the halves of a bf16 pair that are infinite or NaN (there,
// and only there, one more in the exponent carries into the sign's place).
__device__ __forceinline__ uint32_t odd_halves(uint32_t v) {
  return ((v & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}
// The pair with +-2^-126, by their sign, in the halves of `odd` (of
// odd_halves).  As a partner of an infinity it leaves the infinity its sign.
__device__ __forceinline__ uint32_t tame_halves(uint32_t v, uint32_t odd) {
  const uint32_t m = (odd << 1) - (odd >> 15);   // all bits of those halves
  return (v & ~m) | (((v & 0x80008000u) | 0x00800080u) & m);
}

}  // namespace bnbx
