// Register byte tables of a row block's 16 dequantized values, and the
// decode of packed 4-bit codes through them (v_perm_b32 only).
#pragma once

#include "bnbx_device.hpp"
#include "bnbx_internal.hpp"

namespace bnbx {

// The 16 values bf16(L[i] * scale) of one row block, split into a table of
// their high bytes (h[j] holds entries 4j..4j+3) and one of their low bytes.
struct Tab16 {
  uint32_t h[4], l[4];
};

// Levels that are exactly -1, +0, -0 or +1 need no multiply: their products
// are -sc, a zero with sc's sign, one with the opposite sign, and sc.  NF4:
// L[0] = -1, L[7] = 0, L[15] = +1.  FP4 (E2M1 / 6, by code): L[0] = +0,
// L[7] = +1, L[8] = -0, L[15] = -1.
template <bool FP4, bool F16>
__device__ __forceinline__ Tab16 make_tab16(const LevelTable& lv, float sc) {
  const uint32_t sb = __builtin_bit_cast(uint32_t, sc);
  const float neg = __builtin_bit_cast(float, sb ^ 0x80000000u);
  const float zero = __builtin_bit_cast(float, sb & 0x80000000u);
  const float nzero = __builtin_bit_cast(float, (sb ^ 0x80000000u) & 0x80000000u);
  uint32_t pk[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    float a, b;
    if (FP4) {
      a = k == 0 ? zero : k == 4 ? nzero : lv.level[2 * k] * sc;
      b = k == 3 ? sc : k == 7 ? neg : lv.level[2 * k + 1] * sc;
    } else {
      a = k == 0 ? neg : lv.level[2 * k] * sc;
      b = k == 3 ? zero : k == 7 ? sc : lv.level[2 * k + 1] * sc;
    }
    pk[k] = pack16x2<F16>(a, b);
  }
  Tab16 t;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    t.h[j] = perm(pk[2 * j + 1], pk[2 * j], 0x07050301u);
    t.l[j] = perm(pk[2 * j + 1], pk[2 * j], 0x06040200u);
  }
  return t;
}

// The same for levels known only at run time (every product formed).
template <bool F16>
__device__ __forceinline__ Tab16 make_tab16_any(const LevelTable& lv, float sc) {
  uint32_t pk[8];
#pragma unroll
  for (int k = 0; k < 8; ++k)
    pk[k] = pack16x2<F16>(lv.level[2 * k] * sc, lv.level[2 * k + 1] * sc);
  Tab16 t;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    t.h[j] = perm(pk[2 * j + 1], pk[2 * j], 0x07050301u);
    t.l[j] = perm(pk[2 * j + 1], pk[2 * j], 0x06040200u);
  }
  return t;
}

// 8 weights (one packed dword: byte j = codes of weights 2j (high nibble) and
// 2j+1) -> 4 dwords of bf16 pairs in weight order.  Four 4-bit codes held one
// per byte select their entries with v_perm_b32 from each half of the table
// (entries 0-7 and 8-15); a per-byte mask made from bit 3 of the codes
// (v_perm's sign-replicating selectors 8-11) picks between the halves.  The
// codes are grouped as weights (0, 1, 4, 5) and (2, 3, 6, 7), so each output
// dword is one v_perm of a high-byte and a low-byte pick (26 vector
// instructions per 8 weights; grouping even and odd weights took 28).
__device__ __forceinline__ void decode8(uint32_t d, const Tab16& t, uint32_t* o) {
  auto pick = [&](uint32_t sel, uint32_t m, const uint32_t* tt) {
    const uint32_t a = perm(tt[1], tt[0], sel), b = perm(tt[3], tt[2], sel);
    return (m & b) | (~m & a);
  };
  // selectors in weight order: (0, 1, 4, 5) and (2, 3, 6, 7)
  const uint32_t lo3 = d & 0x07070707u, hi3 = (d >> 4) & 0x07070707u;
  const uint32_t sA = perm(hi3, lo3, 0x02060004u), sB = perm(hi3, lo3, 0x03070105u);
  // bit 3 of each selected code: d bits 7, 3, 23, 19 and 15, 11, 31, 27
  const uint32_t mA = perm(d << 12, d << 8, 0x0B090A08u);
  const uint32_t mB = perm(d << 4, d, 0x0B090A08u);
  const uint32_t hiA = pick(sA, mA, t.h), loA = pick(sA, mA, t.l);
  const uint32_t hiB = pick(sB, mB, t.h), loB = pick(sB, mB, t.l);
  o[0] = perm(hiA, loA, 0x05010400u);
  o[1] = perm(hiB, loB, 0x05010400u);
  o[2] = perm(hiA, loA, 0x07030602u);
  o[3] = perm(hiB, loB, 0x07030602u);
}

}  // namespace bnbx
