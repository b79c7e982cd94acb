// Device helpers of the 8-bit operators.
#pragma once

#include <type_traits>

#include "bnbx_device.hpp"
#include "bnbx_int8.hpp"

namespace bnbx {

typedef __amdgpu_buffer_rsrc_t rsrc8_t;
typedef __attribute__((ext_vector_type(4))) int i32x4_t;
typedef __attribute__((ext_vector_type(16))) int i32x16_t;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2_t;

constexpr uint32_t kFar8 = 0x80000000u;   // an offset past every buffer resource

// A buffer resource over `bytes` bytes: loads past them give zero.
__device__ __forceinline__ rsrc8_t rsrc8(const void* base, int64_t bytes) {
  const uint32_t n = bytes <= 0 ? 0u : bytes < (int64_t)kFar8 ? (uint32_t)bytes : kFar8;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)n, 0x00020000);
}

// The same over fewer than 2^31 bytes.
__device__ __forceinline__ rsrc8_t rsrc8_near(const void* base, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)bytes,
                                           0x00020000);
}

// 16 bytes a lane from global memory into LDS at `lds` + 16 lane.
__device__ __forceinline__ void copy16_lds(rsrc8_t r, void* lds, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (void __attribute__((address_space(3)))*)lds, 16,
                                           voff, soff, 0, 0);
}
__device__ __forceinline__ void copy4_lds(rsrc8_t r, void* lds, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (void __attribute__((address_space(3)))*)lds, 4,
                                           voff, soff, 0, 0);
}

__device__ __forceinline__ i32x16_t mfma_i8_32x32x32(u32x4_t a, u32x4_t b, i32x16_t c) {
  return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4_t, a),
                                               __builtin_bit_cast(i32x4_t, b), c, 0, 0, 0);
}
__device__ __forceinline__ i32x4_t mfma_i8_16x16x64(u32x4_t a, u32x4_t b, i32x4_t c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, a),
                                               __builtin_bit_cast(i32x4_t, b), c, 0, 0, 0);
}

// Tile order: workgroup b runs on XCD b % 8; an XCD's tiles are consecutive, and
// consecutive ones walk blocks of up to four row tiles by all column tiles, so that
// the workgroups of an XCD share both operands in its L2.
constexpr int kXcds = 8;
__device__ __forceinline__ bool tile_of(int id, int tiles_m, int tiles_n, int& tm, int& tn) {
  constexpr int G = 4;
  const int total = tiles_m * tiles_n, per = (total + kXcds - 1) / kXcds;
  id = (id % kXcds) * per + id / kXcds;
  if (id >= total || (int)(blockIdx.x / kXcds) >= per) return false;
  const int group = id / (G * tiles_n), in = id - group * G * tiles_n;
  const int left = tiles_m - group * G, g = left < G ? left : G;
  tn = in / g;
  tm = group * G + (in - tn * g);
  return true;
}

// f(0), f(1), .. f(N - 1) with the numbers as types (unrolled buffers).
template <int N, int K = 0, typename F>
__device__ __forceinline__ void in_turn(F&& f) {
  if constexpr (K < N) {
    f(std::integral_constant<int, K>{});
    in_turn<N, K + 1>(f);
  }
}

// Codes of a row.  With a = max |x| the code is 127 x / a, exact quotient,
// rounded to an integer, ties to even.  x and a are first multiplied by a power
// of two 2^-e that keeps 127 x and 1 / a inside binary32's range; t = 127 x 2^-e
// is exact (11 and 7 significant bits).  q = t r with r = fl(1 / a') is within a
// step or two of t / a', and one exact residual brings it within half a step and
// to the quotient itself where that is a half-integer.  With X, A the 11-bit
// significands and d the difference of the exponents, t / a' that is no
// half-integer is at least 2^-d / 2A > 2^-(d + 12) away from one, and a step of q
// < 2^(8 - d) is at most 2^-(d + 16): the rounding of q is that of the quotient.
// Adding 1.5 2^23 rounds q to the integer, ties to even, and leaves it in the low
// byte.
struct RowQuant {
  float c, a, r;   // 127 2^-e, a 2^-e, 1 / (a 2^-e); c = 0 for rows of zeros
  float scale;
};
// `top`: the largest |x| of the row as 16 bits (infinities and NaN above all).
template <bool F16>
__device__ __forceinline__ RowQuant row_quant(uint32_t top) {
  RowQuant p;
  const uint32_t inf = F16 ? 0x7c00u : 0x7f80u;
  float a;
  if (F16)
    a = (float)__builtin_bit_cast(_Float16, (uint16_t)top);
  else
    a = __uint_as_float(top << 16);
  if (top >= inf || top == 0) {
    p.c = 0.0f;
    p.a = 1.0f;
    p.r = 1.0f;
    p.scale = top == 0 ? 0.0f : __uint_as_float(0x7fc00000u);
    return p;
  }
  int e = (int)(__float_as_uint(a) >> 23) - 127;   // below -126 for subnormals
  e = e < -112 ? -112 : e;
  const float two = __uint_as_float((uint32_t)(127 - e) << 23);   // 2^-e, e -112 .. 127
  p.c = 127.0f * (e == 127 ? 0x1p-127f : two);
  p.a = a * (e == 127 ? 0x1p-127f : two);
  p.r = 1.0f / p.a;
  p.scale = a / 127.0f;
  return p;
}
// The code in the low byte.  In a row with infinities or NaN c is zero: t is then a
// zero or a NaN, whose low byte is zero too (16-bit NaN have no more bits to hand
// on).
__device__ __forceinline__ uint32_t code_of(float x, const RowQuant& p) {
  const float t = x * p.c;
  float q = t * p.r;
  q = __builtin_fmaf(__builtin_fmaf(-q, p.a, t), p.r, q);
  return __float_as_uint(q + 12582912.0f);
}
// The low bytes of four words as one.
__device__ __forceinline__ uint32_t pack_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return perm(perm(d, c, 0x0c0c0400u), perm(b, a, 0x0c0c0400u), 0x05040100u);
}

typedef __attribute__((ext_vector_type(2))) uint16_t u16x2_t;

__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t,
                            __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a),
                                                      __builtin_bit_cast(u16x2_t, b)));
}
// |x| as integers order like the values, infinities and NaN above them.
__device__ __forceinline__ uint32_t max_piece(uint32_t m, u32x4_t v) {
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max_halves(m, v[i] & 0x7fff7fffu);
  return m;
}

template <bool F16>
__device__ __forceinline__ u32x2_t codes_of(u32x4_t v, const RowQuant& p) {
  uint32_t q[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    if (F16) {
      const f16x2_t h = __builtin_bit_cast(f16x2_t, (uint32_t)v[i]);
      lo = (float)h[0];
      hi = (float)h[1];
    } else {
      lo = bf16lo_to_f32(v[i]);
      hi = bf16hi_to_f32(v[i]);
    }
    q[2 * i] = code_of(lo, p);
    q[2 * i + 1] = code_of(hi, p);
  }
  u32x2_t r = {pack_bytes(q[0], q[1], q[2], q[3]), pack_bytes(q[4], q[5], q[6], q[7])};
  return r;
}
// The largest of the wave's halves, in every lane.
__device__ __forceinline__ uint32_t wave_top(uint32_t m) {
  m = (m >> 16) > (m & 0xffffu) ? m >> 16 : m & 0xffffu;
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) {
    const uint32_t other = (uint32_t)__shfl_xor((int)m, o);
    m = m > other ? m : other;
  }
  return m;
}

// The value of code `i` of four, times a scale, in binary32.
__device__ __forceinline__ float code_value(uint32_t four, int i, float scale) {
  return (float)(int8_t)(four >> (8 * i)) * scale;
}

}  // namespace bnbx
