// Rows of 16-bit values to int8 codes with one scale a row, and back
// (include/bnbx_int8.h has the format).
//
// Both stream: 2 bytes in and 1 out an element, or 1 in and 2 out.  The
// quantizer holds its row in registers between the maximum and the codes, so X is
// read once: a team of T threads owns a row, thread t the 8-element pieces t, t +
// T, ...
#include "bnbx_int8_device.hpp"

namespace bnbx {
namespace {

constexpr int kThreads = 256;

// Piece p of a row: 8 values as 16-bit pairs, zero behind the row's end.  VEC: the
// row starts at 16 bytes.
template <bool VEC>
__device__ __forceinline__ u32x4_t load_piece(const uint16_t* row, int p, int cols) {
  const int k = 8 * p;
  if (VEC && k + 8 <= cols) return *(const u32x4_t*)(row + k);
  u32x4_t v = {0, 0, 0, 0};
  if (k < cols) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t e = k + i < cols ? row[k + i] : 0u;
      v[i / 2] |= e << (16 * (i & 1));
    }
  }
  return v;
}

// The largest of the team's maxima, in every thread of it.
template <int T>
__device__ __forceinline__ uint32_t team_max(uint32_t m, uint32_t* lds) {
  m = wave_top(m);
  if constexpr (T > 64) {
    constexpr int W = T / 64;
    __syncthreads();   // the last row's maxima are read
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = m;
    __syncthreads();
    m = lds[0];
#pragma unroll
    for (int w = 1; w < W; ++w) m = m > lds[w] ? m : lds[w];
  }
  return m;
}

// T threads a row, NP pieces a thread (0: any number, the row read twice).
template <int T, int NP, bool F16, bool VEC>
__global__ __launch_bounds__(T > kThreads ? T : kThreads) void quantize_rows_kernel(
    const uint16_t* __restrict__ x, int64_t ldx, Int8Rows q) {
  constexpr int kRows = T < kThreads ? kThreads / T : 1;   // rows a workgroup
  __shared__ uint32_t lds[T > 64 ? T / 64 : 1];
  const int t = threadIdx.x % T;
  const int pieces = (q.cols + 15) / 16 * 2;
  for (int64_t r = (int64_t)blockIdx.x * kRows + threadIdx.x / T; r < q.rows;
       r += (int64_t)gridDim.x * kRows) {
    const uint16_t* row = x + r * ldx;
    int8_t* out = q.codes + r * q.ld;
    uint32_t m = 0;
    if constexpr (NP > 0) {
      u32x4_t v[NP];
#pragma unroll
      for (int i = 0; i < NP; ++i) v[i] = load_piece<VEC>(row, t + i * T, q.cols);
#pragma unroll
      for (int i = 0; i < NP; ++i) m = max_piece(m, v[i]);
      const RowQuant p = row_quant<F16>(team_max<T>(m, lds));
#pragma unroll
      for (int i = 0; i < NP; ++i)
        if (t + i * T < pieces) *(u32x2_t*)(out + 8 * (t + i * T)) = codes_of<F16>(v[i], p);
      if (t == 0) q.scale[r] = p.scale;
    } else {
      for (int i = t; i < pieces; i += T) m = max_piece(m, load_piece<VEC>(row, i, q.cols));
      const RowQuant p = row_quant<F16>(team_max<T>(m, lds));
      for (int i = t; i < pieces; i += T)
        *(u32x2_t*)(out + 8 * i) = codes_of<F16>(load_piece<VEC>(row, i, q.cols), p);
      if (t == 0) q.scale[r] = p.scale;
    }
  }
}

// Values: T threads a row, 8 codes a thread and step.
template <int T, bool F16, bool VEC>
__global__ __launch_bounds__(kThreads) void dequantize_rows_kernel(Int8Rows q,
                                                                   uint16_t* __restrict__ out,
                                                                   int64_t ldo) {
  constexpr int kRows = kThreads / T;
  const int t = threadIdx.x % T;
  const int pieces = (q.cols + 7) / 8;
  for (int64_t r = (int64_t)blockIdx.x * kRows + threadIdx.x / T; r < q.rows;
       r += (int64_t)gridDim.x * kRows) {
    const int8_t* row = q.codes + r * q.ld;
    uint16_t* o = out + r * ldo;
    const float s = q.scale[r];
    for (int p = t; p < pieces; p += T) {
      const u32x2_t c = *(const u32x2_t*)(row + 8 * p);
      u32x4_t v;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = pack16x2<F16>(code_value(c[i / 2], 2 * (i & 1), s),
                             code_value(c[i / 2], 2 * (i & 1) + 1, s));
      if (VEC && 8 * p + 8 <= q.cols) {
        *(u32x4_t*)(o + 8 * p) = v;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (8 * p + i < q.cols) o[8 * p + i] = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
      }
    }
  }
}

constexpr int kMostGroups = 1 << 16;   // workgroups of a launch; they walk over the rows

int groups_for(int64_t rows, int per) {
  const int64_t n = (rows + per - 1) / per;
  return (int)(n < kMostGroups ? n : kMostGroups);
}

template <int T, int NP, bool F16, bool VEC>
hipError_t quantize(const uint16_t* x, int64_t ldx, const Int8Rows& q, hipStream_t s) {
  constexpr int threads = T > kThreads ? T : kThreads;
  quantize_rows_kernel<T, NP, F16, VEC>
      <<<groups_for(q.rows, threads / T), threads, 0, s>>>(x, ldx, q);
  return hipGetLastError();
}

// The team that holds a row with few idle pieces and enough loads a thread.
// Measured (us), (T, NP): 301 x 11008 (512, 3) 4.8, (256, 8) 5.4, (1024, 2) 5.4; 16 x
// 4096 (256, 2) 2.9, (1024, 1) 3.1; 2048 x 8192 (256, 4) 10.3, (1024, 1) 13.4; 8192 x
// 4096 (256, 2) 18.2, (64, 8) 19.3; 8192 x 14336 (512, 4) 64.0, (256, 8) 64.9.
template <bool F16, bool VEC>
hipError_t quantize(const uint16_t* x, int64_t ldx, const Int8Rows& q, hipStream_t s) {
  const int pieces = (q.cols + 15) / 16 * 2;
  if (pieces <= 64) return quantize<64, 1, F16, VEC>(x, ldx, q, s);
  if (pieces <= 256) return quantize<64, 4, F16, VEC>(x, ldx, q, s);
  if (pieces <= 512) return quantize<256, 2, F16, VEC>(x, ldx, q, s);
  if (pieces <= 1024) return quantize<256, 4, F16, VEC>(x, ldx, q, s);
  if (pieces <= 1536) return quantize<512, 3, F16, VEC>(x, ldx, q, s);
  if (pieces <= 2048) return quantize<512, 4, F16, VEC>(x, ldx, q, s);
  if (pieces <= 4096) return quantize<1024, 4, F16, VEC>(x, ldx, q, s);
  return quantize<1024, 0, F16, VEC>(x, ldx, q, s);
}

template <bool F16, bool VEC>
hipError_t dequantize(const Int8Rows& q, uint16_t* out, int64_t ldo, hipStream_t s) {
  if (q.cols <= 512) {
    dequantize_rows_kernel<64, F16, VEC><<<groups_for(q.rows, 4), kThreads, 0, s>>>(q, out, ldo);
  } else {
    dequantize_rows_kernel<256, F16, VEC><<<groups_for(q.rows, 1), kThreads, 0, s>>>(q, out, ldo);
  }
  return hipGetLastError();
}

bool pieces_at_16(const void* p, int64_t ld) { return (uintptr_t)p % 16 == 0 && ld % 8 == 0; }

}  // namespace

hipError_t launch_quantize_rows(const uint16_t* x, int64_t ldx, const Int8Rows& q, bool f16,
                                hipStream_t s) {
  if (q.rows == 0) return hipSuccess;
  const bool vec = pieces_at_16(x, ldx);
  if (f16) return vec ? quantize<true, true>(x, ldx, q, s) : quantize<true, false>(x, ldx, q, s);
  return vec ? quantize<false, true>(x, ldx, q, s) : quantize<false, false>(x, ldx, q, s);
}

hipError_t launch_dequantize_rows(const Int8Rows& q, uint16_t* out, int64_t ldo, bool f16,
                                  hipStream_t s) {
  if (q.rows == 0) return hipSuccess;
  const bool vec = pieces_at_16(out, ldo);
  if (f16) return vec ? dequantize<true, true>(q, out, ldo, s) : dequantize<true, false>(q, out, ldo, s);
  return vec ? dequantize<false, true>(q, out, ldo, s) : dequantize<false, false>(q, out, ldo, s);
}

}  // namespace bnbx
