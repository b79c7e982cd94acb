// Y = X . W^T over int8 codes for up to four rows of X (decode), for gfx950.
//
// Bound: streaming W once (N K bytes); for K = 4096 a row of W is four 16-byte
// loads a lane.  A wave owns a row of W at a time; lane l multiplies its pieces l, l
// + 64, ... with the same pieces of X's codes (v_dot4, four products an
// instruction) and the wave adds its lanes' int32 sums.  X's codes lie in LDS, and
// every workgroup makes them itself from the 16-bit rows (FUSED) while its first
// loads of W are under way: X is M K values, little beside a workgroup's part of W,
// and a launch of its own would cost more than the product.
#include "bnbx_int8_device.hpp"
#include "bnbx_int8_form.hpp"

namespace bnbx {
namespace {

constexpr int kWaves = kInt8FewWaves, kThreads = 64 * kWaves;
constexpr int kLdsCodes = 65536;   // most bytes of X's codes
constexpr int U = 4;               // loads of W a lane has under way, twice

struct FewArgs {
  const uint16_t* x;     // FUSED: 16-bit rows
  int64_t ldx;
  int8_t* xq;            // codes: read, or written if not null (FUSED)
  float* sx;
  int64_t ldq;
  const int8_t* w;
  const float* sw;
  int64_t ldw;
  int M, N, K;
  int rows;              // of W a wave
  uint16_t* y;
  int64_t ldy;
};

__device__ __forceinline__ u32x4_t piece_of(const uint16_t* row, int p, int cols, bool vec) {
  const int k = 8 * p;
  if (vec && k + 8 <= cols) return *(const u32x4_t*)(row + k);
  u32x4_t v = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t e = k + i < cols ? row[k + i] : 0u;
    v[i / 2] |= e << (16 * (i & 1));
  }
  return v;
}

// The wave's sum, in lane 63: within rows of 16 lanes, then across them.
__device__ __forceinline__ int lane63_sum(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);   // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);   // row_shr:2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);   // row_shr:4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);   // row_shr:8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);   // row_bcast:15
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);   // row_bcast:31
  return v;
}

template <int M, bool FUSED, bool F16>
__global__ __launch_bounds__(kThreads) void int8_few_kernel(FewArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];   // codes [M][kp]
  __shared__ uint32_t tops[kWaves];
  __shared__ float scales[M];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kp = (a.K + 15) / 16 * 16;
  const int n0 = ((int)blockIdx.x * kWaves + wave) * a.rows;
  const int batches = (kp + 16 * 64 * U - 1) / (16 * 64 * U);

  u32x4_t wv[2][U];
  auto load = [&](int set, int n, int b) {
    // rows past the end, and pieces past the row's: zeros (a piece's whole place is in
    // the lane's offset, since the range check leaves out the scalar one)
    const rsrc8_t r = rsrc8(a.w + (int64_t)n * a.ldw, n < a.N ? kp : 0);
    const uint32_t at = 16u * lane + (uint32_t)b * (1024u * U);
#pragma unroll
    for (int i = 0; i < U; ++i)
      wv[set][i] = __builtin_amdgcn_raw_buffer_load_b128(r, at + 1024u * i, 0, 2 /* streamed */);
  };
  load(0, n0, 0);

  if constexpr (FUSED) {
    constexpr int MT = M == 3 ? 4 : M, T = kThreads / MT, W = T / 64;   // threads a row
    const int m = threadIdx.x / T, t = threadIdx.x % T;
    const bool mine = m < M;
    const bool vec = (uintptr_t)a.x % 16 == 0 && a.ldx % 8 == 0;
    const uint16_t* row = a.x + (mine ? m : 0) * a.ldx;
    const int pieces = kp / 8;
    uint32_t top = 0;
    for (int p = t; p < pieces; p += T) top = max_piece(top, piece_of(row, p, a.K, vec));
    top = wave_top(top);
    if (lane == 0) tops[wave] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const uint32_t o = tops[(mine ? m : 0) * W + i];
      top = top > o ? top : o;
    }
    const RowQuant q = row_quant<F16>(top);
    if (mine) {
      for (int p = t; p < pieces; p += T) {
        const u32x2_t c = codes_of<F16>(piece_of(row, p, a.K, vec), q);
        *(u32x2_t*)(lds + m * kp + 8 * p) = c;
        if (a.xq != nullptr && blockIdx.x == 0) *(u32x2_t*)(a.xq + m * a.ldq + 8 * p) = c;
      }
      if (t == 0) {
        scales[m] = q.scale;
        if (a.xq != nullptr && blockIdx.x == 0) a.sx[m] = q.scale;
      }
    }
  } else {
    for (int p = threadIdx.x; p < M * (kp / 16); p += kThreads) {
      const int m = p / (kp / 16), c = p - m * (kp / 16);
      *(u32x4_t*)(lds + 16 * p) = *(const u32x4_t*)(a.xq + m * a.ldq + 16 * c);
    }
    if (threadIdx.x < M) scales[threadIdx.x] = a.sx[threadIdx.x];
  }
  __syncthreads();

  int set = 0;
  for (int j = 0; j < a.rows; ++j) {
    const int n = n0 + j;
    int sum[M];
#pragma unroll
    for (int m = 0; m < M; ++m) sum[m] = 0;
    auto batch = [&](int cur, int b) {
      const bool last = b + 1 == batches;
      if (!last || j + 1 < a.rows) load(cur ^ 1, last ? n + 1 : n, last ? 0 : b + 1);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int at = (b * U + i) * 1024 + 16 * lane;
        if (at < kp) {
#pragma unroll
          for (int m = 0; m < M; ++m) {
            const u32x4_t c = *(const u32x4_t*)(lds + m * kp + at);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              sum[m] = __builtin_amdgcn_sdot4((int)wv[cur][i][e], (int)c[e], sum[m], false);
          }
        }
      }
    };
    for (int b = 0; b < batches; ++b) {
      if (set == 0)
        batch(0, b);
      else
        batch(1, b);
      set ^= 1;
    }
#pragma unroll
    for (int m = 0; m < M; ++m) sum[m] = lane63_sum(sum[m]);
    if (lane == 63 && n < a.N) {
      const float s = a.sw[n];
#pragma unroll
      for (int m = 0; m < M; ++m)
        a.y[(int64_t)m * a.ldy + n] = f32_to_16<F16>(((float)sum[m] * scales[m]) * s);
    }
  }
}

template <int M, bool FUSED>
hipError_t launch(const FewArgs& a, bool f16, hipStream_t s) {
  const int kp = (a.K + 15) / 16 * 16;
  const int64_t per = (int64_t)kWaves * a.rows, grid = (a.N + per - 1) / per;
  if (f16)
    int8_few_kernel<M, FUSED, true><<<(int)grid, kThreads, M * kp, s>>>(a);
  else
    int8_few_kernel<M, FUSED, false><<<(int)grid, kThreads, M * kp, s>>>(a);
  return hipGetLastError();
}

template <bool FUSED>
hipError_t launch(const FewArgs& a, bool f16, hipStream_t s) {
  switch (a.M) {
    case 1: return launch<1, FUSED>(a, f16, s);
    case 2: return launch<2, FUSED>(a, f16, s);
    case 3: return launch<3, FUSED>(a, f16, s);
    default: return launch<4, FUSED>(a, f16, s);
  }
}

}  // namespace

bool int8_few_takes(int M, int K) {
  return M <= 4 && (int64_t)M * ((K + 15) / 16 * 16) <= kLdsCodes;
}

bool int8_few_fits(int N) { return launch_fits((int64_t)N / kWaves + 1, kThreads); }

hipError_t launch_int8_few(const uint16_t* x, int64_t ldx, const Int8Rows& q, const Int8Rows& w,
                           uint16_t* y, int64_t ldy, bool f16, hipStream_t s) {
  FewArgs a{};
  a.x = x;
  a.ldx = ldx;
  a.xq = q.codes;
  a.sx = q.scale;
  a.ldq = q.ld;
  a.w = w.codes;
  a.sw = w.scale;
  a.ldw = w.ld;
  a.M = q.rows;
  a.N = w.rows;
  a.K = w.cols;
  a.rows = int8_few_rows(a.M, a.N, int8_cus());
  a.y = y;
  a.ldy = ldy;
  return x != nullptr ? launch<true>(a, f16, s) : launch<false>(a, f16, s);
}

}  // namespace bnbx
