// Y = X . W^T over int8 codes for up to 32 rows of X (decode batches), for gfx950.
//
// Bound: streaming W once.  A workgroup owns 16 rows of W and all rows of X (16 FM);
// its waves take the 128-byte steps of K in turn, each with a tile of its own (FM of
// v_mfma_i32_16x16x64_i8, W the A operand), and add their int32 sums
// through LDS at the end.  So no wave waits for another until then, and a launch
// needs no second one to join parts of K.
//
// Both operands go from global memory straight into a wave's own LDS (buffer_load
// ... lds, eight rows of 128 bytes an instruction, 16-byte chunks permuted by the
// row pair so that 16 lanes reading one chunk of 16 rows meet all banks once); two
// steps are under way at a time, and a wave waits for the older one only (16 x 11008 x
// 4096, timed with eight waves a workgroup: three steps 15.7 us, two 13.5, for fewer
// workgroups fit a CU; the four waves that this size takes 10.2-12.5).  Rows
// past the end and chunks past K read as zeros through the buffer range check.
#include "bnbx_int8_device.hpp"
#include "bnbx_int8_form.hpp"

namespace bnbx {
namespace {

constexpr int BK = 128;

struct Rows16Args {
  const int8_t* x;
  const int8_t* w;
  const float* sx;
  const float* sw;
  int64_t ldx, ldw;
  int M, N, K;
  uint16_t* y;
  int64_t ldy;
};

template <int FM, int WV, bool F16>
__global__ __launch_bounds__(WV * 64) void int8_rows16_kernel(Rows16Args a) {
  constexpr int kTile = 16 * BK, kStep = (1 + FM) * kTile;   // bytes of a wave's step
  constexpr int C = 2 * (1 + FM);                            // copies of a step
  __shared__ __attribute__((aligned(16))) uint8_t buf0[WV * kStep];
  __shared__ __attribute__((aligned(16))) uint8_t buf1[WV * kStep];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = (int)blockIdx.x * 16;
  const int steps = (a.K + BK - 1) / BK, kp = (a.K + 15) / 16 * 16;
  const rsrc8_t rw = rsrc8(a.w + (int64_t)n0 * a.ldw, (int64_t)kFar8);
  const rsrc8_t rx = rsrc8(a.x, (int64_t)kFar8);

  // copies: instruction i fills rows 8 i .. 8 i + 7 of the step (16 of W, then X's), lane
  // l chunk slot l % 8 of row l / 8; odd instructions permute by 4 more
  uint32_t off[C];
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const bool isw = i < 2;
    const int r = 8 * (isw ? i : i - 2) + (lane >> 3);
    const int chunk = (lane & 7) ^ ((r >> 1) & 7);
    const bool in = isw ? n0 + r < a.N : r < a.M;
    off[i] = in ? (uint32_t)r * (uint32_t)(isw ? a.ldw : a.ldx) + 16u * chunk : kFar8;
  }
  const int c0 = (lane & 7) ^ ((lane >> 4) & 3);
  auto copies = [&](uint8_t* buf, int t) {
    const int left = kp - t * BK;
    const bool ok0 = 16 * c0 < left, ok1 = 16 * (c0 ^ 4) < left;
    uint8_t* const mine = buf + wave * kStep;
#pragma unroll
    for (int i = 0; i < C; ++i)
      copy16_lds(i < 2 ? rw : rx, mine + i * 1024, ((i & 1) ? ok1 : ok0) ? off[i] : kFar8,
                 (uint32_t)t * BK);
  };

  i32x4_t acc[FM];
#pragma unroll
  for (int j = 0; j < FM; ++j) acc[j] = i32x4_t{0, 0, 0, 0};
  // operand reads: row l % 16, chunk 4 s + l / 16
  const int row = lane & 15, q4 = lane >> 4;
  uint32_t rd[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) rd[s] = row * BK + 16 * ((4 * s + q4) ^ ((row >> 1) & 7));
  auto products = [&](const uint8_t* buf) {
    const uint8_t* const mine = buf + wave * kStep;
    u32x4_t ow[2], ox[2][FM];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      ow[s] = *(const u32x4_t*)(mine + rd[s]);
#pragma unroll
      for (int j = 0; j < FM; ++j) ox[s][j] = *(const u32x4_t*)(mine + (1 + j) * kTile + rd[s]);
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int j = 0; j < FM; ++j) acc[j] = mfma_i8_16x16x64(ow[s], ox[s][j], acc[j]);
  };
  // steps past the end copy zeros, which nothing multiplies
  int t = wave;
  copies(buf0, t);
  copies(buf1, t + WV);
  auto step = [&](uint8_t* buf) {
    __builtin_amdgcn_s_waitcnt(0x0F70 | C);   // vmcnt(C): the older of two steps has landed
    asm volatile("" ::: "memory");
    products(buf);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // its operands have been read
    copies(buf, t + 2 * WV);
    t += WV;
  };
  static_assert(C < 16, "the memory counter's low bits");
  while (t < steps) {
    step(buf0);
    if (t >= steps) break;
    step(buf1);
  }
  __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0): no copy is in flight
  __syncthreads();

  // the waves' sums: a lane's four values of a tile in 16 bytes, wave by wave
  static_assert(FM * 1024 <= kStep, "a buffer holds every wave's tiles");
#pragma unroll
  for (int j = 0; j < FM; ++j) *(i32x4_t*)(buf0 + 16 * ((wave * FM + j) * 64 + lane)) = acc[j];
  __syncthreads();
  if (wave < FM) {
    i32x4_t s = {0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < WV; ++w)
      s += *(const i32x4_t*)(buf0 + 16 * ((w * FM + wave) * 64 + lane));
    const int m = 16 * wave + row, n = n0 + 4 * q4;
    if (m < a.M && n < a.N) {
      const float sx = a.sx[m];
      float f[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) f[k] = ((float)s[k] * sx) * (n + k < a.N ? a.sw[n + k] : 0.0f);
      uint16_t* y = a.y + (int64_t)m * a.ldy + n;
      const u32x2_t v = {pack16x2<F16>(f[0], f[1]), pack16x2<F16>(f[2], f[3])};
      if (n + 4 <= a.N && ((uintptr_t)a.y % 8 == 0) && a.ldy % 4 == 0) {
        *(u32x2_t*)y = v;
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (n + k < a.N) y[k] = (uint16_t)(v[k / 2] >> (16 * (k & 1)));
      }
    }
  }
}

template <int FM, int WV>
hipError_t launch(const Rows16Args& a, bool f16, hipStream_t s) {
  const int64_t grid = ((int64_t)a.N + 15) / 16;
  if (f16)
    int8_rows16_kernel<FM, WV, true><<<(int)grid, WV * 64, 0, s>>>(a);
  else
    int8_rows16_kernel<FM, WV, false><<<(int)grid, WV * 64, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

bool int8_rows16_takes(int M) { return M <= kInt8WaveRows; }

bool int8_rows16_fits(int N) { return launch_fits((int64_t)N / 16 + 1, 512); }

hipError_t launch_int8_rows16(const Int8Rows& x, const Int8Rows& w, uint16_t* y, int64_t ldy,
                              bool f16, hipStream_t s) {
  const Rows16Args a{x.codes, w.codes, x.scale, w.scale, x.ld, w.ld, x.rows, w.rows, x.cols,
                     y,       ldy};
  // Many groups of 16 rows of W: four waves each, so that a CU holds more of them;
  // few: eight, which split K further.  16 x 11008 x 4096 12.7 us / 13.5 with eight, 16
  // x 4096 x 4096 6.5 / 6.2; 32 x 11008 x 4096 15.4 / 18.8, 32 x 4096 x 11008 17.9 / 16.4.
  const bool many = w.rows / 16 > 2 * int8_cus();
  if (x.rows <= 16) return many ? launch<1, 4>(a, f16, s) : launch<1, 8>(a, f16, s);
  return many ? launch<2, 4>(a, f16, s) : launch<2, 8>(a, f16, s);
}

}  // namespace bnbx
