// Rows to groups for gfx950: the stable counting sort of row numbers by a
// small group id, and each group's bounds.
//
// place(i) = #{j : key_j < key_i} + #{j < i : key_j = key_i}, with key = id, or
// `groups` for an id outside 0 .. groups-1.
//
// A workgroup of 16 waves takes a chunk of rows, wave w the w-th of 16 equal
// parts of it, 64 rows at a time in row order.  Lanes of one key find each
// other by one ballot per key bit (the lanes that agree in every bit), so a
// row's rank among the wave's 64 is a population count and one lane per key
// adds the count to the wave's own counter in LDS, so the order never
// depends on timing.  A first pass counts, a prefix over waves and then
// keys turns the counters into places, and a second pass writes each row to
// its place.
//
// Bound: latency at every size here (4 bytes read and 4 written a row; the
// launch, the dependent passes and, for many chunks, a second launch, which
// counts its rows once more before it places them).  Up to
// kOneChunk rows one workgroup does everything in one launch; more rows are cut
// into at most kMaxChunks chunks, whose key counts go to the workspace in a
// first launch; in the second, every workgroup adds the counts of all chunks
// itself (groups + 1 counters a chunk, from L2, wave w the chunks w, w + 16, ..;
// integer sums, whose order does not matter) instead of waiting for a third
// launch to do it.  Measured: 32 rows 3.3 us; 131072 rows into 64 groups 4.0 us
// and 8.1 us (with one thread adding each key's counts 26 us).
#include "bnbx_device.hpp"
#include "bnbx_rows.hpp"

namespace bnbx {
namespace {

constexpr int kWaves = 16, kThreads = kWaves * 64;
constexpr int kOneChunk = 8192;    // rows one workgroup sorts alone
constexpr int kMinChunk = 2048;    // rows per chunk otherwise
constexpr int kMaxChunks = 128;
constexpr int kStride = kMaxGroups + 1;   // counters per wave: every group, and "none"

struct Chunks {
  int n, rows;   // chunks, rows per chunk (a multiple of kThreads)
};
Chunks chunks_of(int rows) {
  if (rows <= kOneChunk) return Chunks{1, (rows + kThreads - 1) / kThreads * kThreads};
  int64_t per = ((int64_t)rows + kMaxChunks - 1) / kMaxChunks;
  per = (per + kThreads - 1) / kThreads * kThreads;
  per = per < kMinChunk ? kMinChunk : per;
  return Chunks{(int)(((int64_t)rows + per - 1) / per), (int)per};
}

// The lanes of the wave with this lane's key (all 64 lanes active).
__device__ __forceinline__ uint64_t peers(int key, int bits) {
  uint64_t m = ~0ull;
  for (int b = 0; b < bits; ++b) {
    const bool one = (key >> b) & 1;
    const uint64_t set = __ballot(one);
    m &= one ? set : ~set;
  }
  return m;
}

// One wave over its rows [i0, i1): `each(row, key, rank, count, first)` for
// every row inside, with rank among the wave's 64 rows of that key.
template <typename F>
__device__ __forceinline__ void walk(const int32_t* __restrict__ ids, int64_t i0, int64_t i1,
                                     int groups, int bits, F each) {
  const int lane = threadIdx.x & 63;
  const uint64_t below = (1ull << lane) - 1ull;
  int32_t next = i0 + lane < i1 ? ids[i0 + lane] : -1;
  for (int64_t i = i0; i < i1; i += 64) {
    const int32_t id = next;
    next = i + 64 + lane < i1 ? ids[i + 64 + lane] : -1;
    const bool in = i + lane < i1;
    const int key = id >= 0 && id < groups ? id : groups;
    // lanes past the end take part with a key of their own (all bits set)
    const uint64_t m = peers(in ? key : (1 << bits) - 1, bits);
    if (in) each((int)(i + lane), key, __popcll(m & below), __popcll(m), (m & below) == 0);
    // the next 64 rows read counters that other lanes have just written
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}

// PHASE 0: all in one workgroup.  1: the chunk's key counts into counts[chunk].
// 2: places from all chunks' counts.
template <int PHASE>
__global__ __launch_bounds__(kThreads) void group_rows_kernel(
    const int32_t* __restrict__ ids, int rows, int groups, int bits, int chunk_rows, int nchunks,
    int32_t* __restrict__ counts, int32_t* __restrict__ offsets, int32_t* __restrict__ order) {
  __shared__ int hist[kWaves * kStride];
  __shared__ int wsum[kWaves];
  // PHASE 2: each key's rows in all chunks, and in the chunks before this one
  __shared__ int total[PHASE == 2 ? kStride : 1], earlier[PHASE == 2 ? kStride : 1];
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int keys = groups + 1;
  const int64_t c0 = (int64_t)blockIdx.x * chunk_rows;
  const int64_t c1 = c0 + chunk_rows < rows ? c0 + chunk_rows : rows;
  // the wave's part: equal multiples of 64 rows
  const int64_t per = (((c1 - c0) + kThreads - 1) / kThreads) * 64;
  const int64_t a = c0 + wave * per;
  const int64_t i0 = a < c1 ? a : c1, i1 = a + per < c1 ? a + per : c1;
  int* const mine = hist + wave * kStride;

  for (int k = lane; k < keys; k += 64) mine[k] = 0;
  if (PHASE == 2)
    for (int k = t; k < keys; k += kThreads) total[k] = earlier[k] = 0;
  __syncthreads();
  if (PHASE == 2) {
    for (int k = lane; k < keys; k += 64) {
      int all = 0, before = 0;
#pragma unroll 8
      for (int c = wave; c < nchunks; c += kWaves) {
        const int n = counts[(int64_t)c * keys + k];
        all += n;
        before += c < (int)blockIdx.x ? n : 0;
      }
      atomicAdd(&total[k], all);
      atomicAdd(&earlier[k], before);
    }
  }
  walk(ids, i0, i1, groups, bits, [&](int, int key, int, int n, bool first) {
    if (first) mine[key] += n;
  });
  __syncthreads();

  if (PHASE == 1) {
    for (int k = t; k < keys; k += kThreads) {
      int n = 0;
      for (int w = 0; w < kWaves; ++w) n += hist[w * kStride + k];
      counts[(int64_t)blockIdx.x * keys + k] = n;
    }
    return;
  }

  // Thread k: key k's rows in all chunks (`all`) and in the chunks before
  // this one (`before`); then the exclusive prefix of `all` over the keys.
  // Key `groups` (none) starts where the last group ends.
  int all = 0, before = 0;
  if (t < groups) {
    if (PHASE == 0) {
      for (int w = 0; w < kWaves; ++w) all += hist[w * kStride + t];
    } else {
      all = total[t];
      before = earlier[t];
    }
  }
  int incl = all;
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 63) wsum[wave] = incl;
  __syncthreads();
  int start = incl - all;
  for (int w = 0; w < wave; ++w) start += wsum[w];
  if (blockIdx.x == 0 && t < groups) {
    offsets[t] = start;
    if (t == groups - 1) offsets[groups] = start + all;
  }
  if (t < groups) {
    int at = start + before;
    for (int w = 0; w < kWaves; ++w) {
      const int n = hist[w * kStride + t];
      hist[w * kStride + t] = at;
      at += n;
    }
  }
  if (t == kThreads - 1) {
    // rows of no group: behind every group, after the earlier chunks' ones
    int at = 0;
    for (int w = 0; w < kWaves; ++w) at += wsum[w];
    if (PHASE == 2) at += earlier[groups];
    for (int w = 0; w < kWaves; ++w) {
      const int n = hist[w * kStride + groups];
      hist[w * kStride + groups] = at;
      at += n;
    }
  }
  __syncthreads();
  walk(ids, i0, i1, groups, bits, [&](int row, int key, int rank, int n, bool first) {
    const int at = mine[key];
    order[at + rank] = row;
    if (first) mine[key] = at + n;
  });
}

}  // namespace

size_t group_rows_workspace_bytes(int rows, int groups) {
  const Chunks c = chunks_of(rows);
  return c.n == 1 ? 0 : (size_t)c.n * (size_t)(groups + 1) * sizeof(int32_t);
}

hipError_t launch_group_rows(const int32_t* ids, int rows, int groups, int32_t* offsets,
                             int32_t* order, int32_t* workspace, hipStream_t stream) {
  const Chunks c = chunks_of(rows);
  int bits = 1;
  while ((1 << bits) <= groups + 1) ++bits;   // keys 0 .. groups, and a pattern of its own
  if (c.n == 1) {
    hipLaunchKernelGGL(group_rows_kernel<0>, dim3(1), dim3(kThreads), 0, stream, ids, rows,
                       groups, bits, c.rows, 1, nullptr, offsets, order);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(group_rows_kernel<1>, dim3(c.n), dim3(kThreads), 0, stream, ids, rows,
                     groups, bits, c.rows, c.n, workspace, nullptr, nullptr);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(group_rows_kernel<2>, dim3(c.n), dim3(kThreads), 0, stream, ids, rows,
                     groups, bits, c.rows, c.n, workspace, offsets, order);
  return hipGetLastError();
}

}  // namespace bnbx
