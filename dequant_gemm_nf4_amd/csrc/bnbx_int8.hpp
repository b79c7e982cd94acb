// Internal declarations of libbnbx_int8 (include/bnbx_int8.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace bnbx {

// Rows of codes (bnbx_int8_rows, checked).
struct Int8Rows {
  int8_t* codes;
  float* scale;
  int64_t ld;
  int rows, cols;
};

hipError_t launch_quantize_rows(const uint16_t* x, int64_t ldx, const Int8Rows& q, bool f16,
                                hipStream_t stream);
hipError_t launch_dequantize_rows(const Int8Rows& q, uint16_t* out, int64_t ldo, bool f16,
                                  hipStream_t stream);

// Y = X . W^T over codes.
// (fits: whether a launch counts its threads in 32 bits)
bool int8_gemm_fits(int M, int N, int K);
size_t int8_gemm_workspace(int M, int N, int K);
hipError_t launch_int8_gemm(const Int8Rows& x, const Int8Rows& w, uint16_t* y, int64_t ldy,
                            bool f16, void* workspace, hipStream_t stream);

// The same for few rows of X, in one launch: x null, the codes q; else X's 16-bit
// rows, whose codes are written to q where it has any.
bool int8_few_takes(int M, int K);
bool int8_few_fits(int N);
hipError_t launch_int8_few(const uint16_t* x, int64_t ldx, const Int8Rows& q, const Int8Rows& w,
                           uint16_t* y, int64_t ldy, bool f16, hipStream_t stream);

// The same for up to 32 rows of X, without a workspace.
bool int8_rows16_takes(int M);
bool int8_rows16_fits(int N);
hipError_t launch_int8_rows16(const Int8Rows& x, const Int8Rows& w, uint16_t* y, int64_t ldy,
                              bool f16, hipStream_t stream);

// out[r, c] = sum_t A(r, t) v(t, c) over the values v of the codes [T, C], T and
// C their rows and columns: A(r, t) is dy[r ldy + t], or dy[t ldy + r] (`turned`).
enum { kOutBf16 = 0, kOutF16 = 1, kOutF32 = 2 };
struct GradGemm {
  const uint16_t* dy;
  int64_t ldy;
  int R;
  Int8Rows v;
  void* out;
  int64_t ldo;
  int out_type;
};
size_t int8_grad_workspace(int R, int C, int T);
hipError_t launch_int8_grad(const GradGemm& g, bool turned, bool f16, void* workspace,
                            hipStream_t stream);

// Workgroups of `threads` threads that a launch takes: it counts threads in 32 bits.
inline bool launch_fits(int64_t groups, int threads) {
  return groups < ((int64_t)1 << 32) / threads;
}

// Compute units of the device that was current when the process first asked (256 if it
// could not be asked): one number for all, so that a workspace's size and the call that
// takes it count alike whatever device is current.
int int8_cus();

// Workspaces are cut into pieces of whole 256 bytes.
inline size_t whole256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace bnbx
