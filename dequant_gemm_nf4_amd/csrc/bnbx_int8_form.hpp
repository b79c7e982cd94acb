// Which form a product of the 8-bit operators takes, from its sizes and the GPU's
// compute units.  Plain host code with no HIP in it, so that a test can ask which form
// its sizes reach.
#pragma once

namespace bnbx {

// A tile: rows and columns of the result a workgroup, and the time of a step of the
// summed axis with a workgroup on every CU (us).
struct Int8Shape {
  int rows, cols;
  double step;
};
struct Int8Form {
  int shape;               // in its table
  int splits, steps_per;   // of the summed axis
};

// The forward product (2048 x 8192 x 8192 and the sizes below, timed one form after the
// other), in steps of 128 of K.
constexpr int kInt8GemmStep = 128;
constexpr Int8Shape kInt8GemmShapes[] = {
    {256, 256, 1.72}, {256, 128, 1.05}, {128, 128, 0.60}, {128, 64, 0.36}, {64, 64, 0.23}};
// The gradients (4096 x 11008 x 4096 and the sizes below), in steps of 64 of t.
constexpr int kInt8GradStep = 64;
constexpr Int8Shape kInt8GradShapes[] = {
    {256, 256, 1.72}, {128, 256, 0.92}, {128, 128, 0.57}, {64, 128, 0.36}, {32, 128, 0.31}};

// The form and the split of the summed axis that take the least by this count: rounds of
// workgroups over the CUs (a last round that is not full is a little faster),
// their steps, 4 us for a launch's first copies and its results, and for a split 3 us
// for the second launch and the partial sums written and read at 6.5 TB/s.
template <int N>
Int8Form int8_form(const Int8Shape (&shapes)[N], int rows, int cols, int steps, int most_splits,
                   int cus) {
  Int8Form best{0, 1, steps};
  double least = 1e30;
  for (int i = 0; i < N; ++i) {
    const Int8Shape& f = shapes[i];
    const long long tiles = (((long long)rows + f.rows - 1) / f.rows) *
                            (((long long)cols + f.cols - 1) / f.cols);
    for (int splits = 1; splits <= most_splits && (splits == 1 || steps / splits >= 4); ++splits) {
      const int per = (steps + splits - 1) / splits, n = per > 0 ? (steps + per - 1) / per : 1;
      if (n > 1 && tiles * n > 2 * (long long)cus) break;
      const double fill = (double)(tiles * n) / cus;
      const double rounds = fill <= 1.0 ? 0.7 + 0.3 * fill : (double)((tiles * n + cus - 1) / cus);
      const double us = rounds * per * f.step + 4.0 +
                        (n > 1 ? 3.0 + 8.0 * n * (double)rows * (double)cols / 6.5e6 : 0.0);
      if (us < least) {
        least = us;
        best = {i, n, per};
      }
    }
  }
  return best;
}

// Y [M, N] summed over K.  Counted and measured (us), 301 x 4096 x 11008: 128 x 64
// whole 33 / 31, 128 x 128 in two splits 34 / 34, 64 x 64 whole 44 / 44; 1000 x 4096 x
// 11008: 128 x 128 whole 56 / 58, 256 x 128 in two 61 / 64; 2048 x 4096 x 4096: 256 x
// 128 whole 38 / 38, 256 x 256 whole 51 / 48.
inline Int8Form int8_gemm_form(int M, int N, int K, int cus) {
  const int steps = (int)(((long long)K + kInt8GemmStep - 1) / kInt8GemmStep);
  return int8_form(kInt8GemmShapes, M, N, steps, 16, cus);
}

// A gradient [R, C] summed over T.  Counted and measured (us), R x T x C = 200 x 4096 x
// 4096: 128 x 128 in four 20 / 21, 64 x 128 in two 21 / 23, 128 x 256 in eight 22 / 25;
// 1000 x 4096 x 4096: 128 x 128 whole 40 / 42, 128 x 256 in two 43 / 46; 1001 x 777 x
// 4100: 128 x 256 whole 14 / 21, 64 x 128 whole 18 / 23.
inline Int8Form int8_grad_form(int R, int C, int T, int cus) {
  const int steps = (int)(((long long)T + kInt8GradStep - 1) / kInt8GradStep);
  return int8_form(kInt8GradShapes, R, C, steps, 32, cus);
}

// Forward products of up to this many rows of X run the form whose waves split K.  From 33
// rows on the tiles are faster: 64 x 11008 x 4096 15.6 us against 22.3 there, 64 x 4096 x
// 11008 17.9 / 21.8 (but 64 x 4096 x 4096 10.3 / 9.1); 32 x 11008 x 4096 16.2 / 15.4,
// 16 x 11008 x 4096 15.1 / 12.7.
constexpr int kInt8WaveRows = 32;

// Rows of W a wave of the form for up to four rows of X takes, 16 waves a workgroup.
// One row of X: one.  More rows of X cost a workgroup more before its first product: then
// as many as keep the launch to one workgroup a CU, up to eight.  1, 2, 4 rows beside
// 11008 x 4096: 11.1, 15.3, 19.4 us a row a wave, 11.5, 12.1, 13.4 three a wave; beside
// 32000 x 4096 25.6, 36.8, 46.9 and 30.8, 31.9, 33.0 eight a wave.
constexpr int kInt8FewWaves = 16;
inline int int8_few_rows(int M, int N, int cus) {
  if (M == 1) return 1;
  const long long groups = ((long long)N + kInt8FewWaves - 1) / kInt8FewWaves;
  const long long each = (groups + cus - 1) / cus;
  return (int)(each < 8 ? each : 8);
}

}  // namespace bnbx
