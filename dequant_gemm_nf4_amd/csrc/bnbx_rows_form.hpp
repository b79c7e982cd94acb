// Which form a product over grouped rows takes, from what the host knows: the
// plan's rows, its groups (0: all rows are one group), the output columns, the
// low-rank term and the GPU's compute units.  Plain host code with no HIP in it, so that a test
// can ask which form its sizes reach.
#pragma once

namespace bnbx {

// Rounds of workgroups that a launch over grouped rows takes on a GPU with
// `slots` of them: tiles of tm places and tn of the `cols` columns, a group's
// last tile half full (and one tile at least); a launch ends `late` rounds
// after its tiles have filled the GPU on average.
inline double rounds_of(int rows, int groups, int cols, int tm, int tn, int slots, double late) {
  const double used = groups == 0 ? 1 : groups < rows ? groups : rows;
  double tiles = groups == 0 ? (double)(((long long)rows + tm - 1) / tm)
                             : (double)rows / tm + 0.5 * used;
  tiles = tiles < used ? used : tiles;
  const double r = tiles * (((long long)cols + tn - 1) / tn) / slots + late;
  return r < 1.0 ? 1.0 : r;
}

// Adapters that meet a tile of tm places: `adapters` of them in use alike (the
// host does not know which have rows), the places in their order.
inline double segments_of(int rows, int adapters, int tm) {
  const double used = adapters < rows ? adapters : rows;
  const double met = 1.0 + tm * used / rows, most = used < tm ? used : tm;
  return met < most ? met : most;
}

// Whether the tiled form is likely to be the faster one.  Its workgroups (256
// places x 256 columns, one a CU) take about 1.5 us per 64 k, those of the
// streaming form (64 places x 128 columns, two a CU) about 1.0 us, each with a
// full GPU.  Measured, 8 groups of N = K = 4096: 64 rows a group 69 us streaming
// / 106 us tiled, 160 rows 101 / 104, 256 rows 158 / 110; one group, 333 rows,
// N = 4096, K = 11008: 93 / 229.
//
// With a low-rank term of `rank` (0: none) every adapter that meets a tile adds
// work: two or three products a 32 x 32 tile and 16 ranks, each behind its loads,
// in a tiled workgroup, and less in a streaming one.  Counted as 1.0 us per 16
// ranks against 0.6 us per 32, the form chosen takes 0.5 % more than the faster of
// the two over 10600 drawn sizes of 150 to 2048 rows whose adapters change often
// and 0.7 % over 5100 with few of the pool in use (5.7 % and 1.8 % without the
// term); 2 % of all are more than 10 % off, at worst 1.9 times.  With 1.55 and
// 0.8 us, nearer to measured times, the first is 0.45 %, the second 0.9 %.
// Measured, 600 rows, N = 11008, K = 4096, 64 adapters: rank 16 141 us streaming
// / 143 tiled, rank 256 338 / 736; 2048 rows, N = K = 8192: 8 adapters of rank 64
// 544 / 282, 64 of rank 256 743 / 518.
inline bool prefer_tiles(int rows, int groups, int N, int K, int adapters, int rank, int cus) {
  if (rows <= 32 * (long long)(groups == 0 ? 1 : groups)) return false;
  double tiled = 1.5 * (K / 64), streaming = K / 64;
  if (rank > 0) {
    tiled += 1.0 * segments_of(rows, adapters, 256) * (rank / 16);
    streaming += 0.6 * segments_of(rows, adapters, 64) * ((rank + 31) / 32);
  }
  return tiled * rounds_of(rows, groups, N, 256, 256, cus, 0.5) <
         streaming * rounds_of(rows, groups, N, 64, 128, 2 * cus, 0.5);
}

// The same for the input gradient: 256 x 256 tiles at 2.0 us per 64 weight
// rows, the streaming form's 32 places x 128 columns at 0.38 us.  Measured, 8
// groups of N = K = 4096: 50 rows a group 49 us streaming / 126 us tiled, 128
// rows 116 / 129, 160 rows 136 / 128, 256 rows 209 / 134.
inline bool prefer_dx_tiles(int rows, int groups, int K, int cus) {
  return 5.2 * rounds_of(rows, groups, K, 256, 256, cus, 0.25) <
         rounds_of(rows, groups, K, 32, 128, cus, 0.25);
}

}  // namespace bnbx
