// Which form a product over grouped rows takes, from what the host knows: the
// plan's rows, its groups (0: all rows are one group), the output columns and
// the GPU's compute units.  Plain host code with no HIP in it, so that a test
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

// Whether the tiled form is likely to be the faster one.  Its workgroups (256
// places x 256 columns, one a CU) take about 1.5 us per 64 k, those of the
// streaming form (64 places x 128 columns, two a CU) about 1.0 us, each with a
// full GPU.  Measured, 8 groups of N = K = 4096: 64 rows a group 69 us streaming
// / 106 us tiled, 160 rows 101 / 104, 256 rows 158 / 110; one group, 333 rows,
// N = 4096, K = 11008: 93 / 229.
inline bool prefer_tiles(int rows, int groups, int N, int cus) {
  if (rows <= 32 * (long long)(groups == 0 ? 1 : groups)) return false;
  return 1.5 * rounds_of(rows, groups, N, 256, 256, cus, 0.5) <
         rounds_of(rows, groups, N, 64, 128, 2 * cus, 0.5);
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
