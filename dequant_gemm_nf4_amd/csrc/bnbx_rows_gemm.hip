// Expert-grouped 4-bit products for gfx950, many rows a group: the tiles of
// bnbx_gemm_core.hpp, a tile's 256 rows the places of one group.  Bound: the
// matrix cores and their feed, as the ungrouped form, and the groups' last tiles
// (half empty on average).  8192 rows in 8 uneven groups of 14336 x 4096: 1005
// us, 957 TFLOP/s.
#include "bnbx_rows_gemm.hpp"

namespace bnbx {

hipError_t launch_rows_gemm(const RowsGemm& a, int quant_type, bool f16, hipStream_t stream,
                            bool launch) {
  return launch_rows_tiles<false>(a, quant_type, f16, stream, launch);
}

}  // namespace bnbx
