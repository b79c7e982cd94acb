// The shared 4-bit weight beside many adapters for gfx950, many rows: the tiles
// of bnbx_gemm_core.hpp over the rows in adapter order, each place with its
// adapter's low-rank term accumulated before the 4-bit product.  Bound: the
// matrix cores and their feed; the low-rank term adds about 1.5 us per 16 ranks of
// every adapter that meets a tile (its loads are waited for one by one).  2048
// rows of 8 adapters of rank 64 beside an 8192 x 8192 weight: 264 us (and 27 us of
// down-projection before it).
#include "bnbx_rows_gemm.hpp"

namespace bnbx {

hipError_t launch_rows_gemm_lora(const RowsGemm& a, int quant_type, bool f16, hipStream_t stream,
                                 bool launch) {
  return launch_rows_tiles<true>(a, quant_type, f16, stream, launch);
}

}  // namespace bnbx
