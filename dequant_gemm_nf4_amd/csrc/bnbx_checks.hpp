// Host-side argument checks shared by the C entry points of both libraries.
#pragma once

#include "../../include/bnbx.h"
#include "bnbx_internal.hpp"

namespace bnbx {

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

inline int check_state(const bnbx_nf4_state* st) {
  if (!tables_ok()) return BNBX_E_INTERNAL;
  if (st == nullptr) return BNBX_E_INVAL;
  if (st->n < 2 || (st->n & 1)) return BNBX_E_INVAL;
  if (st->blocksize != kBlock) return BNBX_E_UNSUPPORTED;
  if (st->double_quant != kDqNone && st->double_quant != kDqLinear &&
      st->double_quant != kDqDynamic)
    return BNBX_E_INVAL;
  if (st->quant_type != BNBX_QUANT_NF4 && st->quant_type != BNBX_QUANT_FP4) return BNBX_E_INVAL;
  if (st->compute_dtype != BNBX_DTYPE_BF16 && st->compute_dtype != BNBX_DTYPE_F16)
    return BNBX_E_INVAL;
  if (st->absmax == nullptr) return BNBX_E_INVAL;
  if (st->double_quant && (st->absmax2 == nullptr || st->absmax_mean == nullptr))
    return BNBX_E_INVAL;
  return BNBX_OK;
}

inline int hip_status(hipError_t e) { return e == hipSuccess ? BNBX_OK : BNBX_E_HIP; }

}  // namespace bnbx
