// gate_norm_grad_wide.cu -- the backward kernels of the gated residual and norms for
// rows that a cluster shares.
#include "gate_norm.cuh"
#include "variants.h"

namespace sptg {

template <bool BF16, bool BLOCK>
const void* gate_norm_grad_wide_of(int gate_kind) {
  switch (gate_kind) {
    case GATE_COLS: return reinterpret_cast<const void*>(&gate_norm_grad_kernel<BF16, 2, GATE_COLS, BLOCK, GRAD_WIDE>);
    case GATE_ROWS: return reinterpret_cast<const void*>(&gate_norm_grad_kernel<BF16, 2, GATE_ROWS, BLOCK, GRAD_WIDE>);
    case GATE_FULL: return reinterpret_cast<const void*>(&gate_norm_grad_kernel<BF16, 2, GATE_FULL, BLOCK, GRAD_WIDE>);
    default: return reinterpret_cast<const void*>(&gate_norm_grad_kernel<BF16, 2, GATE_NONE, BLOCK, GRAD_WIDE>);
  }
}

const void* gate_norm_grad_wide_variant(bool bf16, int gate_kind, bool block) {
  if (bf16) return block ? gate_norm_grad_wide_of<true, true>(gate_kind) : gate_norm_grad_wide_of<true, false>(gate_kind);
  return block ? gate_norm_grad_wide_of<false, true>(gate_kind) : gate_norm_grad_wide_of<false, false>(gate_kind);
}

}  // namespace sptg
