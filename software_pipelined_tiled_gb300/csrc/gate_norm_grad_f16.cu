// gate_norm_grad_f16.cu -- the backward kernels of the gated residual and norms, f16 rows.
#include "gate_norm.cuh"
#include "variants.h"

namespace sptg {

template <bool BLOCK, int FORM>
const void* gate_norm_grad_of(int gate_kind) {
  switch (gate_kind) {
    case GATE_COLS: return reinterpret_cast<const void*>(&gate_norm_grad_kernel<false, 2, GATE_COLS, BLOCK, FORM>);
    case GATE_ROWS: return reinterpret_cast<const void*>(&gate_norm_grad_kernel<false, 2, GATE_ROWS, BLOCK, FORM>);
    case GATE_FULL: return reinterpret_cast<const void*>(&gate_norm_grad_kernel<false, 2, GATE_FULL, BLOCK, FORM>);
    default: return reinterpret_cast<const void*>(&gate_norm_grad_kernel<false, 2, GATE_NONE, BLOCK, FORM>);
  }
}

const void* gate_norm_grad_f16(int gate_kind, bool block, bool cut) {
  if (block)
    return cut ? gate_norm_grad_of<true, GRAD_CUT>(gate_kind) : gate_norm_grad_of<true, GRAD_WHOLE>(gate_kind);
  return cut ? gate_norm_grad_of<false, GRAD_CUT>(gate_kind) : gate_norm_grad_of<false, GRAD_WHOLE>(gate_kind);
}

}  // namespace sptg
