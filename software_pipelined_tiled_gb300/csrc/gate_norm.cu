// gate_norm.cu -- instantiations of the gated residual's and norms' kernels, forwards,
// and of the sums over blocks and the backward kernel for any row.
#include "gate_norm.cuh"
#include "variants.h"

namespace sptg {

template <bool BF16>
const void* gate_norm_variant_of(int kind) {
  switch (kind) {
    case GATE_NORM_1: return reinterpret_cast<const void*>(&gate_norm_kernel<BF16, 1, true>);
    case GATE_NORM_2: return reinterpret_cast<const void*>(&gate_norm_kernel<BF16, 2, true>);
    case GATE_NORM_RING: return reinterpret_cast<const void*>(&gate_norm_ring_kernel<BF16, 4>);
    case GATE_NORM_SHIFTED: return reinterpret_cast<const void*>(&gate_norm_kernel<BF16, 2, false>);
    default: return reinterpret_cast<const void*>(&gate_norm_any_kernel<BF16>);
  }
}

const void* gate_norm_variant(bool bf16, int kind) {
  return bf16 ? gate_norm_variant_of<true>(kind) : gate_norm_variant_of<false>(kind);
}

const void* gate_norm_grad_any_variant(bool bf16) {
  return bf16 ? reinterpret_cast<const void*>(&gate_norm_grad_any_kernel<true>)
              : reinterpret_cast<const void*>(&gate_norm_grad_any_kernel<false>);
}

const void* gate_norm_columns_variant(bool bf16) {
  return bf16 ? reinterpret_cast<const void*>(&gate_norm_columns_kernel<true, 32>)
              : reinterpret_cast<const void*>(&gate_norm_columns_kernel<false, 32>);
}

}  // namespace sptg
