// gate_norm.cu -- instantiations of the gated residual's and norms' kernels.
#include "gate_norm.cuh"
#include "variants.h"

namespace sptg {

template <bool BF16>
const void* gate_norm_variant_of(int kind) {
  switch (kind) {
    case GATE_NORM_1: return reinterpret_cast<const void*>(&gate_norm_kernel<BF16, 1>);
    case GATE_NORM_2: return reinterpret_cast<const void*>(&gate_norm_kernel<BF16, 2>);
    default: return reinterpret_cast<const void*>(&gate_norm_any_kernel<BF16>);
  }
}

template <bool BF16>
const void* gate_norm_grad_variant_of(int kind) {
  switch (kind) {
    case GATE_GRAD_512: return reinterpret_cast<const void*>(&gate_norm_grad_kernel<BF16, 1, 512>);
    case GATE_GRAD_1024: return reinterpret_cast<const void*>(&gate_norm_grad_kernel<BF16, 1, 1024>);
    case GATE_GRAD_2048: return reinterpret_cast<const void*>(&gate_norm_grad_kernel<BF16, 2, 1024>);
    default: return reinterpret_cast<const void*>(&gate_norm_grad_any_kernel<BF16>);
  }
}

const void* gate_norm_variant(bool bf16, int kind) {
  return bf16 ? gate_norm_variant_of<true>(kind) : gate_norm_variant_of<false>(kind);
}
const void* gate_norm_grad_variant(bool bf16, int kind) {
  return bf16 ? gate_norm_grad_variant_of<true>(kind) : gate_norm_grad_variant_of<false>(kind);
}
const void* gate_norm_columns_variant() { return reinterpret_cast<const void*>(&gate_norm_columns_kernel<32>); }

}  // namespace sptg
