// add_rms_norm.cu -- instantiations of the residual-addition and norm kernels.
#include "add_rms_norm.cuh"
#include "variants.h"

namespace sptg {

template <bool BF16, int OUTK>
const void* norm_variant_of(int kind) {
  switch (kind) {
    case NORM_WARP_2: return reinterpret_cast<const void*>(&add_rms_norm_kernel<BF16, OUTK, true, 2>);
    case NORM_WARP_4: return reinterpret_cast<const void*>(&add_rms_norm_kernel<BF16, OUTK, true, 4>);
    case NORM_BLOCK_2: return reinterpret_cast<const void*>(&add_rms_norm_kernel<BF16, OUTK, false, 2>);
    case NORM_BLOCK_4: return reinterpret_cast<const void*>(&add_rms_norm_kernel<BF16, OUTK, false, 4>);
    case NORM_RING_4: return reinterpret_cast<const void*>(&add_rms_norm_ring_kernel<BF16, OUTK, 4, 512>);
    default: return reinterpret_cast<const void*>(&add_rms_norm_any_kernel<BF16, OUTK>);
  }
}

const void* norm_variant(bool bf16, int out_kind, int kind) {
  switch (out_kind) {
    case NORM_S8:
      return bf16 ? norm_variant_of<true, NORM_S8>(kind) : norm_variant_of<false, NORM_S8>(kind);
    case NORM_E4M3:
      return bf16 ? norm_variant_of<true, NORM_E4M3>(kind) : norm_variant_of<false, NORM_E4M3>(kind);
    default:
      return bf16 ? norm_variant_of<true, NORM_16>(kind) : norm_variant_of<false, NORM_16>(kind);
  }
}

}  // namespace sptg
