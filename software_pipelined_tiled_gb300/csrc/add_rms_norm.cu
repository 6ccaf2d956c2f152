// add_rms_norm.cu -- instantiations of the residual-addition and norm kernels.
#include "add_rms_norm.cuh"
#include "variants.h"

namespace sptg {

template <bool BF16, int OUTK>
NormVariant norm_variant_of(int cols, bool vectors) {
  if (!vectors || cols > 32768)
    return {reinterpret_cast<const void*>(&add_rms_norm_any_kernel<BF16, OUTK>), 512, 1};
  if (cols <= 1024)
    return {reinterpret_cast<const void*>(&add_rms_norm_kernel<BF16, OUTK, 32, 128, 4>), 128, 4};
  if (cols <= 4096)
    return {reinterpret_cast<const void*>(&add_rms_norm_kernel<BF16, OUTK, 128, 128, 4>), 128, 1};
  if (cols <= 8192)
    return {reinterpret_cast<const void*>(&add_rms_norm_kernel<BF16, OUTK, 256, 256, 4>), 256, 1};
  if (cols <= 16384)
    return {reinterpret_cast<const void*>(&add_rms_norm_kernel<BF16, OUTK, 512, 512, 4>), 512, 1};
  return {reinterpret_cast<const void*>(&add_rms_norm_kernel<BF16, OUTK, 1024, 1024, 4>), 1024, 1};
}

NormVariant norm_variant(bool bf16, int out_kind, int cols, bool vectors) {
  switch (out_kind) {
    case NORM_S8:
      return bf16 ? norm_variant_of<true, NORM_S8>(cols, vectors)
                  : norm_variant_of<false, NORM_S8>(cols, vectors);
    case NORM_E4M3:
      return bf16 ? norm_variant_of<true, NORM_E4M3>(cols, vectors)
                  : norm_variant_of<false, NORM_E4M3>(cols, vectors);
    default:
      return bf16 ? norm_variant_of<true, NORM_16>(cols, vectors)
                  : norm_variant_of<false, NORM_16>(cols, vectors);
  }
}

}  // namespace sptg
