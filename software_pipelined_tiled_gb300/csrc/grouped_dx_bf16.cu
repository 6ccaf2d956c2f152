// grouped_dx_bf16.cu -- grouped products, mode DX, bf16 operands.
#include "grouped_gemm.cuh"
#include "variants.h"

namespace sptg {

KernelVariant grouped_variant_dx_bf16(int out_kind, int tt) {
  return grouped_variant_of<GROUPED_DX, true, OUT_BF16>(out_kind, tt);
}

}  // namespace sptg
