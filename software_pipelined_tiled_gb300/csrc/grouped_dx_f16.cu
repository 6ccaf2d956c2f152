// grouped_dx_f16.cu -- grouped products, mode DX, f16 operands.
#include "grouped_gemm.cuh"
#include "variants.h"

namespace sptg {

KernelVariant grouped_variant_dx_f16(int out_kind, int tt) {
  return grouped_variant_of<GROUPED_DX, false, OUT_F16>(out_kind, tt);
}

}  // namespace sptg
