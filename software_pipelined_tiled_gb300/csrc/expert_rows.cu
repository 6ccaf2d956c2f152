// expert_rows.cu -- instantiations of the kernels that dispatch rows to experts
// and combine their outputs.
#include "expert_rows.cuh"
#include "variants.h"

namespace sptg {

const void* dispatch_sort_variant() { return reinterpret_cast<const void*>(&dispatch_sort_kernel<SORT_WARPS>); }

const void* dispatch_copy_variant(bool vectors) {
  return vectors ? reinterpret_cast<const void*>(&dispatch_copy_kernel<8>)
                 : reinterpret_cast<const void*>(&dispatch_copy_kernel<1>);
}

const void* combine_rows_variant(bool bf16, bool vectors) {
  if (bf16)
    return vectors ? reinterpret_cast<const void*>(&combine_rows_kernel<true, 8>)
                   : reinterpret_cast<const void*>(&combine_rows_kernel<true, 1>);
  return vectors ? reinterpret_cast<const void*>(&combine_rows_kernel<false, 8>)
                 : reinterpret_cast<const void*>(&combine_rows_kernel<false, 1>);
}

const void* combine_rows_grad_variant(bool bf16, bool vectors) {
  if (bf16)
    return vectors ? reinterpret_cast<const void*>(&combine_rows_grad_kernel<true, 8>)
                   : reinterpret_cast<const void*>(&combine_rows_grad_kernel<true, 1>);
  return vectors ? reinterpret_cast<const void*>(&combine_rows_grad_kernel<false, 8>)
                 : reinterpret_cast<const void*>(&combine_rows_grad_kernel<false, 1>);
}

}  // namespace sptg
