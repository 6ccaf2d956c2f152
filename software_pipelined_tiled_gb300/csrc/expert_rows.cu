// expert_rows.cu -- instantiations of the kernels that dispatch rows to experts
// and combine their outputs.
#include "expert_rows.cuh"
#include "variants.h"

namespace sptg {

const void* dispatch_sort_variant() { return reinterpret_cast<const void*>(&dispatch_sort_kernel<SORT_WARPS>); }

const void* dispatch_copy_variant(bool aligned) {
  return aligned ? reinterpret_cast<const void*>(&dispatch_copy_kernel<true>)
                 : reinterpret_cast<const void*>(&dispatch_copy_kernel<false>);
}

const void* dispatch_small_variant(bool aligned) {
  return aligned ? reinterpret_cast<const void*>(&dispatch_small_kernel<true>)
                 : reinterpret_cast<const void*>(&dispatch_small_kernel<false>);
}

const void* combine_rows_variant(bool bf16, bool aligned) {
  if (bf16)
    return aligned ? reinterpret_cast<const void*>(&combine_rows_kernel<true, true>)
                   : reinterpret_cast<const void*>(&combine_rows_kernel<true, false>);
  return aligned ? reinterpret_cast<const void*>(&combine_rows_kernel<false, true>)
                 : reinterpret_cast<const void*>(&combine_rows_kernel<false, false>);
}

const void* combine_rows_grad_variant(bool bf16, bool aligned) {
  if (bf16)
    return aligned ? reinterpret_cast<const void*>(&combine_rows_grad_kernel<true>)
                   : reinterpret_cast<const void*>(&combine_rows_grad_cut_kernel<true>);
  return aligned ? reinterpret_cast<const void*>(&combine_rows_grad_kernel<false>)
                 : reinterpret_cast<const void*>(&combine_rows_grad_cut_kernel<false>);
}

}  // namespace sptg
