// w4_bf16.cu -- the 4-bit-weight product for rows of x in bf16.
#include "w4_gemm.cuh"
#include "variants.h"

namespace sptg {

const void* w4_kernel_bf16(int nt, int group) { return w4_kernel_of<W4_BF16>(nt, group); }

}  // namespace sptg
