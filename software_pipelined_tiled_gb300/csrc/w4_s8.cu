// w4_s8.cu -- the 4-bit-weight product for rows of x in s8.
#include "w4_gemm.cuh"
#include "variants.h"

namespace sptg {

const void* w4_kernel_s8(int nt, int group) { return w4_kernel_of<W4_S8>(nt, group); }

}  // namespace sptg
