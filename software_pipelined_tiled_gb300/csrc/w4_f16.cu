// w4_f16.cu -- the 4-bit-weight product for rows of x in f16.
#include "w4_gemm.cuh"
#include "variants.h"

namespace sptg {

const void* w4_kernel_f16(int nt, int group) { return w4_kernel_of<W4_F16>(nt, group); }

}  // namespace sptg
