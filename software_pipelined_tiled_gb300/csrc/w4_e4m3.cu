// w4_e4m3.cu -- the 4-bit-weight product for rows of x in e4m3.
#include "w4_gemm.cuh"
#include "variants.h"

namespace sptg {

const void* w4_kernel_e4m3(int nt, int group) { return w4_kernel_of<W4_E4M3>(nt, group); }

}  // namespace sptg
