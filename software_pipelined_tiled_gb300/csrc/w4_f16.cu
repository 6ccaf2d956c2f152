// w4_f16.cu -- the 4-bit-weight products for rows of x in f16.
#include "w4_gemm.cuh"
#include "w4_tile_gemm.cuh"
#include "variants.h"

namespace sptg {

const void* w4_kernel_f16(int group) { return w4_kernel_of<W4_F16>(group); }
const void* w4_tile_kernel_f16(int ntok, int group) { return w4_tile_kernel_of<W4_F16>(ntok, group); }

}  // namespace sptg
