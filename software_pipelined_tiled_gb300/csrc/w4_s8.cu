// w4_s8.cu -- the 4-bit-weight products for rows of x in s8.
#include "w4_gemm.cuh"
#include "w4_tile_gemm.cuh"
#include "variants.h"

namespace sptg {

const void* w4_kernel_s8(int group) { return w4_kernel_of<W4_S8>(group); }
const void* w4_tile_kernel_s8(int ntok, int group) { return w4_tile_kernel_of<W4_S8>(ntok, group); }

}  // namespace sptg
