// w4_e4m3.cu -- the 4-bit-weight products for rows of x in e4m3.
#include "w4_gemm.cuh"
#include "w4_tile_gemm.cuh"
#include "variants.h"

namespace sptg {

const void* w4_kernel_e4m3(int group) { return w4_kernel_of<W4_E4M3>(group); }
const void* w4_tile_kernel_e4m3(int ntok, int group) { return w4_tile_kernel_of<W4_E4M3>(ntok, group); }

}  // namespace sptg
