// w4_bf16.cu -- the 4-bit-weight products for rows of x in bf16.
#include "w4_gemm.cuh"
#include "w4_tile_gemm.cuh"
#include "variants.h"

namespace sptg {

const void* w4_kernel_bf16(int group) { return w4_kernel_of<W4_BF16>(group); }
const void* w4_tile_kernel_bf16(int ntok, int group) { return w4_tile_kernel_of<W4_BF16>(ntok, group); }

}  // namespace sptg
