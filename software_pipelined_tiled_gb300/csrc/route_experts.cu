// route_experts.cu -- instantiations of the router's kernels.
#include "route_experts.cuh"
#include "variants.h"

namespace sptg {

template <int TYPE>
const void* route_variant_of(int kind) {
  switch (kind) {
    case ROUTE_8_8: return reinterpret_cast<const void*>(&route_experts_kernel<TYPE, 8, 8>);
    case ROUTE_16_8: return reinterpret_cast<const void*>(&route_experts_kernel<TYPE, 16, 8>);
    case ROUTE_32_8: return reinterpret_cast<const void*>(&route_experts_kernel<TYPE, 32, 8>);
    case ROUTE_8_16: return reinterpret_cast<const void*>(&route_experts_kernel<TYPE, 8, 16>);
    case ROUTE_32_16: return reinterpret_cast<const void*>(&route_experts_kernel<TYPE, 32, 16>);
    case ROUTE_32_32: return reinterpret_cast<const void*>(&route_experts_kernel<TYPE, 32, 32>);
    default: return reinterpret_cast<const void*>(&route_experts_kernel<TYPE, 32, 64>);
  }
}

const void* route_variant(int type, int kind) {
  return type == ROUTE_F32    ? route_variant_of<ROUTE_F32>(kind)
         : type == ROUTE_BF16 ? route_variant_of<ROUTE_BF16>(kind)
                              : route_variant_of<ROUTE_F16>(kind);
}

template <int SLOTS>
const void* route_dlogits_of(int type) {
  return type == ROUTE_F32    ? reinterpret_cast<const void*>(&route_experts_dlogits_kernel<ROUTE_F32, SLOTS>)
         : type == ROUTE_BF16 ? reinterpret_cast<const void*>(&route_experts_dlogits_kernel<ROUTE_BF16, SLOTS>)
                              : reinterpret_cast<const void*>(&route_experts_dlogits_kernel<ROUTE_F16, SLOTS>);
}

const void* route_dlogits_variant(int type, int slots) {
  return slots == 8 ? route_dlogits_of<8>(type) : route_dlogits_of<16>(type);
}

}  // namespace sptg
