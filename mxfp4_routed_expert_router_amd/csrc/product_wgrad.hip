// The weight gradient form of the products through LDS tiles.
#include "product_lds.h"

namespace moe_fp4 {

void launch_product_wgrad(const ProductArgs& a, int shape, hipStream_t stream) {
  if (a.type == kBf16)
    launch_tiles<Bf16, kWgrad, 2>(a, shape, stream);
  else
    launch_tiles<F16, kWgrad, 2>(a, shape, stream);
}

}  // namespace moe_fp4
