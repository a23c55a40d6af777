// The input gradient form of the products through LDS tiles.
#include "product_lds.h"

namespace moe_fp4 {
namespace {

template <typename T>
void launch(const ProductArgs& a, hipStream_t stream) {
  switch (product_shape(a, kDgrad)) {
    case kBig: return launch_shape<T, kDgrad, Big>(a, stream);
    case kMid: return launch_shape<T, kDgrad, Mid>(a, stream);
    default: return launch_shape<T, kDgrad, Low>(a, stream);
  }
}

}  // namespace

void launch_product_dgrad(const ProductArgs& a, hipStream_t stream) {
  if (a.type == kBf16)
    launch<Bf16>(a, stream);
  else
    launch<F16>(a, stream);
}

}  // namespace moe_fp4
