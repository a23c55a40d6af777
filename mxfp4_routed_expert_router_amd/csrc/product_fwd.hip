// The forward form of the products through LDS tiles.
#include "product_lds.h"

namespace moe_fp4 {
namespace {

template <typename T>
void launch(const ProductArgs& a, hipStream_t stream) {
  switch (product_shape(a, kFwd)) {
    case kBig: return launch_shape<T, kFwd, Big>(a, stream);
    case kMid: return launch_shape<T, kFwd, Mid>(a, stream);
    default: return launch_shape<T, kFwd, Low>(a, stream);
  }
}

}  // namespace

void launch_product_fwd(const ProductArgs& a, hipStream_t stream) {
  if (a.type == kBf16)
    launch<Bf16>(a, stream);
  else
    launch<F16>(a, stream);
}

}  // namespace moe_fp4
