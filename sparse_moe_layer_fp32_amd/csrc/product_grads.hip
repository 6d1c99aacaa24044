// The gradients' products: dx = dy W and dW = dy^T x.

#include "product_blocks.h"

namespace moe {

hipError_t launch_input_grad(const ProductArgs& p, int shape, hipStream_t stream) {
  return launch_op<kInputGrad>(p, shape, stream);
}

hipError_t launch_weight_grad(const ProductArgs& p, int shape, hipStream_t stream) {
  return launch_op<kWeightGrad>(p, shape, stream);
}

}  // namespace moe
