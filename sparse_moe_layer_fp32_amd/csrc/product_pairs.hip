// Both gradients of a map in one launch.

#include "product_blocks.h"

namespace moe {

namespace {

// Both gradients in one launch: blocks 0 .. first - 1 form x's product, the
// others w's, so that the two fill the GPU together where neither does alone
// and only one launch ends with idle CUs.
template <class TX, class TW, bool GATHER>
__global__ __launch_bounds__(TX::THREADS, 2) void gradients_kernel(ProductArgs x, ProductArgs w,
                                                                   int first) {
  static_assert(TX::THREADS == TW::THREADS, "one block size");
  constexpr int RING = TX::RING > TW::RING ? TX::RING : TW::RING;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[RING];
  const int bid = blockIdx.x;
  if (bid < first)
    run_block<kInputGrad, TX, false>(x, bid, smem);
  else
    run_block<kWeightGrad, TW, GATHER>(w, bid - first, smem);
}

template <class TX, class TW>
hipError_t launch_both(ProductArgs x, ProductArgs w, hipStream_t stream) {
  const unsigned first = grid_of<kInputGrad, TX>(&x), more = grid_of<kWeightGrad, TW>(&w);
  if (first + more == 0) return hipSuccess;
  if (w.src && w.y)
    gradients_kernel<TX, TW, true><<<first + more, TX::THREADS, 0, stream>>>(x, w, first);
  else
    gradients_kernel<TX, TW, false><<<first + more, TX::THREADS, 0, stream>>>(x, w, first);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_grad_pair(const ProductArgs& x, int sx, const ProductArgs& w, int sw,
                            hipStream_t stream) {
  if (sx == kShapeSmall) return launch_both<Small<kInputGrad>, Small<kWeightGrad>>(x, w, stream);
  if (sx == kShapeBig)
    return sw == kShapeBig ? launch_both<Big<kInputGrad>, Big<kWeightGrad>>(x, w, stream)
                           : launch_both<Big<kInputGrad>, Half<kWeightGrad>>(x, w, stream);
  return sw == kShapeBig ? launch_both<Half<kInputGrad>, Big<kWeightGrad>>(x, w, stream)
                         : launch_both<Half<kInputGrad>, Half<kWeightGrad>>(x, w, stream);
}

}  // namespace moe
