// kern_xent_grad.hip -- one of the cross entropy's products, in a translation
// unit of its own.
#include "kern_xent_launch.hpp"

namespace trt {

hipError_t launch_xent_grad(XentGradArgs a, int dt, bool wide, bool pipelined, hipStream_t s) {
  return launch_xent_product<XentGrad, true, true>(a, dt, wide, pipelined, 0, s);
}

}  // namespace trt
