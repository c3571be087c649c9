// kern_xent_weight.hip -- one of the cross entropy's products, in a translation
// unit of its own.
#include "kern_xent_launch.hpp"

namespace trt {

hipError_t launch_xent_weight(XentWeightArgs a, int dt, bool wide, bool pipelined, hipStream_t s) {
  return launch_xent_product<XentWeight, false, false>(a, dt, wide, pipelined, 0, s);
}

}  // namespace trt
