// kern_xent_input.hip -- one of the cross entropy's products, in a translation
// unit of its own.
#include "kern_xent_launch.hpp"

namespace trt {

hipError_t launch_xent_input(XentInputArgs a, int dt, bool wide, bool pipelined, int64_t groups,
                             hipStream_t s) {
  return launch_xent_product<XentInput, true, false>(a, dt, wide, pipelined, groups, s);
}

}  // namespace trt
