// kern_blocknorm_bwd_f16.hip -- the block norm's backward kernel for one type of rows,
// in a translation unit of its own.
#include "kern_blocknorm_bwd.hpp"

namespace trt {

template hipError_t launch_block_norm_rows<DT_F16, false>(const BlockNormArgs&, int64_t, hipStream_t);

}  // namespace trt
