// kern_blocknorm_bwd_bf16_8bit.hip -- the block norm's backward kernel for one type of rows, r' and y saved in 8 bits,
// in a translation unit of its own.
#include "kern_blocknorm_bwd.hpp"

namespace trt {

template hipError_t launch_block_norm_rows<DT_BF16, true>(const BlockNormArgs&, int64_t, hipStream_t);

}  // namespace trt
