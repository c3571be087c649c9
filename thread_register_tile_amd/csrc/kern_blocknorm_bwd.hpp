// kern_blocknorm_bwd.hpp -- launches of the block norm's backward kernel over
// the rows, included only by the kern_blocknorm_bwd_*.hip units, one type each.
#pragma once

#include "blocknorm.hpp"
#include "blocknorm_shape.hpp"
#include "launch.hpp"

namespace trt {

template <int DT>
hipError_t launch_block_norm_rows(const BlockNormArgs& a, int64_t groups, hipStream_t s) {
  return with_block_shape(block_chunks(a.cols, DT), [&]<int W, int K>() {
    constexpr int MANY = kBlockWaves<W>, FEW = kBlockFewWaves<W>;
    const dim3 grid(groups * a.slices);
    if (block_large<W>(a.rows))
      return a.rms ? launch(block_norm_bwd_kernel<DT, W, K, MANY, true>, grid, dim3(64 * MANY), 0, s, a)
                   : launch(block_norm_bwd_kernel<DT, W, K, MANY, false>, grid, dim3(64 * MANY), 0, s, a);
    return a.rms ? launch(block_norm_bwd_kernel<DT, W, K, FEW, true>, grid, dim3(64 * FEW), 0, s, a)
                 : launch(block_norm_bwd_kernel<DT, W, K, FEW, false>, grid, dim3(64 * FEW), 0, s, a);
  });
}

}  // namespace trt
