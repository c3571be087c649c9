// kern_blocknorm_bwd.hpp -- launches of the block norm's backward kernel over
// the rows, included only by the kern_blocknorm_bwd_*.hip units, one type and form of the saved rows each.
#pragma once

#include "blocknorm.hpp"
#include "blocknorm_shape.hpp"
#include "launch.hpp"

namespace trt {

template <int DT, bool BYTES>
hipError_t launch_block_norm_rows(const BlockNormArgs& a, int64_t groups, hipStream_t s) {
  return with_block_shape(block_chunks(a.cols, DT), [&]<int W, int K>() {
    constexpr int MANY = kBlockWaves<W>, FEW = kBlockFewWaves<W>;
    const dim3 grid(groups * a.slices);
    auto run = [&]<int WAVES, bool TINY>() {
      const dim3 block(64 * WAVES);
      return a.rms ? launch(block_norm_bwd_kernel<DT, BYTES, W, K, WAVES, true, TINY>, grid, block, 0, s, a)
                   : launch(block_norm_bwd_kernel<DT, BYTES, W, K, WAVES, false, TINY>, grid, block, 0, s, a);
    };
    const bool large = block_large<W>(a.rows);
    if constexpr (W == 1 && K == 1)
      if (a.cols < RowChunk<DT>::VEC)
        return large ? run.template operator()<MANY, true>() : run.template operator()<FEW, true>();
    return large ? run.template operator()<MANY, false>() : run.template operator()<FEW, false>();
  });
}

}  // namespace trt
