// kern_xent.hip -- the cross entropy's small kernels.
#include "launch.hpp"
#include "xent_rows.hpp"
#include "xent_stream.hpp"

namespace trt {

hipError_t launch_xent_prep(const XentPrepArgs& a, hipStream_t s) {
  if (a.dloss) return launch(xent_prep_kernel<true>, dim3(1), dim3(kPrepThreads), 0, s, a);
  return launch(xent_prep_kernel<false>, dim3(1), dim3(kPrepThreads), 0, s, a);
}

hipError_t launch_xent_stream(const XentStatsArgs& a, int dt, hipStream_t s) {
  const dim3 grid((a.N + kXentStreamTile - 1) / kXentStreamTile);
  auto run = [&]<int T>() {
    const dim3 block(kXentStreamThreads);
    if (dt == DT_F16) return launch(xent_stream_kernel<DT_F16, T>, grid, block, 0, s, a);
    return launch(xent_stream_kernel<DT_BF16, T>, grid, block, 0, s, a);
  };
  if (a.M == 1) return run.template operator()<1>();
  if (a.M == 2) return run.template operator()<2>();
  return run.template operator()<4>();
}

// Rows to a workgroup: 64, so that a wave reads whole lines of a tile's
// pairs; fewer tokens take fewer, so that more threads share a row's tiles.
hipError_t launch_xent_combine(const XentCombineArgs& a, hipStream_t s) {
  auto run = [&]<int R>() {
    return launch(xent_combine_kernel<R>, dim3((a.tokens + R - 1) / R), dim3(256), 0, s, a);
  };
  if (a.tokens <= 4) return run.template operator()<1>();
  if (a.tokens <= 256) return run.template operator()<8>();
  return run.template operator()<64>();
}

hipError_t launch_xent_rows(const XentRowsArgs& a, int dt, hipStream_t s) {
  const dim3 grid(a.prep.tokens), block(256);
  if (dt == DT_F16) return launch(xent_rows_kernel<DT_F16>, grid, block, 0, s, a);
  return launch(xent_rows_kernel<DT_BF16>, grid, block, 0, s, a);
}

hipError_t launch_xent_input_finish(const XentInputFinishArgs& a, int64_t tokens, int odt,
                                    hipStream_t s) {
  // few tokens have many slices to add: a wave for 256 columns, so that their
  // reads spread over the units
  const bool few = tokens <= 512;
  const dim3 grid((unsigned)tokens, few ? (a.width + 255) / 256 : 1), block(few ? 64 : 256);
  if (odt == DT_F16) return launch(xent_input_finish_kernel<DT_F16>, grid, block, 0, s, a);
  if (odt == DT_BF16) return launch(xent_input_finish_kernel<DT_BF16>, grid, block, 0, s, a);
  return launch(xent_input_finish_kernel<DT_F32>, grid, block, 0, s, a);
}

}  // namespace trt
