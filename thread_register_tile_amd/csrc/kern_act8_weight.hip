// kern_act8_weight.hip -- the product of the weight gradient from 8-bit rows, in
// a translation unit of its own.
#include "act8_weight.hpp"
#include "gemm_wide.hpp"
#include "launch.hpp"
#include "tiles.hpp"

namespace trt {

namespace {

template <class TL, class F>
hipError_t with_tile(Act8WeightArgs a, int64_t slices, F&& f) {
  a.tiles_m = (a.M + TL::BM - 1) / TL::BM;
  a.tiles_n = (a.N + TL::BN - 1) / TL::BN;
  return f(a, dim3(a.tiles_m * a.tiles_n, slices), dim3(TL::THREADS));
}

}  // namespace

hipError_t launch_act8_weight(Act8WeightArgs a, int dt, bool wide, int64_t slices, hipStream_t s) {
  if (wide)
    return with_tile<Tile256F>(a, slices, [&](const Act8WeightArgs& a, dim3 grid, dim3 block) {
      using EPI = Act8Weight<Tile256F, true>;
      if (dt == DT_F16) return launch(gemm_wide_kernel<Tile256F, DT_F16, false, false, EPI>, grid, block, 0, s, a);
      return launch(gemm_wide_kernel<Tile256F, DT_BF16, false, false, EPI>, grid, block, 0, s, a);
    });
  return with_tile<Tile128D>(a, slices, [&](const Act8WeightArgs& a, dim3 grid, dim3 block) {
    using EPI = Act8Weight<Tile128D, true>;
    if (dt == DT_F16) return launch(gemm_dma_kernel<Tile128D, DT_F16, false, false, 4, EPI>, grid, block, 0, s, a);
    return launch(gemm_dma_kernel<Tile128D, DT_BF16, false, false, 4, EPI>, grid, block, 0, s, a);
  });
}

}  // namespace trt
