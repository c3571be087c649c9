// kern_xent_launch.hpp -- the launchers of the cross entropy's products,
// included only by the kern_xent*.hip units, one product each.
#pragma once

#include "gemm_wide.hpp"
#include "launch.hpp"
#include "tiles.hpp"
#include "xent.hpp"

namespace trt {

// EPI_OF<tile, pipelined>: the product's epilogue.  groups: workgroups, or 0 for
// one to a tile.
template <template <class, bool> class EPI_OF, class TL, bool A_KC, bool B_KC, class Args>
hipError_t launch_xent_tile(Args a, int dt, int64_t groups, hipStream_t s) {
  using EPI = EPI_OF<TL, true>;
  a.tiles_m = (a.M + TL::BM - 1) / TL::BM;
  a.tiles_n = (a.N + TL::BN - 1) / TL::BN;
  const dim3 grid(groups ? groups : a.tiles_m * a.tiles_n), block(TL::THREADS);
  if constexpr (TL::BM == 256) {
    // one workgroup per compute unit walks the tiles, or one per tile
    const int tiles = a.tiles_m * a.tiles_n;
    const dim3 grid(EPI::STREAMS && tiles > kWideUnits ? kWideUnits : groups ? groups : tiles);
    if (dt == DT_F16) return launch(gemm_wide_kernel<TL, DT_F16, A_KC, B_KC, EPI>, grid, block, 0, s, a);
    return launch(gemm_wide_kernel<TL, DT_BF16, A_KC, B_KC, EPI>, grid, block, 0, s, a);
  } else {
    if (dt == DT_F16) return launch(gemm_dma_kernel<TL, DT_F16, A_KC, B_KC, 4, EPI>, grid, block, 0, s, a);
    return launch(gemm_dma_kernel<TL, DT_BF16, A_KC, B_KC, 4, EPI>, grid, block, 0, s, a);
  }
}

template <template <class, bool> class EPI_OF, bool A_KC, bool B_KC, class Args>
hipError_t launch_xent_product(Args a, int dt, bool wide, bool pipelined, int64_t groups, hipStream_t s) {
  if (pipelined)
    return wide ? launch_xent_tile<EPI_OF, Tile256F, A_KC, B_KC>(a, dt, groups, s)
                : launch_xent_tile<EPI_OF, Tile128D, A_KC, B_KC>(a, dt, groups, s);
  using EPI = EPI_OF<Tile128, false>;
  a.tiles_m = (a.M + Tile128::BM - 1) / Tile128::BM;
  a.tiles_n = (a.N + Tile128::BN - 1) / Tile128::BN;
  const dim3 grid(groups ? groups : a.tiles_m * a.tiles_n), block(Tile128::THREADS);
  if (dt == DT_F16) return launch(gemm_kernel<Tile128, DT_F16, A_KC, B_KC, false, EPI>, grid, block, 0, s, a);
  return launch(gemm_kernel<Tile128, DT_BF16, A_KC, B_KC, false, EPI>, grid, block, 0, s, a);
}

}  // namespace trt
