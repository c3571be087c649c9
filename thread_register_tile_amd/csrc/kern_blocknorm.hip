// kern_blocknorm.hip -- instances of the block norm's forward kernel and of the
// kernel that adds the backward pass's sums, and the rules that pick the
// shapes.
#include "blocknorm.hpp"
#include "blocknorm_shape.hpp"
#include "blockparams.hpp"
#include "launch.hpp"

namespace trt {

namespace {

template <class F>
hipError_t with_type(int dt, F&& f) {
  if (dt == DT_F16) return f.template operator()<DT_F16>();
  if (dt == DT_BF16) return f.template operator()<DT_BF16>();
  return f.template operator()<DT_F32>();
}

}  // namespace

BlockCut block_norm_cut(int64_t rows, int64_t cols, int64_t span, int dt) {
  const int64_t groups = (rows + span - 1) / span;
  return {groups, block_slices(rows, span, groups, block_chunks(cols, dt))};
}

hipError_t launch_block_norm(BlockNormArgs a, int dt, hipStream_t s) {
  // a gate row of few rows is read with each of them: as workgroups of their own
  // they would start for a few turns only
  const bool each = a.gate && (a.span <= 8 || a.rows / a.span >= 1 << 20);
  const int64_t span = each ? a.rows : a.span, groups = (a.rows + span - 1) / span;
  return with_type(dt, [&]<int DT>() {
    return with_forward_shape(block_chunks(a.cols, DT), [&]<int W, int K>() {
      a.slices = (int32_t)forward_slices<W, K>(span, groups);
      const dim3 grid(groups * a.slices), block(NormShape<W>::THREADS);
      auto run = [&]<bool TINY>() {
        if (each) return launch(block_norm_kernel<DT, W, K, true, TINY>, grid, block, 0, s, a);
        return launch(block_norm_kernel<DT, W, K, false, TINY>, grid, block, 0, s, a);
      };
      if constexpr (W == 1 && K == 1)
        if (a.cols < RowChunk<DT>::VEC) return run.template operator()<true>();
      return run.template operator()<false>();
    });
  });
}

hipError_t launch_block_norm_bwd(const BlockNormArgs& a, const BlockParamsArgs& q, int dt, hipStream_t s) {
  const int64_t groups = q.groups;
  const bool bytes = a.y.scale != nullptr;
  hipError_t e;
  if (dt == DT_F16) e = bytes ? launch_block_norm_rows<DT_F16, true>(a, groups, s) : launch_block_norm_rows<DT_F16, false>(a, groups, s);
  else if (dt == DT_BF16) e = bytes ? launch_block_norm_rows<DT_BF16, true>(a, groups, s) : launch_block_norm_rows<DT_BF16, false>(a, groups, s);
  else e = bytes ? launch_block_norm_rows<DT_F32, true>(a, groups, s) : launch_block_norm_rows<DT_F32, false>(a, groups, s);
  if (e != hipSuccess || !a.part) return e;
  // gate rows: a workgroup's 16 waves take one each, or share one of many slices
  int64_t gates = 0;
  if (q.dgate) gates = q.slices >= kBlockParamsWaves ? groups : (groups + kBlockParamsWaves - 1) / kBlockParamsWaves;
  return launch(block_params_kernel, dim3((q.cols + 63) / 64, 4 + (gates < 4096 ? gates : 4096)),
                dim3(64 * kBlockParamsWaves), 0, s, q);
}

}  // namespace trt
