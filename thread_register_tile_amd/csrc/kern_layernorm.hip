// kern_layernorm.hip -- instances of the layer norm kernels and the rule that
// picks one from a row's length.
#include "launch.hpp"
#include "layernorm.hpp"
#include "norm.hpp"

namespace trt {

namespace {

// Waves per row W and 16-byte chunks per lane K for a row of `chunks` chunks,
// the same for both directions.  A row of up to 128 chunks (1024 16-bit
// elements) is one wave's: no barrier, four rows to a workgroup.  Longer rows
// take 4, 8 and 16 waves, so that a lane holds no more than 2 chunks up to
// 2048 of them and 4 beyond: the backward pass keeps two running sums per
// element of them in registers.
struct Shape {
  int w, k;
};
constexpr Shape shape_of(int64_t chunks) {
  if (chunks <= 64) return {1, 1};
  if (chunks <= 128) return {1, 2};
  if (chunks <= 256) return {4, 1};
  if (chunks <= 512) return {4, 2};
  if (chunks <= 1024) return {8, 2};
  if (chunks <= 2048) return {16, 2};
  return {16, 4};
}
static_assert(kNormMaxRowBytes / 16 == 16 * 64 * 4, "the longest row is one workgroup's");

// Workgroups: at most `most` a compute unit (256 of them), each with the same
// number of turns over its rows but for the last.
int grid_of(int64_t rows, int groups, int most) {
  const int64_t need = (rows + groups - 1) / groups;
  const int64_t turns = (need + 256 * most - 1) / (256 * most);
  return (int)((need + turns - 1) / turns);
}

template <int W>
constexpr int forward_most() { return W <= 4 ? 8 : (W == 8 ? 4 : 2); }
template <int W>
constexpr int backward_most() { return W <= 4 ? 2 : 1; }

template <int DT, class F>
auto with_shape(int64_t cols, F&& f) {
  const Shape s = shape_of((cols + RowChunk<DT>::VEC - 1) / RowChunk<DT>::VEC);
  if (s.w == 1) return s.k == 1 ? f.template operator()<1, 1>() : f.template operator()<1, 2>();
  if (s.w == 4) return s.k == 1 ? f.template operator()<4, 1>() : f.template operator()<4, 2>();
  if (s.w == 8) return f.template operator()<8, 2>();
  return s.k == 2 ? f.template operator()<16, 2>() : f.template operator()<16, 4>();
}

template <class F>
hipError_t with_types(int dt, int pdt, F&& f) {
  if (dt == DT_F32) return f.template operator()<DT_F32, DT_F32>();
  if (dt == DT_F16)
    return pdt == DT_F32 ? f.template operator()<DT_F16, DT_F32>() : f.template operator()<DT_F16, DT_F16>();
  return pdt == DT_F32 ? f.template operator()<DT_BF16, DT_F32>() : f.template operator()<DT_BF16, DT_BF16>();
}

template <int DT>
int slices_of(int64_t rows, int64_t cols) {
  return with_shape<DT>(cols, [&]<int W, int K>() {
    return grid_of(rows, NormShape<W>::GROUPS, backward_most<W>());
  });
}

}  // namespace

int norm_slices(int64_t rows, int64_t cols, int dt) {
  return dt == DT_F32 ? slices_of<DT_F32>(rows, cols) : slices_of<DT_F16>(rows, cols);
}

hipError_t launch_layernorm(const NormArgs& a, int dt, int pdt, hipStream_t s) {
  return with_types(dt, pdt, [&]<int DT, int PDT>() {
    return with_shape<DT>(a.cols, [&]<int W, int K>() {
      const int wgs = grid_of(a.rows, NormShape<W>::GROUPS, forward_most<W>());
      return launch(layernorm_kernel<DT, PDT, W, K>, dim3(wgs), dim3(NormShape<W>::THREADS), 0, s, a);
    });
  });
}

hipError_t launch_layernorm_bwd(const NormArgs& a, void* dgamma, void* dbeta, int dt, int pdt,
                                hipStream_t s) {
  const int slices = norm_slices(a.rows, a.cols, dt);
  return with_types(dt, pdt, [&]<int DT, int PDT>() {
    const hipError_t e = with_shape<DT>(a.cols, [&]<int W, int K>() {
      return launch(layernorm_bwd_kernel<DT, PDT, W, K>, dim3(slices), dim3(NormShape<W>::THREADS), 0, s, a);
    });
    if (e != hipSuccess || !a.part) return e;
    const NormParamsArgs q{a.part, dgamma, dbeta, slices, a.cols};
    return launch(norm_params_kernel<PDT>, dim3((a.cols + 63) / 64, 2), dim3(64 * kNormParamsWaves), 0, s, q);
  });
}

}  // namespace trt
