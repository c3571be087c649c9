// kern_layernorm.hip -- instances of the layer norm kernels and the rule that
// picks one from a row's length.
#include "launch.hpp"
#include "layernorm.hpp"
#include "norm.hpp"

namespace trt {

namespace {

// Waves per row W and 16-byte chunks per lane K for a row of `chunks` chunks.
// A row of up to 128 chunks (1024 16-bit elements) is one wave's: no barrier,
// several rows to a workgroup.  Longer rows take 4, 8 and 16 waves, so that a
// lane holds few chunks.  The backward pass keeps two running sums per element
// of them in registers: it stays at 8 waves, whose lanes have 256 (1000 rows of
// 8200 binary32 elements: 78 us in 16 waves of 128 registers, 33 in 8), and
// with as many gives a wave rows of up to 256 chunks (8192 rows of 2048 bf16
// elements: 30.5 us in four waves a row, 25 in one; 64000 rows 181 and 148).
struct Shape {
  int w, k;
};
constexpr Shape shape_of(int64_t chunks, bool backward) {
  if (chunks <= 64) return {1, 1};
  if (chunks <= 128) return {1, 2};
  if (backward && chunks <= 256) return {1, chunks <= 192 ? 3 : 4};
  if (chunks <= 256) return {4, 1};
  if (chunks <= 512) return {4, 2};
  if (chunks <= 768 && !backward) return {4, 3};
  if (chunks <= 1024) return {8, 2};
  if (!backward) return chunks <= 2048 ? Shape{16, 2} : Shape{16, 4};
  return {8, chunks <= 4 * 512 ? 4 : chunks <= 6 * 512 ? 6 : 8};
}
static_assert(kNormMaxRowBytes / 16 == 16 * 64 * 4, "the longest row is one workgroup's");

// Workgroups: at most `most` a compute unit (256 of them), each with the same
// number of turns over its rows but for the last.
int grid_of(int64_t rows, int groups, int most) {
  const int64_t need = (rows + groups - 1) / groups;
  const int64_t turns = (need + 256 * most - 1) / (256 * most);
  return (int)((need + turns - 1) / turns);
}

// Forward workgroups to a compute unit, 16 waves in all (measured on 16384
// rows of 8192 16-bit elements: 93 us, against 106 with twice as many), but
// for one-wave rows, whose short loads want 32 (65536 rows of 512: 26.7 us,
// against 28.7 with 16).  Backward: one, of 16 or 8 waves (kBwdWaves).
template <int W>
constexpr int forward_most() { return W == 1 ? 8 : 16 / W; }

template <int DT, bool BACKWARD, class F>
auto with_shape(int64_t cols, F&& f) {
  const Shape s = shape_of((cols + RowChunk<DT>::VEC - 1) / RowChunk<DT>::VEC, BACKWARD);
  if constexpr (BACKWARD) {
    if (s.w == 1 && s.k == 3) return f.template operator()<1, 3>();
    if (s.w == 1 && s.k == 4) return f.template operator()<1, 4>();
  }
  if (s.w == 1) return s.k == 1 ? f.template operator()<1, 1>() : f.template operator()<1, 2>();
  if (s.w == 4) {
    if constexpr (!BACKWARD) {
      if (s.k == 1) return f.template operator()<4, 1>();
      if (s.k == 3) return f.template operator()<4, 3>();
    }
    return f.template operator()<4, 2>();
  }
  if constexpr (BACKWARD) {
    if (s.k == 2) return f.template operator()<8, 2>();
    if (s.k == 4) return f.template operator()<8, 4>();
    return s.k == 6 ? f.template operator()<8, 6>() : f.template operator()<8, 8>();
  } else {
    if (s.w == 8) return f.template operator()<8, 2>();
    return s.k == 2 ? f.template operator()<16, 2>() : f.template operator()<16, 4>();
  }
}

// Waves of a backward workgroup: 16, or 8 where a lane holds three chunks and
// more, if such workgroups fill the 256 units; else as the forward pass has them.
template <int W, int K>
constexpr int kBwdWaves = K >= 3 ? 8 : 16;
template <int W, int K>
bool bwd_large(int64_t rows) {
  return (rows + kBwdWaves<W, K> / W - 1) / (kBwdWaves<W, K> / W) >= 256;
}
template <int W>
constexpr int kBwdFewWaves = W == 1 ? 4 : W;

template <class F>
hipError_t with_types(int dt, int pdt, F&& f) {
  if (dt == DT_F32) return f.template operator()<DT_F32, DT_F32>();
  if (dt == DT_F16)
    return pdt == DT_F32 ? f.template operator()<DT_F16, DT_F32>() : f.template operator()<DT_F16, DT_F16>();
  return pdt == DT_F32 ? f.template operator()<DT_BF16, DT_F32>() : f.template operator()<DT_BF16, DT_BF16>();
}

template <int DT>
int slices_of(int64_t rows, int64_t cols) {
  return with_shape<DT, true>(cols, [&]<int W, int K>() {
    return grid_of(rows, (bwd_large<W, K>(rows) ? kBwdWaves<W, K> : kBwdFewWaves<W>) / W, 1);
  });
}

}  // namespace

int norm_slices(int64_t rows, int64_t cols, int dt) {
  return dt == DT_F32 ? slices_of<DT_F32>(rows, cols) : slices_of<DT_F16>(rows, cols);
}

hipError_t launch_layernorm(const NormArgs& a, int dt, int pdt, hipStream_t s) {
  return with_types(dt, pdt, [&]<int DT, int PDT>() {
    return with_shape<DT, false>(a.cols, [&]<int W, int K>() {
      const int wgs = grid_of(a.rows, NormShape<W>::GROUPS, forward_most<W>());
      return launch(layernorm_kernel<DT, PDT, W, K>, dim3(wgs), dim3(NormShape<W>::THREADS), 0, s, a);
    });
  });
}

hipError_t launch_layernorm_bwd(const NormArgs& a, void* dgamma, void* dbeta, int dt, int pdt,
                                hipStream_t s) {
  const int slices = norm_slices(a.rows, a.cols, dt);
  return with_types(dt, pdt, [&]<int DT, int PDT>() {
    const hipError_t e = with_shape<DT, true>(a.cols, [&]<int W, int K>() {
      constexpr int MANY = kBwdWaves<W, K>, FEW = kBwdFewWaves<W>;
      if (bwd_large<W, K>(a.rows))
        return launch(layernorm_bwd_kernel<DT, PDT, W, K, MANY>, dim3(slices), dim3(64 * MANY), 0, s, a);
      return launch(layernorm_bwd_kernel<DT, PDT, W, K, FEW>, dim3(slices), dim3(64 * FEW), 0, s, a);
    });
    if (e != hipSuccess || !a.part) return e;
    const NormParamsArgs q{a.part, dgamma, dbeta, slices, a.cols};
    return launch(norm_params_kernel<PDT>, dim3((a.cols + 63) / 64, 2), dim3(64 * kNormParamsWaves), 0, s, q);
  });
}

}  // namespace trt
