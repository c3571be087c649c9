// trt_norm.hip -- the layer norm's entry points: argument checks and launches.
// Declarations and contracts are in include/trt.h.
#include <cmath>

#include "buffers.hpp"
#include "norm.hpp"

namespace {

using trt::Buf;
using trt::check_buffers;
using trt::fail;

trt_status check_sizes(int64_t rows, int64_t cols, float eps, int32_t dtype, int32_t param_dtype) {
  if (rows < 1 || cols < 1 || rows > trt::kMaxDim || cols > trt::kMaxDim)
    return fail(TRT_ERR_SIZE, "rows and cols must be in [1, 2^30]");
  if (dtype != TRT_F16 && dtype != TRT_BF16 && dtype != TRT_F32)
    return fail(TRT_ERR_DTYPE, "dtype must be TRT_F16, TRT_BF16 or TRT_F32");
  if (param_dtype != dtype && param_dtype != TRT_F32)
    return fail(TRT_ERR_DTYPE, "param_dtype must be dtype or TRT_F32");
  if (!(eps >= 0.f) || std::isinf(eps)) return fail(TRT_ERR_ARG, "eps must be finite and not negative");
  if (cols * trt::elem_bytes(dtype) > trt::kNormMaxRowBytes)
    return fail(TRT_ERR_UNSUPPORTED, "a row must not exceed 65536 bytes");
  return TRT_OK;
}

int64_t bwd_workspace(int64_t rows, int64_t cols, int32_t dtype) {
  return (int64_t)trt::norm_slices(rows, cols, dtype) * 2 * cols * 4;
}

}  // namespace

extern "C" {

trt_status trt_layernorm(int64_t rows, int64_t cols, const void* x, int64_t ldx,
                         const void* gamma, const void* beta, float eps, void* y, int64_t ldy,
                         int32_t dtype, int32_t param_dtype, void* stream) {
  if (const trt_status s = check_sizes(rows, cols, eps, dtype, param_dtype); s != TRT_OK) return s;
  if (!x || !y) return fail(TRT_ERR_NULL, "x and y must be non-null");
  const int64_t e = trt::elem_bytes(dtype), pe = trt::elem_bytes(param_dtype);
  const Buf bufs[] = {{"y", y, rows, cols, ldy, e},
                      {"x", x, rows, cols, ldx, e},
                      {"gamma", gamma, 1, cols, cols, pe},
                      {"beta", beta, 1, cols, cols, pe}};
  if (const trt_status s = check_buffers(bufs, 1); s != TRT_OK) return s;
  trt::NormArgs a{};
  a.x = x;
  a.gamma = gamma;
  a.beta = beta;
  a.out = y;
  a.ldx = ldx;
  a.ldo = ldy;
  a.rows = (int32_t)rows;
  a.cols = (int32_t)cols;
  a.eps = eps;
  return trt::launched(trt::launch_layernorm(a, dtype, param_dtype, static_cast<hipStream_t>(stream)),
                       "layer norm launch");
}

int64_t trt_layernorm_bwd_workspace_size(int64_t rows, int64_t cols, int32_t dtype) {
  if (check_sizes(rows, cols, 0.f, dtype, dtype) != TRT_OK) return -1;
  trt::g_err.clear();
  return bwd_workspace(rows, cols, dtype);
}

trt_status trt_layernorm_bwd(int64_t rows, int64_t cols, const void* dy, int64_t lddy,
                             const void* x, int64_t ldx, const void* gamma, float eps, void* dx,
                             int64_t lddx, void* dgamma, void* dbeta, int32_t dtype,
                             int32_t param_dtype, void* workspace, int64_t workspace_bytes,
                             void* stream) {
  if (const trt_status s = check_sizes(rows, cols, eps, dtype, param_dtype); s != TRT_OK) return s;
  if (!dy || !x || !dx) return fail(TRT_ERR_NULL, "dy, x and dx must be non-null");
  const bool params = dgamma || dbeta;
  const int64_t need = params ? bwd_workspace(rows, cols, dtype) : 0;
  if (params) {
    if (const trt_status s = trt::check_workspace(workspace, workspace_bytes, need); s != TRT_OK) return s;
  }
  const int64_t e = trt::elem_bytes(dtype), pe = trt::elem_bytes(param_dtype);
  const Buf bufs[] = {{"dx", dx, rows, cols, lddx, e},
                      {"dgamma", dgamma, 1, cols, cols, pe},
                      {"dbeta", dbeta, 1, cols, cols, pe},
                      {"the workspace", params ? workspace : nullptr, 1, need, need, 1},
                      {"dy", dy, rows, cols, lddy, e},
                      {"x", x, rows, cols, ldx, e},
                      {"gamma", gamma, 1, cols, cols, pe}};
  if (const trt_status s = check_buffers(bufs, 4); s != TRT_OK) return s;
  trt::NormArgs a{};
  a.x = x;
  a.dy = dy;
  a.gamma = gamma;
  a.out = dx;
  a.part = params ? static_cast<float*>(workspace) : nullptr;
  a.ldx = ldx;
  a.lddy = lddy;
  a.ldo = lddx;
  a.rows = (int32_t)rows;
  a.cols = (int32_t)cols;
  a.eps = eps;
  return trt::launched(trt::launch_layernorm_bwd(a, dgamma, dbeta, dtype, param_dtype,
                                                 static_cast<hipStream_t>(stream)),
                       "layer norm gradient launch");
}

}  // extern "C"
