// trt_blocknorm.hip -- the block norm's entry points: argument checks and
// launches.  Declarations and contracts are in include/trt.h.
#include <cmath>

#include "blocknorm_args.hpp"
#include "buffers.hpp"

namespace {

using trt::Buf;
using trt::fail;

trt_status check_sizes(int64_t rows, int64_t cols, int32_t dtype) {
  if (rows < 1 || cols < 1 || rows > trt::kMaxDim || cols > trt::kMaxDim)
    return fail(TRT_ERR_SIZE, "rows and cols must be in [1, 2^30]");
  if (dtype != TRT_F16 && dtype != TRT_BF16 && dtype != TRT_F32)
    return fail(TRT_ERR_DTYPE, "dtype must be TRT_F16, TRT_BF16 or TRT_F32");
  if (cols * trt::elem_bytes(dtype) > trt::kBlockMaxRowBytes)
    return fail(TRT_ERR_UNSUPPORTED, "a row must not exceed 32768 bytes");
  return TRT_OK;
}

trt_status check_block(const trt_block* b, int32_t dtype) {
  if (!b) return fail(TRT_ERR_NULL, "block must be non-null");
  if ((b->post != 0 && b->post != 1) || (b->rms != 0 && b->rms != 1))
    return fail(TRT_ERR_ARG, "post and rms must be 0 or 1");
  if (!(b->eps >= 0.f) || std::isinf(b->eps) || !std::isfinite(b->alpha))
    return fail(TRT_ERR_ARG, "alpha and eps must be finite, eps not negative");
  if (!b->post && (b->post_gamma || b->post_beta))
    return fail(TRT_ERR_ARG, "post_gamma and post_beta need the norm behind the block");
  if (b->param_dtype != dtype && b->param_dtype != TRT_F32)
    return fail(TRT_ERR_DTYPE, "param_dtype must be dtype or TRT_F32");
  if (!b->gate) return TRT_OK;
  if (b->gate_dtype != dtype && b->gate_dtype != TRT_F32)
    return fail(TRT_ERR_DTYPE, "gate_dtype must be dtype or TRT_F32");
  if (b->rows_per_gate < 1) return fail(TRT_ERR_SIZE, "rows_per_gate must be >= 1");
  return TRT_OK;
}

// Rows under one gate row, of those that there are.
int64_t span_of(int64_t rows, int64_t rows_per_gate) {
  return rows_per_gate < 1 || rows_per_gate > rows ? rows : rows_per_gate;
}

// How the backward pass is cut; a gate of its own for every row is no cut.
trt_status make_cut(int64_t rows, int64_t cols, int64_t rows_per_gate, int32_t dtype, trt::BlockCut& cut) {
  const int64_t span = span_of(rows, rows_per_gate);
  if (span > 1 && (rows + span - 1) / span >= int64_t(1) << 22)
    return fail(TRT_ERR_SIZE, "2^22 or more gate rows of several rows");
  cut = trt::block_norm_cut(rows, cols, span == 1 ? rows : span, dtype);
  return TRT_OK;
}

int64_t workspace_of(const trt::BlockCut& cut, int64_t cols) { return cut.groups * cut.slices * 16 * cols; }

trt::BlockNormArgs block_args(int64_t rows, int64_t cols, const trt_block& b, int32_t dtype) {
  trt::BlockNormArgs a{};
  a.gate = b.gate;
  a.post_gamma = b.post_gamma;
  a.post_beta = b.post_beta;
  a.gamma = b.gamma;
  a.beta = b.beta;
  a.ldg = b.ldg;
  a.span = (int32_t)span_of(rows, b.gate ? b.rows_per_gate : 0);
  a.rows = (int32_t)rows;
  a.cols = (int32_t)cols;
  a.alpha = b.alpha;
  a.eps = b.eps;
  a.rms = b.rms;
  a.post = b.post;
  a.wide_params = b.param_dtype != dtype;
  a.wide_gate = b.gate && b.gate_dtype != dtype;
  return a;
}

Buf saved_buf(const char* name, const trt_saved& s, int64_t rows, int64_t cols, int64_t e) {
  return {name, s.x, rows, cols, s.ld, s.scale ? 1 : e};
}
Buf scale_buf(const char* name, const trt_saved& s, int64_t rows, int64_t cols) {
  return {name, s.scale, rows, (cols + 31) / 32, s.lds, 1};
}

}  // namespace

extern "C" {

trt_status trt_block_norm(int64_t rows, int64_t cols, const void* r, int64_t ldr, const void* y, int64_t ldy,
                          const trt_block* block, void* r_out, int64_t ldro, void* h, int64_t ldh,
                          int32_t dtype, void* stream) {
  if (const trt_status s = check_sizes(rows, cols, dtype); s != TRT_OK) return s;
  if (const trt_status s = check_block(block, dtype); s != TRT_OK) return s;
  if (!r || !y || !r_out) return fail(TRT_ERR_NULL, "r, y and r_out must be non-null");
  trt::BlockNormArgs a = block_args(rows, cols, *block, dtype);
  const int64_t e = trt::elem_bytes(dtype), pe = trt::elem_bytes(block->param_dtype);
  const Buf bufs[] = {{"r_out", r_out, rows, cols, ldro, e},
                      {"h", h, rows, cols, ldh, e},
                      {"r", r, rows, cols, ldr, e},
                      {"y", y, rows, cols, ldy, e},
                      {"gate", a.gate, (rows + a.span - 1) / a.span, cols, a.ldg, trt::elem_bytes(block->gate_dtype)},
                      {"post_gamma", a.post_gamma, 1, cols, cols, pe},
                      {"post_beta", a.post_beta, 1, cols, cols, pe},
                      {"gamma", a.gamma, 1, cols, cols, pe},
                      {"beta", a.beta, 1, cols, cols, pe}};
  if (const trt_status s = trt::check_buffers(bufs, 2); s != TRT_OK) return s;
  a.r = {r, nullptr, ldr, 0};
  a.y = {y, nullptr, ldy, 0};
  a.out_r = r_out;
  a.out_y = h;
  a.ld_r = ldro;
  a.ld_y = ldh;
  return trt::launched(trt::launch_block_norm(a, dtype, static_cast<hipStream_t>(stream)), "block norm launch");
}

int64_t trt_block_norm_bwd_workspace_size(int64_t rows, int64_t cols, int64_t rows_per_gate, int32_t dtype) {
  if (check_sizes(rows, cols, dtype) != TRT_OK) return -1;
  if (rows_per_gate < 0) {
    fail(TRT_ERR_SIZE, "rows_per_gate must be >= 0");
    return -1;
  }
  trt::BlockCut cut;
  if (make_cut(rows, cols, rows_per_gate, dtype, cut) != TRT_OK) return -1;
  trt::g_err.clear();
  return workspace_of(cut, cols);
}

trt_status trt_block_norm_bwd(int64_t rows, int64_t cols, const void* dh, int64_t lddh, const void* dr_out,
                              int64_t lddro, const trt_saved* r_out, const trt_saved* y, const trt_block* block,
                              void* dr, int64_t lddr, void* dy, int64_t lddy, const trt_block_grads* grads,
                              int32_t dtype, void* workspace, int64_t workspace_bytes, void* stream) {
  if (const trt_status s = check_sizes(rows, cols, dtype); s != TRT_OK) return s;
  if (const trt_status s = check_block(block, dtype); s != TRT_OK) return s;
  if (!grads || !y || !y->x || !dr || !dy) return fail(TRT_ERR_NULL, "y, dr, dy and grads must be non-null");
  if (!dh && !dr_out) return fail(TRT_ERR_NULL, "dh or dr_out must be non-null");
  if (dh && (!r_out || !r_out->x)) return fail(TRT_ERR_NULL, "dh needs r_out");
  if (dh && !r_out->scale != !y->scale) return fail(TRT_ERR_ARG, "r_out and y must both be 8-bit rows, or neither");
  const trt_block_grads& g = *grads;
  if (!dh && (g.gamma || g.beta)) return fail(TRT_ERR_NULL, "dgamma and dbeta need dh");
  if (!block->gate && g.gate) return fail(TRT_ERR_NULL, "dgate needs the gate");
  if (!block->post && (g.post_gamma || g.post_beta))
    return fail(TRT_ERR_ARG, "dpost_gamma and dpost_beta need the norm behind the block");
  trt::BlockNormArgs a = block_args(rows, cols, *block, dtype);
  const bool each = a.gate && a.span == 1;
  const bool sums = g.post_gamma || g.post_beta || g.gamma || g.beta || (g.gate && !each);
  trt::BlockCut cut;
  if (const trt_status s = make_cut(rows, cols, block->gate ? block->rows_per_gate : 0, dtype, cut); s != TRT_OK) return s;
  const int64_t need = workspace_of(cut, cols);
  if (sums) {
    if (const trt_status s = trt::check_workspace(workspace, workspace_bytes, need); s != TRT_OK) return s;
  }
  const trt_saved absent{};
  const trt_saved& sr = dh ? *r_out : absent;
  const int64_t e = trt::elem_bytes(dtype), pe = trt::elem_bytes(block->param_dtype);
  const int64_t ge = trt::elem_bytes(block->gate_dtype), gates = (rows + a.span - 1) / a.span;
  const Buf bufs[] = {{"dr", dr, rows, cols, lddr, e},
                      {"dy", dy, rows, cols, lddy, e},
                      {"dgate", g.gate, gates, cols, g.ldg, ge},
                      {"dpost_gamma", g.post_gamma, 1, cols, cols, pe},
                      {"dpost_beta", g.post_beta, 1, cols, cols, pe},
                      {"dgamma", g.gamma, 1, cols, cols, pe},
                      {"dbeta", g.beta, 1, cols, cols, pe},
                      {"the workspace", sums ? workspace : nullptr, 1, need, need, 1},
                      {"dh", dh, rows, cols, lddh, e},
                      {"dr_out", dr_out, rows, cols, lddro, e},
                      saved_buf("r_out", sr, rows, cols, e),
                      scale_buf("r_out's scale", sr, rows, cols),
                      saved_buf("y", *y, rows, cols, e),
                      scale_buf("y's scale", *y, rows, cols),
                      {"gate", a.gate, gates, cols, a.ldg, ge},
                      {"post_gamma", a.post_gamma, 1, cols, cols, pe},
                      {"post_beta", a.post_beta, 1, cols, cols, pe},
                      {"gamma", a.gamma, 1, cols, cols, pe}};
  if (const trt_status s = trt::check_buffers(bufs, 8); s != TRT_OK) return s;
  a.r = {sr.x, sr.scale, sr.ld, sr.lds};
  a.y = {y->x, y->scale, y->ld, y->lds};
  a.out_r = dr;
  a.out_y = dy;
  a.ld_r = lddr;
  a.ld_y = lddy;
  a.dh = dh;
  a.dr = dr_out;
  a.lddh = lddh;
  a.lddr = lddro;
  a.dgate = each ? g.gate : nullptr;
  a.lddg = g.ldg;
  a.part = sums ? static_cast<float*>(workspace) : nullptr;
  a.slices = (int32_t)cut.slices;
  trt::BlockParamsArgs q{};
  q.part = a.part;
  q.gate = a.gate;
  q.post_gamma = a.post_gamma;
  q.post_beta = a.post_beta;
  q.ldg = a.ldg;
  q.lddg = g.ldg;
  q.dgate = each ? nullptr : g.gate;
  q.dpost_gamma = g.post_gamma;
  q.dpost_beta = g.post_beta;
  q.dgamma = g.gamma;
  q.dbeta = g.beta;
  q.cols = (int32_t)cols;
  q.groups = (int32_t)cut.groups;
  q.slices = (int32_t)cut.slices;
  q.each = each;
  q.pdt = block->param_dtype;
  q.gdt = block->gate_dtype;
  return trt::launched(trt::launch_block_norm_bwd(a, q, dtype, static_cast<hipStream_t>(stream)),
                       "block norm gradient launch");
}

}  // extern "C"
