// trt_act8.hip -- the entry points of activations saved in 8 bits: argument
// checks, the plan, and the launches.  Declarations and contracts are in
// include/trt.h.
#include "act8_args.hpp"
#include "buffers.hpp"

namespace {

using trt::Buf;
using trt::fail;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int64_t blocks_of(int64_t cols) { return (cols + trt::kAct8Block - 1) / trt::kAct8Block; }

trt_status check_rows(int64_t rows, int64_t cols, int32_t dtype) {
  if (rows < 1 || cols < 1 || rows > trt::kMaxDim || cols > trt::kMaxDim)
    return fail(TRT_ERR_SIZE, "rows and cols must be in [1, 2^30]");
  if (dtype != TRT_F16 && dtype != TRT_BF16 && dtype != TRT_F32)
    return fail(TRT_ERR_DTYPE, "dtype must be TRT_F16, TRT_BF16 or TRT_F32");
  if (trt::act8_groups(rows, cols, trt::elem_bytes(dtype)) < 0)
    return fail(TRT_ERR_SIZE, "2^34 or more chunks of 16 bytes in one launch");
  return TRT_OK;
}

trt::Act8Args rows_args(const void* x, void* out, int64_t ldx, const int8_t* q, int64_t ldq,
                        const uint8_t* scale, int64_t lds, int64_t rows, int64_t cols) {
  trt::Act8Args a{};
  a.x = x;
  a.out = out;
  a.q = const_cast<int8_t*>(q);
  a.scale = const_cast<uint8_t*>(scale);
  a.ldx = ldx;
  a.ldq = ldq;
  a.lds = lds;
  a.rows = rows;
  a.cols = (int32_t)cols;
  return a;
}

trt_status check_product(int64_t tokens, int64_t outputs, int64_t inputs) {
  if (tokens < 1 || outputs < 1 || inputs < 1) return fail(TRT_ERR_SIZE, "tokens, outputs and inputs must be >= 1");
  if (tokens > trt::kAct8MaxTokens || outputs > trt::kAct8MaxWidth || inputs > trt::kAct8MaxWidth)
    return fail(TRT_ERR_SIZE, "tokens must be <= 2^23, outputs and inputs <= 2^20");
  // every launch counts its threads in 32 bits
  const int64_t x = trt::act8_groups(tokens, inputs, 2), y = trt::act8_groups(tokens, outputs, 2);
  if (x < 0 || y < 0 || x + y >= int64_t(1) << 24)
    return fail(TRT_ERR_SIZE, "2^34 or more chunks of 16 bytes in one launch");
  return TRT_OK;
}

// dy's rows as the product's copies take them: whole aligned chunks, one row
// behind the other.
bool in_place(const void* dy, int64_t lddy, int64_t outputs) {
  return aligned16(dy) && lddy % 8 == 0 && outputs % 8 == 0 && lddy >= outputs && lddy <= trt::kAct8MaxInPlace;
}

trt_status make_plan(int64_t tokens, int64_t outputs, int64_t inputs, const void* dy, int64_t lddy,
                     trt::Act8WeightPlan& p) {
  if (const trt_status s = check_product(tokens, outputs, inputs); s != TRT_OK) return s;
  p = trt::act8_weight_plan(tokens, outputs, inputs, lddy, in_place(dy, lddy, outputs));
  const int64_t tile = p.wide ? 256 : 128;
  if (((outputs + tile - 1) / tile) * ((inputs + tile - 1) / tile) * p.slices >= int64_t(1) << 24)
    return fail(TRT_ERR_SIZE, "2^24 or more output tiles in one launch");
  return TRT_OK;
}

}  // namespace

extern "C" {

trt_status trt_act8_pack(int64_t rows, int64_t cols, const void* x, int64_t ldx, int8_t* q, int64_t ldq,
                         uint8_t* scale, int64_t lds, int32_t dtype, void* stream) {
  if (const trt_status s = check_rows(rows, cols, dtype); s != TRT_OK) return s;
  if (!x || !q || !scale) return fail(TRT_ERR_NULL, "x, q and scale must be non-null");
  const Buf bufs[] = {{"q", q, rows, cols, ldq, 1},
                      {"scale", scale, rows, blocks_of(cols), lds, 1},
                      {"x", x, rows, cols, ldx, trt::elem_bytes(dtype)}};
  if (const trt_status s = trt::check_buffers(bufs, 2); s != TRT_OK) return s;
  const trt::Act8Args a = rows_args(x, nullptr, ldx, q, ldq, scale, lds, rows, cols);
  return trt::launched(trt::launch_act8_pack(a, dtype, trt::act8_groups(rows, cols, trt::elem_bytes(dtype)),
                                             static_cast<hipStream_t>(stream)),
                       "8-bit packing launch");
}

trt_status trt_act8_unpack(int64_t rows, int64_t cols, const int8_t* q, int64_t ldq, const uint8_t* scale,
                           int64_t lds, void* x, int64_t ldx, int32_t dtype, void* stream) {
  if (const trt_status s = check_rows(rows, cols, dtype); s != TRT_OK) return s;
  if (!x || !q || !scale) return fail(TRT_ERR_NULL, "q, scale and x must be non-null");
  const Buf bufs[] = {{"x", x, rows, cols, ldx, trt::elem_bytes(dtype)},
                      {"q", q, rows, cols, ldq, 1},
                      {"scale", scale, rows, blocks_of(cols), lds, 1}};
  if (const trt_status s = trt::check_buffers(bufs, 1); s != TRT_OK) return s;
  const trt::Act8Args a = rows_args(nullptr, x, ldx, q, ldq, scale, lds, rows, cols);
  return trt::launched(trt::launch_act8_unpack(a, dtype, trt::act8_groups(rows, cols, trt::elem_bytes(dtype)),
                                               static_cast<hipStream_t>(stream)),
                       "8-bit unpacking launch");
}

int64_t trt_act8_weight_grad_workspace_size(int64_t tokens, int64_t outputs, int64_t inputs, const void* dy,
                                            int64_t lddy) {
  trt::Act8WeightPlan plan;
  if (make_plan(tokens, outputs, inputs, dy, lddy, plan) != TRT_OK) return -1;
  trt::g_err.clear();
  return plan.bytes;
}

trt_status trt_act8_weight_grad(int64_t tokens, int64_t outputs, int64_t inputs, const void* dy, int64_t lddy,
                                const int8_t* q, int64_t ldq, const uint8_t* scale, int64_t lds, void* dw,
                                int64_t lddw, int32_t in_dtype, int32_t out_dtype, void* workspace,
                                int64_t workspace_bytes, void* stream) {
  trt::Act8WeightPlan plan;
  if (const trt_status s = make_plan(tokens, outputs, inputs, dy, lddy, plan); s != TRT_OK) return s;
  if (in_dtype != TRT_F16 && in_dtype != TRT_BF16) return fail(TRT_ERR_DTYPE, "dy must be TRT_F16 or TRT_BF16");
  if (out_dtype != TRT_F16 && out_dtype != TRT_BF16 && out_dtype != TRT_F32)
    return fail(TRT_ERR_DTYPE, "out_dtype must be TRT_F16, TRT_BF16 or TRT_F32");
  if (!dy || !q || !scale || !dw) return fail(TRT_ERR_NULL, "dy, q, scale and dw must be non-null");
  if (const trt_status s = trt::check_workspace(workspace, workspace_bytes, plan.bytes); s != TRT_OK) return s;
  const int64_t oe = trt::elem_bytes(out_dtype);
  const Buf bufs[] = {{"dw", dw, outputs, inputs, lddw, oe},
                      {"the workspace", workspace, 1, plan.bytes, plan.bytes, 1},
                      {"dy", dy, tokens, outputs, lddy, 2},
                      {"q", q, tokens, inputs, ldq, 1},
                      {"scale", scale, tokens, blocks_of(inputs), lds, 1}};
  if (const trt_status s = trt::check_buffers(bufs, 2); s != TRT_OK) return s;

  const hipStream_t st = static_cast<hipStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  auto done = [](hipError_t e) { return trt::launched(e, "weight gradient launch"); };
  trt::Act8OperandArgs o{};
  o.x = rows_args(nullptr, ws + plan.x, plan.x_ld, q, ldq, scale, lds, tokens, inputs);
  int64_t groups = trt::act8_groups(tokens, inputs, 2);
  o.x_groups = (int32_t)groups;
  if (plan.dy_ld) {
    o.dy = static_cast<const uint16_t*>(dy);
    o.dy_out = reinterpret_cast<uint16_t*>(ws + plan.dy);
    o.lddy = lddy;
    o.dy_ld = plan.dy_ld;
    o.dy_cols = (int32_t)outputs;
    groups += trt::act8_groups(tokens, outputs, 2);
  }
  if (const hipError_t e = trt::launch_act8_operands(o, in_dtype, groups, st); e != hipSuccess) return done(e);

  const bool parts = plan.slices > 1;
  trt::Act8WeightArgs a{};
  a.A = plan.dy_ld ? o.dy_out : static_cast<const uint16_t*>(dy);
  a.B = reinterpret_cast<const uint16_t*>(ws + plan.x);
  a.C = parts ? static_cast<void*>(ws + plan.part) : dw;
  a.lda = plan.dy_ld ? plan.dy_ld : lddy;
  a.ldb = plan.x_ld;
  a.ldc = parts ? plan.part_ld : lddw;
  a.M = (int32_t)outputs;
  // (a slice's results take the zero columns of x up to a multiple of 4 too)
  a.N = (int32_t)(parts ? plan.part_ld : inputs);
  a.K = (int32_t)tokens;
  a.out_dt = parts ? TRT_F32 : out_dtype;
  a.epi_vec = parts || ((reinterpret_cast<uintptr_t>(dw) & (uintptr_t)(4 * oe - 1)) == 0 && lddw % 4 == 0);
  a.slice = (int32_t)plan.slice;
  a.part = parts ? outputs * plan.part_ld : 0;
  if (const hipError_t e = trt::launch_act8_weight(a, in_dtype, plan.wide, plan.slices, st); e != hipSuccess || !parts)
    return done(e);
  trt::Act8SumArgs c{};
  c.part = reinterpret_cast<const float*>(ws + plan.part);
  c.dw = dw;
  c.ld = lddw;
  c.part_ld = plan.part_ld;
  c.step = a.part;
  c.rows = (int32_t)outputs;
  c.cols = (int32_t)inputs;
  c.slices = (int32_t)plan.slices;
  return done(trt::launch_act8_sum(c, out_dtype, st));
}

}  // extern "C"
