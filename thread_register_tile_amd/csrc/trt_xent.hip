// trt_xent.hip -- the linear cross entropy's entry points: argument checks,
// the plan, and the launches.  Declarations and contracts are in
// include/trt.h.
#include "buffers.hpp"
#include "xent_args.hpp"

namespace {

using trt::Buf;
using trt::fail;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Byte extents a buffer descriptor addresses, with room for the copies' bias.
constexpr int64_t kExtent = (int64_t(1) << 31) - 8192;

trt_status check_sizes(int64_t tokens, int64_t vocab, int64_t width) {
  if (tokens < 1 || vocab < 1 || width < 1) return fail(TRT_ERR_SIZE, "tokens, vocab and width must be >= 1");
  if (tokens > trt::kXentMaxTokens || vocab > trt::kMaxDim || width > trt::kXentMaxWidth)
    return fail(TRT_ERR_SIZE, "tokens must be <= 2^23, vocab <= 2^30 and width <= 2^20");
  // a launch counts its threads in 32 bits: 256 to a tile of 128x128
  const int64_t t = (tokens + 127) / 128, v = (vocab + 127) / 128, d = (width + 127) / 128;
  if (t * v >= int64_t(1) << 24 || v * d >= int64_t(1) << 24 || t * d >= int64_t(1) << 24)
    return fail(TRT_ERR_SIZE, "2^24 or more output tiles of 128x128 in one launch");
  return TRT_OK;
}

trt_status check_dtype(int32_t dtype) {
  if (dtype != TRT_F16 && dtype != TRT_BF16)
    return fail(TRT_ERR_DTYPE, "x and w must be TRT_F16 or TRT_BF16");
  return TRT_OK;
}

trt_status check_piece(int64_t piece) {
  if (piece < 0 || piece % 64 != 0 || piece > trt::kXentMaxPiece)
    return fail(TRT_ERR_ARG, "piece must be 0 or a multiple of 64 up to 2^20");
  return TRT_OK;
}

trt_status check_inputs(const void* x, int64_t ldx, const void* w, int64_t ldw,
                        const int64_t* target, int64_t width) {
  if (!x || !w || !target) return fail(TRT_ERR_NULL, "x, w and target must be non-null");
  if (ldx < width || ldw < width)
    return fail(TRT_ERR_STRIDE, "the leading dimensions of x and w must be >= width");
  return TRT_OK;
}

}  // namespace

extern "C" {

int64_t trt_linear_xent_workspace_size(int64_t tokens, int64_t vocab, int64_t width) {
  if (check_sizes(tokens, vocab, width) != TRT_OK) return -1;
  trt::g_err.clear();
  return trt::xent_fwd_plan(tokens, vocab).bytes;
}

trt_status trt_linear_xent(int64_t tokens, int64_t vocab, int64_t width, const void* x,
                           int64_t ldx, const void* w, int64_t ldw, const int64_t* target,
                           int64_t ignore_index, float* loss, float* lse, int32_t dtype,
                           void* workspace, int64_t workspace_bytes, void* stream) {
  if (const trt_status s = check_sizes(tokens, vocab, width); s != TRT_OK) return s;
  if (const trt_status s = check_dtype(dtype); s != TRT_OK) return s;
  if (const trt_status s = check_inputs(x, ldx, w, ldw, target, width); s != TRT_OK) return s;
  if (!loss || !lse) return fail(TRT_ERR_NULL, "loss and lse must be non-null");
  const trt::XentFwdPlan plan = trt::xent_fwd_plan(tokens, vocab);
  if (const trt_status s = trt::check_workspace(workspace, workspace_bytes, plan.bytes); s != TRT_OK) return s;
  const Buf bufs[] = {{"loss", loss, 1, tokens, tokens, 4},
                      {"lse", lse, 1, tokens, tokens, 4},
                      {"the workspace", workspace, 1, plan.bytes, plan.bytes, 1},
                      {"x", x, tokens, width, ldx, 2},
                      {"w", w, vocab, width, ldw, 2},
                      {"target", target, 1, tokens, tokens, 8}};
  if (const trt_status s = trt::check_buffers(bufs, 3); s != TRT_OK) return s;

  const hipStream_t st = static_cast<hipStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  const bool listed = tokens > trt::kXentInPlace;
  auto* head = reinterpret_cast<trt::XentHead*>(ws + plan.head);
  auto* list = reinterpret_cast<int32_t*>(ws + plan.list);
  auto* want = reinterpret_cast<int32_t*>(ws + plan.want);
  hipError_t e = hipSuccess;
  if (listed) {
    trt::XentPrepArgs a{};
    a.tokens = (int32_t)tokens;
    a.ignore = ignore_index;
    a.target = target;
    a.loss = loss;
    a.lse = lse;
    a.list = list;
    a.want = want;
    a.vocab = (int32_t)vocab;
    a.head = head;
    a.scale = 1.f;
    e = trt::launch_xent_prep(a, st);
    if (e != hipSuccess) return trt::launched(e, "cross entropy launch");
  }

  // one launch per 2 GiB of w (the stream over W addresses it whole)
  trt::XentStatsArgs a{};
  const bool vec = width % 8 == 0 && ldx % 8 == 0 && ldw % 8 == 0 && aligned16(x) && aligned16(w);
  // (of more entries the stream's launch would have 2^32 threads)
  const bool stream_w = vec && tokens <= trt::kXentStreamTokens && vocab <= trt::kMaxDim / 4;
  const int64_t chunk = kExtent / (2 * ldw) / 256 * 256;
  const bool pipelined = vec && chunk >= 256 && ((tokens - 1) * ldx + width) * 2 < kExtent;
  const int64_t step = pipelined && !stream_w ? chunk : vocab;
  const int64_t tile = stream_w ? trt::kXentStreamTile : pipelined && plan.wide ? 256 : 128;
  for (int64_t v0 = 0; v0 < vocab; v0 += step) {
    const int64_t n = vocab - v0 < step ? vocab - v0 : step;
    a.A = static_cast<const uint16_t*>(x);
    a.B = static_cast<const uint16_t*>(w) + v0 * ldw;
    a.lda = ldx;
    a.ldb = ldw;
    a.M = (int32_t)tokens;
    a.N = (int32_t)n;
    a.K = (int32_t)width;
    a.a_bytes = ((tokens - 1) * ldx + width) * 2;
    a.b_bytes = ((n - 1) * ldw + width) * 2;
    a.live = listed ? &head->live : nullptr;
    a.list = listed ? list : nullptr;
    a.want = listed ? want : nullptr;
    a.target = target;
    a.at = reinterpret_cast<float*>(ws + plan.at);
    a.part = reinterpret_cast<trt::f32x2*>(ws + plan.part);
    a.ldp = tokens;
    a.tile0 = (int32_t)(v0 / tile);
    a.col0 = v0;
    e = stream_w ? trt::launch_xent_stream(a, dtype, st)
                 : trt::launch_xent_stats(a, dtype, plan.wide, pipelined, st);
    if (e != hipSuccess) return trt::launched(e, "cross entropy launch");
  }
  trt::XentCombineArgs c{};
  c.part = a.part;
  c.ldp = tokens;
  c.tiles = (int32_t)((vocab + tile - 1) / tile);
  c.tokens = (int32_t)tokens;
  c.vocab = (int32_t)vocab;
  c.head = listed ? head : nullptr;
  c.list = a.list;
  c.target = target;
  c.ignore = ignore_index;
  c.at = a.at;
  c.loss = loss;
  c.lse = lse;
  return trt::launched(trt::launch_xent_combine(c, st), "cross entropy launch");
}

int64_t trt_linear_xent_bwd_workspace_size(int64_t tokens, int64_t vocab, int64_t width,
                                           int64_t piece) {
  if (check_sizes(tokens, vocab, width) != TRT_OK || check_piece(piece) != TRT_OK) return -1;
  trt::g_err.clear();
  return trt::xent_bwd_plan(tokens, vocab, width, piece).bytes;
}

trt_status trt_linear_xent_bwd(int64_t tokens, int64_t vocab, int64_t width, const void* x,
                               int64_t ldx, const void* w, int64_t ldw, const int64_t* target,
                               int64_t ignore_index, const float* lse, const float* dloss,
                               int64_t inc_dloss, const float* dlse, int64_t inc_dlse, void* dx,
                               int64_t lddx, void* dw, int64_t lddw, int32_t in_dtype,
                               int32_t out_dtype, int64_t piece, void* workspace,
                               int64_t workspace_bytes, void* stream) {
  if (const trt_status s = check_sizes(tokens, vocab, width); s != TRT_OK) return s;
  if (const trt_status s = check_dtype(in_dtype); s != TRT_OK) return s;
  if (out_dtype != TRT_F16 && out_dtype != TRT_BF16 && out_dtype != TRT_F32)
    return fail(TRT_ERR_DTYPE, "out_dtype must be TRT_F16, TRT_BF16 or TRT_F32");
  if (const trt_status s = check_piece(piece); s != TRT_OK) return s;
  if (const trt_status s = check_inputs(x, ldx, w, ldw, target, width); s != TRT_OK) return s;
  if (!lse || !dloss) return fail(TRT_ERR_NULL, "lse and dloss must be non-null");
  if (!dx && !dw) return fail(TRT_ERR_NULL, "dx or dw must be non-null");
  if (inc_dloss < 0 || (dlse && inc_dlse < 0))
    return fail(TRT_ERR_STRIDE, "the increments of dloss and dlse must be >= 0");
  const trt::XentBwdPlan plan = trt::xent_bwd_plan(tokens, vocab, width, piece);
  if (const trt_status s = trt::check_workspace(workspace, workspace_bytes, plan.bytes); s != TRT_OK) return s;
  const int64_t oe = trt::elem_bytes(out_dtype);
  // dloss and dlse as columns of `tokens` rows (one row where they do not advance)
  const Buf bufs[] = {{"dx", dx, tokens, width, lddx, oe},
                      {"dw", dw, vocab, width, lddw, oe},
                      {"the workspace", workspace, 1, plan.bytes, plan.bytes, 1},
                      {"x", x, tokens, width, ldx, 2},
                      {"w", w, vocab, width, ldw, 2},
                      {"target", target, 1, tokens, tokens, 8},
                      {"lse", lse, 1, tokens, tokens, 4},
                      {"dloss", dloss, inc_dloss ? tokens : 1, 1, inc_dloss ? inc_dloss : 1, 4},
                      {"dlse", dlse, inc_dlse ? tokens : 1, 1, inc_dlse ? inc_dlse : 1, 4}};
  if (const trt_status s = trt::check_buffers(bufs, 3); s != TRT_OK) return s;

  const hipStream_t st = static_cast<hipStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  auto* head = reinterpret_cast<trt::XentHead*>(ws + plan.head);
  auto* list = reinterpret_cast<int32_t*>(ws + plan.list);
  auto* place = reinterpret_cast<int32_t*>(ws + plan.place);
  auto* info = reinterpret_cast<trt::XentRow*>(ws + plan.info);
  auto* xs = reinterpret_cast<uint16_t*>(ws + plan.x);
  auto* g = reinterpret_cast<uint16_t*>(ws + plan.g);
  auto* sums = reinterpret_cast<float*>(ws + plan.sums);
  auto done = [](hipError_t e) { return trt::launched(e, "cross entropy gradient launch"); };

  trt::XentRowsArgs r{};
  r.prep.tokens = (int32_t)tokens;
  r.prep.ignore = ignore_index;
  r.prep.target = target;
  r.prep.dloss = dloss;
  r.prep.dlse = dlse;
  r.prep.inc_dloss = inc_dloss;
  r.prep.inc_dlse = inc_dlse;
  r.prep.list = list;
  r.prep.place = place;
  r.prep.head = head;
  r.prep.scale = in_dtype == TRT_F16 ? trt::kGradScale<trt::DT_F16> : trt::kGradScale<trt::DT_BF16>;
  r.prep.width = (int32_t)width;
  r.prep.k = (int32_t)(plan.piece < vocab ? plan.piece : vocab);
  r.prep.wide = plan.wide_x;
  r.x = static_cast<const uint16_t*>(x);
  r.out = xs;
  r.lse = lse;
  r.info = info;
  r.prep.halves = plan.halves;
  r.ldx = ldx;
  r.ld = plan.padded;
  r.width = (int32_t)width;
  r.vocab = (int32_t)vocab;
  if (const hipError_t e = trt::launch_xent_prep(r.prep, st); e != hipSuccess) return done(e);
  if (const hipError_t e = trt::launch_xent_rows(r, in_dtype, st); e != hipSuccess) return done(e);

  const int64_t rows256 = trt::round_up(tokens << (plan.halves ? 1 : 0), 256);   // of G and X'
  const bool vec_x = width % 8 == 0 && ldx % 8 == 0 && aligned16(x) &&
                     ((tokens - 1) * ldx + width) * 2 < kExtent;
  const bool vec_w = width % 8 == 0 && ldw % 8 == 0 && aligned16(w) &&
                     trt::round_up(plan.piece, 256) * ldw * 2 < kExtent;
  const bool vec_g = rows256 * plan.piece * 2 < kExtent;
  for (int64_t v0 = 0; v0 < vocab; v0 += plan.piece) {
    const int64_t n = vocab - v0 < plan.piece ? vocab - v0 : plan.piece;
    const int64_t n8 = trt::round_up(n, 8);
    const uint16_t* wp = static_cast<const uint16_t*>(w) + v0 * ldw;

    trt::XentGradArgs a{};
    a.A = static_cast<const uint16_t*>(x);
    a.B = wp;
    a.C = g;
    a.lda = ldx;
    a.ldb = ldw;
    a.ldc = plan.piece;
    a.M = (int32_t)tokens;
    a.N = (int32_t)n8;
    a.K = (int32_t)width;
    a.out_dt = in_dtype;
    a.epi_vec = 1;
    a.a_bytes = ((tokens - 1) * ldx + width) * 2;
    a.b_bytes = ((n - 1) * ldw + width) * 2;
    a.live = &head->live;
    a.list = list;
    a.info = info;
    a.cols = (int32_t)n;
    a.halves = plan.halves;
    a.col0 = v0;
    // the generic kernel reads w's rows up to N: they end at n
    const bool grad_pipelined = vec_x && vec_w;
    if (!grad_pipelined) a.N = (int32_t)n;
    if (const hipError_t e = trt::launch_xent_grad(a, in_dtype, plan.wide_g, grad_pipelined, st); e != hipSuccess)
      return done(e);

    if (dw) {
      trt::XentWeightArgs b{};
      b.A = g;
      b.B = xs;
      b.C = static_cast<char*>(dw) + v0 * lddw * oe;
      b.lda = plan.piece;
      b.ldb = plan.padded;
      b.ldc = lddw;
      b.M = (int32_t)n;
      b.N = (int32_t)width;
      b.K = (int32_t)tokens;
      b.out_dt = out_dtype;
      b.epi_vec = (reinterpret_cast<uintptr_t>(b.C) & (uintptr_t)(4 * oe - 1)) == 0 && lddw % 4 == 0;
      b.live = &head->live;
      b.factor = &head->factor;
      b.g_cols = (int32_t)n8;
      b.halves = plan.halves;
      const bool pipelined = vec_g && rows256 * plan.padded * 2 < kExtent;
      if (const hipError_t e = trt::launch_xent_weight(b, in_dtype, plan.wide_w, pipelined, st); e != hipSuccess)
        return done(e);
    }

    if (dx) {
      trt::XentInputArgs b{};
      b.A = g;
      b.B = wp;
      b.C = sums;
      b.lda = plan.piece;
      b.ldb = ldw;
      b.ldc = plan.padded;
      b.ldr = plan.padded;
      b.M = (int32_t)tokens;
      b.N = (int32_t)width;
      b.out_dt = TRT_F32;
      b.epi_vec = 1;
      b.b_bytes = ((n - 1) * ldw + width) * 2;
      b.head = head;
      b.add = v0 > 0;
      b.halves = plan.halves;
      // the pipelined kernel takes G's zero columns up to a multiple of 8 too,
      // where they are written; W's rows there lie past its extent and read as zero
      const bool pipelined = vec_w && vec_g && (grad_pipelined || n == n8);
      b.K = (int32_t)(pipelined ? n8 : n);
      // the grid holds the most workgroups that any number of live tokens asks
      // for; on a tile of 128 for one of 256, four times as many
      const int64_t groups = plan.most_tiles * (plan.wide_x && !pipelined ? 4 : 1);
      if (const hipError_t e = trt::launch_xent_input(b, in_dtype, plan.wide_x, pipelined, groups, st); e != hipSuccess)
        return done(e);
    }
  }
  if (dx) {
    trt::XentInputFinishArgs f{};
    f.sums = sums;
    f.head = head;
    f.place = place;
    f.halves = plan.halves;
    f.dx = dx;
    f.ld = plan.padded;
    f.lddx = lddx;
    f.width = (int32_t)width;
    f.vec = (reinterpret_cast<uintptr_t>(dx) & (uintptr_t)(4 * oe - 1)) == 0 && lddx % 4 == 0;
    return done(trt::launch_xent_input_finish(f, tokens, out_dtype, st));
  }
  return done(hipSuccess);
}

}  // extern "C"
