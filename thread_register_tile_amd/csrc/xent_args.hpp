// xent_args.hpp -- the arguments of the cross entropy's kernels and their
// launch entry points (kern_xent*.hip).
#pragma once

#include "gemm_kernel.hpp"
#include "xent_plan.hpp"

namespace trt {

constexpr float kLog2E = 1.44269504088896340736f;

// G's scale: binary16's smallest value is 2^-24 (see xent.hpp).
template <int DT>
constexpr float kGradScale = DT == DT_F16 ? 16384.f : 1.f;

// The forward product: logits of the launch's columns, kept as pairs.
struct XentStatsArgs : GemmArgs {
  const int32_t* live;     // number of live tokens, or null: all M
  const int32_t* list;     // their rows in X, or null: in place
  const int32_t* want;     // the live tokens' targets, or null: target in place
  const int64_t* target;   // [tokens]
  float* at;               // [M] the target's logit
  f32x2* part;             // [tiles_n][tokens] (maximum, sum of exp(z - maximum))
  int64_t ldp;             // tokens
  int32_t tile0;           // the launch's first column tile in part
  int64_t col0;            // and its first vocabulary index
};

// What g needs of a live token: g = exp2(z log2(e) - lse2) a - [target] b.
struct XentRow {
  float a, b, lse2;
  int32_t target;   // its vocabulary index, or -1
};

// G over one piece of the vocabulary.
struct XentGradArgs : GemmArgs {   // C: G, of the inputs' type
  const int32_t* live;
  const int32_t* list;
  const XentRow* info;     // [live tokens]
  int32_t cols;            // vocabulary entries of the piece; G's columns past them are zero up to N
  int32_t halves;          // 1: two rows of G to a token, the rounded value and the rest
  int64_t col0;
};

// dX's sums over one piece.
struct XentInputArgs : GemmArgs {
  const XentHead* head;
  int32_t add;             // add to what the sums hold (every piece after the first)
  int32_t halves;          // as XentGradArgs
};

// dW over one piece.
struct XentWeightArgs : GemmArgs {
  const int32_t* live;
  const float* factor;     // c over G's scale
  int32_t g_cols;          // G's columns that are written
  int32_t halves;          // as XentGradArgs
};

struct XentPrepArgs {
  int32_t tokens;
  int64_t ignore;
  const int64_t* target;
  const float *dloss, *dlse;   // backward; dlse may be null
  int64_t inc_dloss, inc_dlse;
  float *loss, *lse;           // forward, else null
  int32_t *list, *place;       // live token -> row of X; row -> live token or -1 (backward)
  int32_t* want;               // forward: the live tokens' targets, -1 outside the vocabulary
  int32_t vocab;
  XentHead* head;
  float scale;                 // backward: G's scale
  int32_t width, k, wide;      // backward: dX's product, K of a whole piece
  int32_t halves;              // backward: as XentGradArgs
};

struct XentCombineArgs {
  const f32x2* part;
  int64_t ldp;
  int32_t tiles, tokens, vocab;
  const XentHead* head;    // null: no list, every token in place
  const int32_t* list;
  const int64_t* target;
  int64_t ignore;
  const float* at;
  float *loss, *lse;
};

struct XentRowsArgs {
  XentPrepArgs prep;
  const uint16_t* x;
  uint16_t* out;           // live tokens' rows of x; with halves, each twice
  const float* lse;
  XentRow* info;
  int64_t ldx, ld;
  int32_t width, vocab;
};

struct XentInputFinishArgs {
  const float* sums;
  const XentHead* head;
  const int32_t* place;
  void* dx;
  int64_t ld, lddx;
  int32_t width;
  int32_t halves;
  int32_t vec;             // dx's rows take aligned runs of four
};

// pipelined: the operands allow 16-byte copies; otherwise the generic kernel
// on 128x128 tiles runs the same epilogue.
hipError_t launch_xent_stats(XentStatsArgs a, int dt, bool wide, bool pipelined, hipStream_t s);
// For up to kXentStreamTokens tokens in place, where the copies' conditions hold.
hipError_t launch_xent_stream(const XentStatsArgs& a, int dt, hipStream_t s);
hipError_t launch_xent_grad(XentGradArgs a, int dt, bool wide, bool pipelined, hipStream_t s);
hipError_t launch_xent_input(XentInputArgs a, int dt, bool wide, bool pipelined, int64_t groups,
                             hipStream_t s);
hipError_t launch_xent_weight(XentWeightArgs a, int dt, bool wide, bool pipelined, hipStream_t s);

hipError_t launch_xent_prep(const XentPrepArgs& a, hipStream_t s);
hipError_t launch_xent_combine(const XentCombineArgs& a, hipStream_t s);
hipError_t launch_xent_rows(const XentRowsArgs& a, int dt, hipStream_t s);
hipError_t launch_xent_input_finish(const XentInputFinishArgs& a, int64_t tokens, int odt,
                                    hipStream_t s);

}  // namespace trt
