// blocknorm_args.hpp -- the arguments of a block's fused norms and their launch
// entry points (kern_blocknorm*.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace trt {

// Rows of the kernel's type, or 8-bit ones where scale is given.
struct SavedRows {
  const void* x;
  const uint8_t* scale;
  int64_t ld, lds;
};

struct BlockNormArgs {
  const void *gate, *post_gamma, *post_beta, *gamma, *beta;   // null: ones, zeros
  int64_t ldg;
  int32_t span;          // rows to a gate row (rows: one for all)
  int32_t rows, cols;
  float alpha, eps;
  int32_t rms, post;
  int32_t wide_params, wide_gate;   // binary32 beside 16-bit rows
  SavedRows r, y;        // forward: the stream and the block's output; backward: the stream behind the block
  void *out_r, *out_y;   // forward: the stream and h (or null); backward: dr and dy
  int64_t ld_r, ld_y;
  // backward
  const void *dh, *dr;   // either may be null
  int64_t lddh, lddr;
  void* dgate;           // a gate of its own for every row: written with dr and dy
  int64_t lddg;
  float* part;           // [groups * slices][4][cols] sums of e, e yhat, dh, dh rhat; or null
                         // (gate rows of few rows have a slice each)
  int32_t slices;        // workgroups to a gate row (both passes)
};

// The parameters' and the gate rows' gradients from the workgroups' sums.
struct BlockParamsArgs {
  const float* part;
  const void *gate, *post_gamma, *post_beta;
  int64_t ldg, lddg;
  void *dgate, *dpost_gamma, *dpost_beta, *dgamma, *dbeta;   // each may be null
  int32_t cols, groups, slices;
  int32_t each;          // the gate has been multiplied in
  int32_t pdt, gdt;
};

// Longest row: 32 KiB, two 16-byte chunks for each lane of 16 waves, whose 128
// registers do not hold more backward (they spill already, with 64 KiB of vectors or
// 128 KiB of sums in LDS).
constexpr int64_t kBlockMaxRowBytes = 32768;

// How the backward pass's rows are dealt: `groups` gate rows (one, where the
// gate is one for all or one for each row) of `slices` workgroups.
struct BlockCut {
  int64_t groups, slices;
};
BlockCut block_norm_cut(int64_t rows, int64_t cols, int64_t span, int dt);

hipError_t launch_block_norm(BlockNormArgs a, int dt, hipStream_t s);   // (a.slices: its own choice)
hipError_t launch_block_norm_bwd(const BlockNormArgs& a, const BlockParamsArgs& q, int dt, hipStream_t s);

// One unit to a type and a form of the saved rows (kern_blocknorm_bwd_*.hip).
template <int DT, bool BYTES>
hipError_t launch_block_norm_rows(const BlockNormArgs& a, int64_t groups, hipStream_t s);

}  // namespace trt
