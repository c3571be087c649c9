// act8_args.hpp -- the arguments of the 8-bit activations' kernels, their
// plan and their launch entry points (kern_act8.hip, kern_act8_weight.hip).
#pragma once

#include "gemm_kernel.hpp"
#include "xent_plan.hpp"

namespace trt {

// 8-bit rows beside rows of a wider type: pack reads x, unpack writes it.
struct Act8Args {
  const void* x;
  void* out;             // unpack
  int8_t* q;
  uint8_t* scale;
  int64_t ldx, ldq, lds;
  int64_t rows;
  int32_t cols;
};

// Chunks of 16 bytes (of the wider type) to a workgroup, 256 threads.
constexpr int kAct8Chunks = 1024;
// Columns to a scale.
constexpr int kAct8Block = 32;

// Workgroups for rows x cols elements of esize bytes; a launch counts its
// threads in 32 bits, so 2^24 of them are too many.
constexpr int64_t act8_groups(int64_t rows, int64_t cols, int64_t esize) {
  const int64_t per = (cols + kAct8Block - 1) / kAct8Block * (kAct8Block * esize / 16);
  const __int128 n = ((__int128)rows * per + kAct8Chunks - 1) / kAct8Chunks;
  return n < (int64_t(1) << 24) ? (int64_t)n : -1;
}

// The operands of the weight gradient's product, as its copies want them: rows
// of whole 16-byte chunks.
struct Act8OperandArgs {
  Act8Args x;            // out: the restored rows, padded
  const uint16_t* dy;    // null: taken in place
  uint16_t* dy_out;
  int64_t lddy, dy_ld;
  int32_t dy_cols;
  int32_t x_groups;      // workgroups that restore x; the rest copy dy
};

// C = dY^T X, over a slice of the tokens to each row of the grid.
struct Act8WeightArgs : GemmArgs {
  int32_t slice;         // tokens of a slice (K: all of them)
  int64_t part;          // elements between the slices' results
};

struct Act8SumArgs {
  const float* part;
  void* dw;
  int64_t ld, part_ld, step;
  int32_t rows, cols, slices;
};

// How a weight gradient is cut: a function of the sizes and of whether dy is
// taken in place.
struct Act8WeightPlan {
  bool wide;             // 256x256 tiles, else 128x128
  int64_t x_ld, dy_ld;   // dy_ld 0: in place
  int64_t slices, slice; // of the tokens
  int64_t x, dy, part;   // byte offsets into the workspace
  int64_t part_ld;       // of a slice's results
  int64_t bytes;
};

// Byte extents a buffer descriptor addresses, with room for the copies' bias.
constexpr int64_t kAct8Extent = (int64_t(1) << 31) - 8192;
constexpr int64_t kAct8MaxTokens = int64_t(1) << 23, kAct8MaxWidth = int64_t(1) << 20;
// Longest rows of dy taken in place: slices of 448 tokens at least, so fewer
// than 2^16 of them.
constexpr int64_t kAct8MaxInPlace = int64_t(1) << 21;

// Time of the product cut into s slices, in picoseconds: what a unit's tiles take for
// each token (alone 5.5 to 7.5 ns of a 128x128 tile and 14.5 to 22 of a 256x256 one,
// as fewer or more of the 256 units share the power; in turn 6.8 and 21), what a tile
// costs beside them, and with slices their results' way to memory and back.
constexpr int64_t act8_cut_cost(int64_t tokens, int64_t outputs, int64_t inputs, int64_t s, bool wide) {
  const int64_t tile = wide ? 256 : 128;
  const int64_t groups = ((outputs + tile - 1) / tile) * ((inputs + tile - 1) / tile) * s, rounds = (groups + 255) / 256;
  const int64_t each = wide ? (rounds > 1 ? 21000 : 14500 + 7500 * groups / 256)
                            : (rounds > 1 ? 6800 : 5500 + 2000 * groups / 256);
  const int64_t joined = s > 1 ? 3'000'000 + s * outputs * inputs * 11 / 10 : 0;
  return rounds * xent_slice((uint32_t)s, (uint32_t)tokens) * each + 5'000'000 + joined;
}

// The cheapest of tiles and slices: in small models tokens are long, and outputs x
// inputs have few tiles.  At least 512 tokens to a slice, and 256-wide tiles from 769
// tokens on (few are all store, and two workgroups to a unit store faster).  Measured
// with one slice of 128-wide tiles, with two, and with 256-wide tiles in as many as
// suit them: 2048 tokens x 2048 x 2048 30, 41, 46 us, 8192 x 3000 x 1500 126, 123, 96, 16384 x
// 2048 x 2048 142, 150, 138.  Slices also keep each operand's extent below 2 GiB.
constexpr Act8WeightPlan act8_weight_plan(int64_t tokens, int64_t outputs, int64_t inputs,
                                          int64_t lddy, bool in_place) {
  Act8WeightPlan p{};
  p.x_ld = round_up(inputs, 8);
  p.dy_ld = in_place ? 0 : round_up(outputs, 8);
  const int64_t dy_ld = in_place ? lddy : p.dy_ld, ld = dy_ld > p.x_ld ? dy_ld : p.x_ld;
  const int64_t most = kAct8Extent / (2 * ld) / 64 * 64;   // tokens below 2 GiB
  const int64_t least = (tokens + most - 1) / most;
  int64_t cost = -1;
  for (int64_t s = least; s == least || (s <= kXentMostSlices && s * 512 <= tokens); ++s)
    for (int wide = tokens > 768; wide >= 0; --wide)
      if (const int64_t c = act8_cut_cost(tokens, outputs, inputs, s, wide); cost < 0 || c < cost)
        cost = c, p.slices = s, p.wide = wide;
  p.slice = xent_slice((uint32_t)p.slices, (uint32_t)tokens);
  p.slices = (tokens + p.slice - 1) / p.slice;
  p.part_ld = round_up(inputs, 4);
  int64_t at = 0;
  auto take = [&](int64_t n) { const int64_t o = at; at += round_up(n, 256); return o; };
  p.x = take(tokens * p.x_ld * 2);
  p.dy = take(tokens * p.dy_ld * 2);
  p.part = take(p.slices > 1 ? p.slices * outputs * p.part_ld * 4 : 0);
  p.bytes = at;
  return p;
}

hipError_t launch_act8_pack(const Act8Args& a, int dt, int64_t groups, hipStream_t s);
hipError_t launch_act8_unpack(const Act8Args& a, int dt, int64_t groups, hipStream_t s);
hipError_t launch_act8_operands(const Act8OperandArgs& a, int dt, int64_t groups, hipStream_t s);
hipError_t launch_act8_weight(Act8WeightArgs a, int dt, bool wide, int64_t slices, hipStream_t s);
hipError_t launch_act8_sum(const Act8SumArgs& a, int odt, hipStream_t s);

}  // namespace trt
