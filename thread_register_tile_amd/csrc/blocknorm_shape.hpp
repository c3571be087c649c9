// blocknorm_shape.hpp -- how the block norm's rows are dealt to waves and
// workgroups: functions of the sizes alone.
#pragma once

#include "layernorm.hpp"

namespace trt {

constexpr int64_t block_chunks(int64_t cols, int dt) {
  return dt == DT_F32 ? (cols + 3) / 4 : (cols + 7) / 8;
}

// W waves to a row, K 16-byte chunks to a lane: two chunks, so that the vectors
// a lane keeps and the sums of the backward pass fit beside the rows, and as few
// waves as hold the row.  f is called with <W, K>.
template <class F>
auto with_block_shape(int64_t chunks, F&& f) {
  if (chunks <= 64) return f.template operator()<1, 1>();
  if (chunks <= 128) return f.template operator()<1, 2>();
  if (chunks <= 256) return f.template operator()<2, 2>();
  if (chunks <= 512) return f.template operator()<4, 2>();
  if (chunks <= 768) return f.template operator()<6, 2>();
  if (chunks <= 1024) return f.template operator()<8, 2>();
  if (chunks <= 1536) return f.template operator()<12, 2>();
  return f.template operator()<16, 2>();
}

// Workgroups for `need` turns, at most `most`, each with the same number of
// turns but for the last.
constexpr int64_t even_grid(int64_t need, int64_t most) {
  const int64_t turns = (need + most - 1) / most;
  return (need + turns - 1) / turns;
}

// Forward workgroups, 16 waves to each of the 256 units (a row's own where it
// has more).
template <int W>
constexpr int64_t forward_units() {
  return 256 * (16 / (NormShape<W>::THREADS / 64) > 0 ? 16 / (NormShape<W>::THREADS / 64) : 1);
}

// Backward workgroups: 8 waves, of which a row has W (and as many as it needs
// where that is not a divisor); half of that where rows are too few to give
// every unit one.
template <int W>
constexpr int kBlockWaves = W < 8 && 8 % W == 0 ? 8 : W;
template <int W>
constexpr int kBlockFewWaves = W <= 2 ? 4 : W;

template <int W>
bool block_large(int64_t rows) {
  constexpr int per = kBlockWaves<W> / W;
  return kBlockWaves<W> != kBlockFewWaves<W> && (rows + per - 1) / per >= 256;
}

// Slices of a gate row of `span` rows: the number that takes the least turns
// where one workgroup runs on a unit at a time, counting a round of starting and
// ending (the sums' store) as two turns.
inline int64_t block_slices(int64_t rows, int64_t span, int64_t groups, int64_t chunks) {
  return with_block_shape(chunks, [&]<int W, int K>() -> int64_t {
    const int64_t per = (block_large<W>(rows) ? kBlockWaves<W> : kBlockFewWaves<W>) / W;
    const int64_t need = ((span < rows ? span : rows) + per - 1) / per;
    if (groups == 1) return even_grid(need, 256);
    int64_t best = 1, least = -1;
    for (int64_t s = 1; s <= need && (s == 1 || s * groups <= 1024); ++s) {
      const int64_t cost = (s * groups + 255) / 256 * ((need + s - 1) / s + 2);
      if (least < 0 || cost < least) best = s, least = cost;
    }
    return best;
  });
}

}  // namespace trt
