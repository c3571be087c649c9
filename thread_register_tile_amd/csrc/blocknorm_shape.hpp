// blocknorm_shape.hpp -- how the block norm's rows are dealt to waves and
// workgroups: functions of the sizes alone.
#pragma once

#include "layernorm.hpp"

namespace trt {

constexpr int64_t block_chunks(int64_t cols, int dt) {
  return dt == DT_F32 ? (cols + 3) / 4 : (cols + 7) / 8;
}

// The shape of a row of `chunks` 16-byte chunks: W waves, K chunks to a lane.  f is
// called with <W, K>.
// Forward: one chunk up to 768 chunks, two beyond (4000 rows of 625 chunks take 36 us
// in 10 waves of one, 52 in 8 of two; 16384 rows of 1024 190 in 8 of two, 207 in 16
// of one; 60000 rows of 138 119 in 3 of one, 135 in 4 of one).
template <class F>
auto with_forward_shape(int64_t chunks, F&& f) {
  if (chunks <= 64) return f.template operator()<1, 1>();
  if (chunks <= 128) return f.template operator()<2, 1>();
  if (chunks <= 192) return f.template operator()<3, 1>();
  if (chunks <= 256) return f.template operator()<4, 1>();
  if (chunks <= 384) return f.template operator()<6, 1>();
  if (chunks <= 512) return f.template operator()<8, 1>();
  if (chunks <= 640) return f.template operator()<10, 1>();
  if (chunks <= 768) return f.template operator()<12, 1>();
  if (chunks <= 1024) return f.template operator()<8, 2>();
  if (chunks <= 1536) return f.template operator()<12, 2>();
  return f.template operator()<16, 2>();
}

// Backward: two chunks, so that the vectors and sums that a lane keeps fit beside
// the rows; one where three waves to a SIMD then share the work evenly (bf16 from 8-bit
// rows: 26214 rows of 320 chunks take 140 us in 6 waves of one, 178 in 4 of two; 43690
// of 192 134 in 3 of one, 150 in 2 of two).
template <class F>
auto with_block_shape(int64_t chunks, F&& f) {
  if (chunks <= 64) return f.template operator()<1, 1>();
  if (chunks <= 128) return f.template operator()<1, 2>();
  if (chunks <= 192) return f.template operator()<3, 1>();
  if (chunks <= 256) return f.template operator()<2, 2>();
  if (chunks <= 384) return f.template operator()<6, 1>();
  if (chunks <= 512) return f.template operator()<4, 2>();
  if (chunks <= 768) return f.template operator()<12, 1>();
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

// Slices of a gate row of `need` turns, where `most` workgroups run at a time: the
// number that takes the least turns, counting a round's start and end as `beside`,
// of up to four rounds.  For each number of rounds that is the most slices that fit,
// or the fewest with as many turns.
constexpr int64_t cheapest_slices(int64_t need, int64_t groups, int64_t most, int64_t beside) {
  if (groups == 1) return even_grid(need, most);
  int64_t best = 1, least = (groups + most - 1) / most * (need + beside);
  for (int64_t rounds = 1; rounds <= 4; ++rounds) {
    int64_t s = rounds * most / groups;
    if (s < 1) continue;
    s = even_grid(need, s < need ? s : need);
    const int64_t cost = (s * groups + most - 1) / most * ((need + s - 1) / s + beside);
    if (cost < least) best = s, least = cost;
  }
  return best;
}

// Forward workgroups, up to 20 waves of one chunk to a lane or 16 to each of the 256
// units, as their registers allow (a row's own where it has more).
template <int W, int K>
int64_t forward_slices(int64_t span, int64_t groups) {
  constexpr int waves = NormShape<W>::THREADS / 64, each = (K == 1 ? 20 : 16) / waves;
  return cheapest_slices((span + NormShape<W>::GROUPS - 1) / NormShape<W>::GROUPS, groups, 256 * each, 1);
}

// Backward workgroups: 8 waves, or 12 of one chunk to a lane, of which a row has W
// (and as many as it needs above 8); fewer where rows are too few to give every unit
// such a workgroup.
template <int W>
constexpr int kBlockWaves = W < 8 ? 8 % W ? 12 : 8 : W;
template <int W>
constexpr int kBlockFewWaves = W <= 2 ? 4 : W;

template <int W>
bool block_large(int64_t rows) {
  constexpr int per = kBlockWaves<W> / W;
  return kBlockWaves<W> != kBlockFewWaves<W> && (rows + per - 1) / per >= 256;
}

// Slices of a gate row of `span` rows; one workgroup runs on a unit at a time, and
// its end is the store of four sums.
inline int64_t block_slices(int64_t rows, int64_t span, int64_t groups, int64_t chunks) {
  return with_block_shape(chunks, [&]<int W, int K>() -> int64_t {
    const int64_t per = (block_large<W>(rows) ? kBlockWaves<W> : kBlockFewWaves<W>) / W;
    return cheapest_slices(((span < rows ? span : rows) + per - 1) / per, groups, 256, 2);
  });
}

}  // namespace trt
