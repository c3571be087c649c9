// xent_plan.hpp -- how a linear cross entropy is cut up, and its workspace:
// a function of the sizes alone.  Pure C++.
#pragma once

#include <stdint.h>

namespace trt {

// What the prep kernel leaves on the device for the others.
struct XentHead {
  int32_t live;      // tokens that take part
  float c;           // largest weight s_t (backward)
  float factor;      // c over G's scale
  int32_t slice;     // K of a slice of dX's product (backward)
  int32_t slices;    // slices of a whole piece
};

// Tokens up to which G is held in two rows each: together they fit one tile of
// 128 rows of dX's product, whose time is reading W.  (Two rows each for up to
// 128 tokens: 77 x 16384 x 1024 63.5 us instead of 52.0, 128 x 131072 x 4096
// 1115 instead of 841.)
constexpr int64_t kXentHalvesTokens = 64;

// Largest number of tokens: one workgroup of 256 threads a token in a launch
// of fewer than 2^32 threads.  Largest width and piece: byte offsets into a
// tile's rows stay below 2^31.
constexpr int64_t kXentMaxTokens = int64_t(1) << 23;
constexpr int64_t kXentMaxWidth = int64_t(1) << 20;
constexpr int64_t kXentMaxPiece = int64_t(1) << 20;

constexpr int64_t round_up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }

// Tokens up to which the forward pass takes every row in place: they fit one
// tile row of 128, so a list of live tokens would save no work.
constexpr int64_t kXentInPlace = 128;

#if defined(__HIPCC__)
#define TRT_XENT_HD __host__ __device__
#else
#define TRT_XENT_HD
#endif

// dX has few tiles where live tokens or the width are few: its K is then cut
// into slices, each with sums of its own.  The number that takes the least
// time, counted in K: rounds of the compute units (two small tiles to one)
// times a slice's K and what a tile costs beside its products (about 10 us,
// of 23 us per 1024 of K); at least 512 of K each, and no more than four
// rounds of 256 in all.
constexpr int kXentMostSlices = 32;
// Time of s slices, or the largest value where so many are not allowed.
TRT_XENT_HD constexpr uint64_t xent_slice_cost(uint32_t s, uint32_t tiles, uint32_t k, bool wide) {
  const uint32_t units = wide ? 256 : 512, beside = 450;
  if (s > 1 && (s * 512 > k || (uint64_t)s * tiles > 1024)) return ~uint64_t(0);
  return (uint64_t)((tiles * s + units - 1) / units) * (k / s + beside);
}
TRT_XENT_HD constexpr uint32_t xent_input_tiles(int64_t rows, int64_t width, bool wide) {
  const uint32_t tile = wide ? 256 : 128;
  return (((uint32_t)rows + tile - 1) / tile) * (((uint32_t)width + tile - 1) / tile);
}
// The number of slices (the least of equal ones).
constexpr int64_t xent_slices(int64_t rows, int64_t width, int64_t k, bool wide) {
  const uint32_t tiles = xent_input_tiles(rows, width, wide);
  uint32_t best = 1;
  for (uint32_t s = 2; s <= kXentMostSlices; ++s)
    if (xent_slice_cost(s, tiles, (uint32_t)k, wide) < xent_slice_cost(best, tiles, (uint32_t)k, wide)) best = s;
  return best;
}
// K of each of s slices: a multiple of 64.
TRT_XENT_HD constexpr uint32_t xent_slice(uint32_t s, uint32_t k) { return ((k + s - 1) / s + 63) / 64 * 64; }
// Rows of a slice's sums: whole tiles.
TRT_XENT_HD constexpr int64_t xent_sum_rows(int64_t rows) { return (rows + 255) / 256 * 256; }

// Tokens up to which the forward pass streams W, 64 entries to a workgroup.
constexpr int64_t kXentStreamTokens = 4;
constexpr int kXentStreamTile = 64;

struct XentFwdPlan {
  bool wide;           // 256x256 tiles, else 128x128
  int64_t part, at, list, want, head;   // byte offsets into the workspace
  int64_t bytes;
};

// 256-wide tiles when they give the 256 compute units at least three quarters
// of a round (the GEMM's rule), else 128-wide ones.
constexpr bool xent_wide(int64_t m, int64_t n) {
  return m > 128 && ((m + 255) / 256) * ((n + 255) / 256) >= 192;
}

constexpr XentFwdPlan xent_fwd_plan(int64_t tokens, int64_t vocab) {
  XentFwdPlan p{};
  p.wide = xent_wide(tokens, vocab);
  int64_t at = 0;
  auto take = [&](int64_t n) { const int64_t o = at; at += round_up(n, 256); return o; };
  p.head = take(sizeof(XentHead));
  // for the smallest tile that any kernel of so many tokens takes
  const int64_t tile = tokens <= kXentStreamTokens ? kXentStreamTile : 128;
  p.part = take((vocab + tile - 1) / tile * tokens * 8);
  p.at = take(tokens * 4);
  p.list = take(tokens > kXentInPlace ? tokens * 4 : 0);
  p.want = take(tokens > kXentInPlace ? tokens * 4 : 0);
  p.bytes = at;
  return p;
}

struct XentBwdPlan {
  int64_t piece;       // vocabulary entries at a time, a multiple of 64
  int64_t pieces;
  int64_t padded;      // width of X' and of the sums' rows, a multiple of 8
  bool halves;         // two rows of G (and of X') to a token
  bool wide_g, wide_x, wide_w;   // 256-wide tiles for G, dX and dW
  int64_t most_tiles;            // workgroups of dX's product, for any number of live tokens
  int64_t head, list, place, info, x, g, sums;   // byte offsets
  int64_t bytes;
};

// The piece the library chooses: G of at most 2^28 elements (512 MiB: up to
// 32768 tokens), but 8192 entries at least, so that adding dX's sums (8 bytes per
// token, width and piece) stays small beside the piece's products; and no more
// than leaves G and as many rows of `width` below 2 GiB, the copies' limit, which
// 256 entries keep up to 2^22 - 256 tokens.  (W's rows count as ldw long against
// that limit: trt_xent.hip.)  X' and dX's sums take room beside G: 65536 tokens of
// width 4096 over 131072 entries 512 MiB and 1 GiB, G another.
constexpr int64_t xent_piece(int64_t tokens, int64_t vocab, int64_t width) {
  int64_t most = (int64_t(1) << 28) / tokens;
  if (most < 8192) most = 8192;
  const int64_t rows = tokens > width ? tokens : width;
  const int64_t limit = ((int64_t(1) << 30) - 4096) / round_up(rows, 256);
  if (most > limit) most = limit;
  if (most > kXentMaxPiece) most = kXentMaxPiece;
  if (most < 256) most = 256;
  most = most / 256 * 256;
  const int64_t pieces = (vocab + most - 1) / most;
  return round_up((vocab + pieces - 1) / pieces, 256);
}

constexpr XentBwdPlan xent_bwd_plan(int64_t tokens, int64_t vocab, int64_t width, int64_t piece) {
  XentBwdPlan p{};
  p.piece = piece > 0 ? piece : xent_piece(tokens, vocab, width);
  if (p.piece > round_up(vocab, 64)) p.piece = round_up(vocab, 64);
  p.pieces = (vocab + p.piece - 1) / p.piece;
  p.padded = round_up(width, 8);
  p.halves = tokens <= kXentHalvesTokens;
  const int64_t g_rows = tokens << (p.halves ? 1 : 0);   // the most there may be
  p.wide_g = xent_wide(tokens, p.piece);
  // dW of few tokens is all store: twice the workgroups to a unit (16 tokens:
  // 185 us against 168, 512: 417 against 401, 1024: 681 against 690, 32000 x 4096)
  p.wide_w = tokens > 768 && xent_wide(p.piece, width);
  p.wide_x = tokens > 192 && width > 192;   // (more than the tokens of halves)
  // the sums' room and the grid, for whatever number of tokens is live
  const int64_t tile = p.wide_x ? 256 : 128, cols = (width + tile - 1) / tile;
  const int64_t k = p.piece < vocab ? p.piece : vocab;
  int64_t sum_rows = 0;
  for (int64_t r = 0; r < g_rows; r += tile) {
    const int64_t rows = g_rows - r < tile ? g_rows : r + tile;
    const int64_t s = xent_slices(rows, width, k, p.wide_x);
    const int64_t tiles = ((rows + tile - 1) / tile) * cols;
    if (s * xent_sum_rows(rows) > sum_rows) sum_rows = s * xent_sum_rows(rows);
    if (s * tiles > p.most_tiles) p.most_tiles = s * tiles;
    // from here on there is one slice and both grow with the rows alone: on to
    // the last
    if (tiles > 512 && rows < g_rows) r = (g_rows - 1) / tile * tile - tile;
  }
  int64_t at = 0;
  auto take = [&](int64_t n) { const int64_t o = at; at += round_up(n, 256); return o; };
  p.head = take(sizeof(XentHead));
  p.list = take(tokens * 4);
  p.place = take(tokens * 4);
  p.info = take(tokens * 16);
  p.x = take(g_rows * p.padded * 2);
  p.g = take(g_rows * p.piece * 2);
  p.sums = take(sum_rows * p.padded * 4);
  p.bytes = at;
  return p;
}

}  // namespace trt
