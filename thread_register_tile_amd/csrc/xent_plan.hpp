// xent_plan.hpp -- how a linear cross entropy is cut up, and its workspace:
// a function of the sizes alone.  Pure C++.
#pragma once

#include <stdint.h>

namespace trt {

// What the prep kernel leaves on the device for the others.
struct XentHead {
  int32_t live;    // tokens that take part
  float c;         // largest weight s_t (backward)
  float factor;    // c over G's scale
};

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
  p.part = take((vocab + 127) / 128 * tokens * 8);   // for either tile
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
  bool wide_g, wide_x, wide_w;   // 256-wide tiles for G, dX and dW
  int64_t slice, slices;         // of a piece's K in dX
  int64_t head, list, place, weight, info, x, g, sums;   // byte offsets
  int64_t bytes;
};

// The piece the library chooses: G of at most 2^28 elements (512 MiB), but
// 8192 entries at least, so that adding dX's sums (8 bytes per token, width
// and piece) stays small beside the piece's products; never 2 GiB or more.
constexpr int64_t xent_piece(int64_t tokens, int64_t vocab) {
  int64_t most = (int64_t(1) << 28) / tokens;
  if (most < 8192) most = 8192;
  const int64_t limit = ((int64_t(1) << 30) - 4096) / round_up(tokens, 256);
  if (most > limit) most = limit;
  if (most > kXentMaxPiece) most = kXentMaxPiece;
  if (most < 256) most = 256;
  most = most / 256 * 256;
  const int64_t pieces = (vocab + most - 1) / most;
  return round_up((vocab + pieces - 1) / pieces, 256);
}

constexpr XentBwdPlan xent_bwd_plan(int64_t tokens, int64_t vocab, int64_t width, int64_t piece) {
  XentBwdPlan p{};
  p.piece = piece > 0 ? piece : xent_piece(tokens, vocab);
  if (p.piece > round_up(vocab, 64)) p.piece = round_up(vocab, 64);
  p.pieces = (vocab + p.piece - 1) / p.piece;
  p.padded = round_up(width, 8);
  p.wide_g = xent_wide(tokens, p.piece);
  p.wide_w = xent_wide(p.piece, width);
  // dX has few tiles where tokens or width are small: its K is cut into
  // slices of at least 512 until there are about two tiles for every compute
  // unit (one of the 256-wide ones)
  p.wide_x = tokens > 192 && width > 192;
  const int64_t tile = p.wide_x ? 256 : 128;
  const int64_t tiles = ((tokens + tile - 1) / tile) * ((width + tile - 1) / tile);
  const int64_t want = (p.wide_x ? 256 : 512) / tiles;
  int64_t slices = want;
  if (slices > p.piece / 512) slices = p.piece / 512;
  if (slices < 1) slices = 1;
  p.slice = round_up((p.piece + slices - 1) / slices, 64);
  p.slices = (p.piece + p.slice - 1) / p.slice;
  int64_t at = 0;
  auto take = [&](int64_t n) { const int64_t o = at; at += round_up(n, 256); return o; };
  p.head = take(sizeof(XentHead));
  p.list = take(tokens * 4);
  p.place = take(tokens * 4);
  p.weight = take(tokens * 4);
  p.info = take(tokens * 16);
  p.x = take(tokens * p.padded * 2);
  p.g = take(tokens * p.piece * 2);
  p.sums = take(p.slices * tokens * p.padded * 4);
  p.bytes = at;
  return p;
}

}  // namespace trt
