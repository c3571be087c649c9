// xent_stream.hpp -- the cross entropy's forward pass for a few tokens: a
// stream over W on the vector lanes.
//
// Each element of W meets a handful of products, so reading W once is the
// whole cost, and what counts is how it is read: a wave instruction takes 1
// KiB of one row, in order, as a plain streaming read does, where matrix-core
// operands would take 64 bytes from each of 16 rows.  A lane keeps elements
// 8l .. 8l + 7 of every 512 of its rows and multiplies them with the same
// elements of the tokens; the lanes' sums meet at the end.  A workgroup owns 64
// vocabulary entries, 8 to a wave; a token's maximum and sum of exponentials
// over the 64 go to `part` as the tile kernels' do (xent.hpp).
#pragma once

#include "layernorm.hpp"
#include "xent_args.hpp"

namespace trt {

// Measured for 65536 x 4096 bf16: 92 us for one or two tokens (5.8 TB/s), 106
// for four, against 120 on the matrix cores; for eight the products cost more
// than the better reads save (137 us), and the tile kernel takes those.
constexpr int kXentStreamWaves = 8, kXentStreamThreads = 64 * kXentStreamWaves;

// T tokens (rounded up; those past p.M read token 0 and are dropped).  A wave's
// rows go together: the tokens' elements are read and converted once for them.
template <int DT, int T>
__global__ __launch_bounds__(kXentStreamThreads) void xent_stream_kernel(XentStatsArgs p) {
  using C = RowChunk<DT>;
  constexpr int R = kXentStreamTile / kXentStreamWaves;
  __shared__ float logits[T][kXentStreamTile];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = blockIdx.x * kXentStreamTile;

  const int v0 = n0 + wave * R;
  const uint16_t *w[R], *x[T];
#pragma unroll
  for (int r = 0; r < R; ++r) w[r] = p.B + (int64_t)(v0 + r < p.N ? v0 + r : p.N - 1) * p.ldb;
#pragma unroll
  for (int t = 0; t < T; ++t) x[t] = p.A + (int64_t)(t < p.M ? t : 0) * p.lda;

  float acc[R][T];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < T; ++t) acc[r][t] = 0.f;

  // the width is a multiple of 8: a lane's 8 elements are in it or not
  u32x4 next[R], at[T];
  auto load = [&](int k) __attribute__((always_inline)) {
    const u32x4 zero = {0u, 0u, 0u, 0u};
    const bool in = k < p.K;
#pragma unroll
    for (int r = 0; r < R; ++r)
      next[r] = in ? __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(w[r] + k)) : zero;
#pragma unroll
    for (int t = 0; t < T; ++t) at[t] = in ? *reinterpret_cast<const u32x4*>(x[t] + k) : zero;
  };
  load(8 * lane);
  for (int k = 8 * lane; k - 8 * lane < p.K; k += 512) {
    u32x4 now[R], xs[T];
#pragma unroll
    for (int r = 0; r < R; ++r) now[r] = next[r];
#pragma unroll
    for (int t = 0; t < T; ++t) xs[t] = at[t];
    if (k - 8 * lane + 512 < p.K) load(k + 512);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float xe[T];
#pragma unroll
      for (int t = 0; t < T; ++t) xe[t] = C::elem(xs[t], e);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float we = C::elem(now[r], e);
#pragma unroll
        for (int t = 0; t < T; ++t) acc[r][t] = __builtin_fmaf(we, xe[t], acc[r][t]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const float z = wave_sum(acc[r][t]);
      if (lane == 0) logits[t][wave * R + r] = z;
    }
  __syncthreads();
  // a wave for each token
  if (wave >= T || wave >= p.M) return;
  const int n = n0 + lane;
  const float z = n < p.N ? logits[wave][lane] : -__builtin_inff();
  // the target's logit is kept apart from the sum
  const bool target = p.target[wave] == n;
  if (target) p.at[wave] = z;
  const float other = target ? -__builtin_inff() : z;
  float top = other;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, off));
  const float base = top == -__builtin_inff() ? 0.f : -top * kLog2E;
  const float sum = wave_sum(__builtin_amdgcn_exp2f(__builtin_fmaf(other, kLog2E, base)));
  if (lane == 0) p.part[(int64_t)blockIdx.x * p.ldp + wave] = f32x2{top, sum};
}

}  // namespace trt
