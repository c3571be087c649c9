// xent_rows.hpp -- the cross entropy's small kernels: the list of live tokens,
// the join of a row's pairs, X' and dX's last step.  xent.hpp has the whole
// picture.
#pragma once

#include "rowchunk.hpp"
#include "xent_args.hpp"

namespace trt {

// The list of live tokens, in order, by one workgroup: each thread counts 8
// tokens of a block of 8192, waves scan their threads' counts by shuffles and
// the workgroup its waves' through LDS.  Backward, a token whose upstream
// gradients are both zero is not live either, and the kernel takes c, the
// largest finite s_t.  Forward, it writes the ignored tokens' results.
constexpr int kPrepThreads = 1024, kPrepEach = 8;

// s_t: zero for a token without weight, NaN if either gradient is (the maximum
// of a number and NaN would be the number; NaN in dl is in both as well).
__device__ __forceinline__ float xent_weight(const XentPrepArgs& a, int64_t t, float& dl, float& both) {
  dl = a.dloss[t * a.inc_dloss];
  both = a.dlse ? dl + a.dlse[t * a.inc_dlse] : dl;
  return both == both ? __builtin_fmaxf(__builtin_fabsf(dl), __builtin_fabsf(both)) : both;
}

// (BACKWARD as a template argument, so that the loads of a thread's tokens are
// all issued before the first of them is used.)
template <bool BACKWARD>
__global__ __launch_bounds__(kPrepThreads) void xent_prep_kernel(XentPrepArgs a) {
  __shared__ int count[16];
  __shared__ float top[16];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  int base = 0;
  float c = 0.f;
  for (int64_t t0 = 0; t0 < a.tokens; t0 += kPrepThreads * kPrepEach) {
    const int64_t first = t0 + (int64_t)t * kPrepEach;
    int64_t target[kPrepEach];
    float s[kPrepEach];
#pragma unroll
    for (int e = 0; e < kPrepEach; ++e) {
      const int64_t tok = first + e < a.tokens ? first + e : a.tokens - 1;
      target[e] = a.target[tok];
      float dl, both;
      s[e] = BACKWARD ? xent_weight(a, tok, dl, both) : 1.f;
    }
    uint32_t keep = 0;
#pragma unroll
    for (int e = 0; e < kPrepEach; ++e) {
      const bool live = first + e < a.tokens && target[e] != a.ignore && s[e] != 0.f;
      keep |= live ? 1u << e : 0u;
      // (of the finite ones: a token whose gradient is not takes its own row of dX
      // with it, and dW, but no other row)
      c = live && s[e] <= __FLT_MAX__ ? __builtin_fmaxf(c, s[e]) : c;
    }
    int upto = __popc(keep);   // inclusive count over the wave's lanes
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int v = __shfl_up(upto, off);
      if (lane >= off) upto += v;
    }
    if (lane == 63) count[wave] = upto;
    __syncthreads();
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) {
      before += w < wave ? count[w] : 0;
      all += count[w];
    }
    int at = base + before + upto - __popc(keep);
#pragma unroll
    for (int e = 0; e < kPrepEach; ++e) {
      const int64_t tok = first + e;
      if (tok >= a.tokens) break;
      const bool live = (keep >> e) & 1u;
      if (BACKWARD) a.place[tok] = live ? at : -1;
      if (live) {
        if (!BACKWARD) a.want[at] = target[e] >= 0 && target[e] < a.vocab ? (int32_t)target[e] : -1;
        a.list[at++] = (int32_t)tok;
      } else if (!BACKWARD) {
        a.loss[tok] = 0.f;
        a.lse[tok] = 0.f;
      }
    }
    base += all;
    __syncthreads();
  }
  if (BACKWARD) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) c = __builtin_fmaxf(c, __shfl_xor(c, off));
    if (lane == 0) top[wave] = c;
    __syncthreads();
    if (wave == 0) {
      c = top[lane & 15];
#pragma unroll
      for (int off = 8; off >= 1; off >>= 1) c = __builtin_fmaxf(c, __shfl_xor(c, off));
      // the number of slices of dX's product: lane s - 1 weighs s of them, the
      // least cost and of those the least number is taken
      const uint32_t tiles = xent_input_tiles((int64_t)base << a.halves, a.width, a.wide != 0);
      const uint32_t mine = lane < kXentMostSlices ? lane + 1 : 1;
      uint64_t cost = xent_slice_cost(mine, tiles, a.k, a.wide != 0);
      uint32_t best = mine;
#pragma unroll
      for (int off = 32; off >= 1; off >>= 1) {
        const uint64_t other = __shfl_xor(cost, off);
        const uint32_t its = __shfl_xor(best, off);
        if (other < cost || (other == cost && its < best)) cost = other, best = its;
      }
      // (the quotients by c and c over G's scale stay normal numbers)
      c = __builtin_fmaxf(c, 0x1p-110f);
      if (lane == 0) {
        const uint32_t slice = xent_slice(best, a.k);
        *a.head = XentHead{base, c, c / a.scale, (int32_t)slice, (int32_t)((a.k + slice - 1) / slice)};
      }
    }
  } else if (t == 0) {
    a.head->live = base;
  }
}

template <int R>
__global__ __launch_bounds__(256) void xent_combine_kernel(XentCombineArgs a) {
  constexpr int EACH = 256 / R;
  __shared__ f32x2 pairs[EACH][R];
  const int r = threadIdx.x % R, j = threadIdx.x / R;
  const int rows = a.head ? a.head->live : a.tokens;
  const int64_t m = (int64_t)blockIdx.x * R + r;
  if ((int64_t)blockIdx.x * R >= rows) return;   // the whole workgroup
  float top = -__builtin_inff(), sum = 0.f;
  auto join = [&](f32x2 q) {
    const float up = __builtin_fmaxf(top, q[0]);
    const float base = up == -__builtin_inff() ? 0.f : up;
    sum = sum * __builtin_amdgcn_exp2f((top - base) * kLog2E) +
          q[1] * __builtin_amdgcn_exp2f((q[0] - base) * kLog2E);
    top = up;
  };
  if (m < rows) {
    const f32x2* p = a.part + m;
#pragma unroll 4
    for (int i = j; i < a.tiles; i += EACH) join(p[(int64_t)i * a.ldp]);
  }
  pairs[j][r] = f32x2{top, sum};
  __syncthreads();
#pragma unroll
  for (int half = EACH / 2; half >= 1; half >>= 1) {
    if (j < half) {
      join(pairs[j + half][r]);
      pairs[j][r] = f32x2{top, sum};
    }
    __syncthreads();
  }
  if (j != 0 || m >= rows) return;
  const int64_t tok = a.list ? a.list[m] : m;
  const int64_t target = a.target[tok];
  if (target == a.ignore) {
    a.loss[tok] = 0.f;
    a.lse[tok] = 0.f;
    return;
  }
  // sum: over every entry but the target (top may be the target's).  A target
  // outside the vocabulary has no loss: NaN, where it can be seen
  const float inf = __builtin_inff(), nan = __builtin_nanf("");
  const bool known = target >= 0 && target < a.vocab;
  const float z = known ? a.at[m] : -inf;
  const float up = __builtin_fmaxf(top, z);
  const float base = up == -inf ? 0.f : up;
  a.lse[tok] = up + logf(sum * expf(top - base) + expf(z - base));
  const float d = top - z;
  float loss;
  if (top == -inf) loss = sum == 0.f && z > -inf && z < inf ? 0.f : nan;   // no other entry
  else if (d < 60.f) loss = log1pf(sum * expf(d));
  else loss = d + logf(sum + expf(-d));
  a.loss[tok] = known && z < inf ? loss : nan;
}

// The live tokens' rows, packed with a row of `ld` elements (zero past the
// width), and what the gradient's epilogue needs of each token.
template <int DT>
__global__ __launch_bounds__(256) void xent_rows_kernel(XentRowsArgs a) {
  using C = RowChunk<DT>;
  const int m = blockIdx.x;
  if (m >= a.prep.head->live) return;   // the whole workgroup
  const int tok = a.prep.list[m];
  if (threadIdx.x == 0) {
    float dl, both;
    xent_weight(a.prep, tok, dl, both);
    const float c = a.prep.head->c;   // never zero
    const int64_t target = a.prep.target[tok];
    const bool known = target >= 0 && target < a.vocab;
    // a target outside the vocabulary: a NaN row, where it can be seen.  The
    // quotients are exactly 1 or -1 for equal dloss and no dlse
    a.info[m] = XentRow{known ? both / c : __builtin_nanf(""), dl / c, a.lse[tok] * kLog2E,
                        known ? (int32_t)target : -1};
  }
  const uint16_t* src = a.x + (int64_t)tok * a.ldx;
  uint16_t* dst = a.out + ((int64_t)m << a.prep.halves) * a.ld;
  for (int i = C::VEC * threadIdx.x; i < a.ld; i += C::VEC * 256) {
    u32x4 v = {0u, 0u, 0u, 0u};
    if (i < a.width) v = C::load(src, i, a.width);
    *reinterpret_cast<u32x4*>(dst + i) = v;
    if (a.prep.halves) *reinterpret_cast<u32x4*>(dst + a.ld + i) = v;
  }
}

// dX from the slices' sums: a row is c times the sum over the slices in order
// (with halves, of its two rows in each), or zeros for a token that is not live.
template <int OT>
__global__ __launch_bounds__(256) void xent_input_finish_kernel(XentInputFinishArgs a) {
  using O = Out<OT>;
  const int64_t t = blockIdx.x;
  const int m = a.place[t];
  const float f = a.head->factor;
  const int slices = a.head->slices;
  const int64_t stride = xent_sum_rows((int64_t)a.head->live << a.halves) * a.ld;
  const int step = 4 * blockDim.x * gridDim.y;
  for (int i = 4 * (blockIdx.y * blockDim.x + threadIdx.x); i < a.width; i += step) {
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
    if (m >= 0) {   // the sums' rows are padded to whole eights
      const float* p = a.sums + ((int64_t)m << a.halves) * a.ld + i;
      if (a.halves) {
#pragma unroll 8
        for (int s = 0; s < slices; ++s)
          v += *reinterpret_cast<const f32x4*>(p + s * stride) + *reinterpret_cast<const f32x4*>(p + s * stride + a.ld);
      } else {
#pragma unroll 8
        for (int s = 0; s < slices; ++s) v += *reinterpret_cast<const f32x4*>(p + s * stride);
      }
      v *= f;
    }
    const int64_t at = t * a.lddx + i;
    if (a.vec && i + 4 <= a.width) {
      const float y[4] = {v[0], v[1], v[2], v[3]};
      O::st4(a.dx, at, O::pack(y));
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (i + e < a.width) O::st(a.dx, at + e, v[e]);
    }
  }
}

}  // namespace trt
