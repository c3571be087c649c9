// layernorm.hpp -- the layer norm over the rows of a matrix, forward and
// backward, for gfx950.
//
//   mu = mean(x), v = mean((x - mu)^2), r = 1 / sqrt(v + eps), h = (x - mu) r
//   forward:   y = h gamma + beta
//   backward:  u = dy gamma,  dx = r (u - mean(u) - h mean(u h)),
//              dgamma = sum over rows of dy h,  dbeta = sum over rows of dy
//
// What bounds it: memory.  The forward pass reads x and writes y once, the
// backward pass reads x and dy and writes dx once; a row lives in registers
// from its load to its store, so the several sums over it cost no traffic.
// The backward pass therefore takes no saved statistics: it forms them again
// from the row it has to read anyway.  Measured on 16384 rows of 8192 bf16
// elements: 91 us forward (5.9 TB/s), 151 backward (5.3 TB/s); a large copy
// reaches 5.2, a streaming read 6.4.
//
// Cooperation: a row is cut into 16-byte chunks, chunk c going to lane
// c mod 64W of the row's W waves, iteration c div 64W ("My Triton From
// Scratch, Part 12: CUDA Tile Layouts", section "Cooperative tile layouts").
// W and the chunks per lane K follow from the row's length alone (kern_layernorm.hip).
// A workgroup walks rows in strides of the grid and loads its next row before
// it works on the present one.
//
// Numerics: sums in binary32.  The first sum gives a mean m accurate to a few
// units in the last place of the largest values; the second round sums d = x - m and
// d^2, and the mean of d corrects both the mean and the variance
// (mean = m + dbar, v = mean(d^2) - dbar^2, where dbar is only m's rounding
// error, so nothing cancels): rows whose mean is large against their spread
// lose no accuracy to the rounding of the mean.
#pragma once

#include "gemm_kernel.hpp"
#include "norm.hpp"
#include "rowchunk.hpp"

namespace trt {

// VEC parameters (gamma or beta) from element i of p, of type PDT; `absent`
// where p is null, zero past n.
template <int PDT, int VEC>
__device__ __forceinline__ void load_params(const void* p, int i, int n, float absent,
                                            float (&v)[VEC]) {
  using C = RowChunk<PDT>;
#pragma unroll
  for (int c = 0; c < VEC; c += C::VEC) {
    u32x4 w = {0u, 0u, 0u, 0u};
    if (p && i + c < n) w = C::load_shared(p, i + c, n);
#pragma unroll
    for (int e = 0; e < C::VEC; ++e) v[c + e] = p ? C::elem(w, e) : absent;
  }
}

// f(e) for the elements e of a chunk that lie in the row, `left` of which
// remain from the chunk's first element on.  Only a row's last chunk can be
// partial; its tests stay inside its branch (the empty asm hides that they are
// the same for every row), where hoisted ones would each hold a pair of scalar
// registers across the loop over rows.
template <int VEC, class F>
__device__ __forceinline__ void for_elems(int left, F&& f) {
  if (left >= VEC) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) f(e);
  } else if (left > 0) {
    int some = left;
    asm volatile("" : "+v"(some));
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (e < some) f(e);
  }
}

// Keeps a row in its packed form between two uses: without it the compiler
// carries the elements' binary32 values, twice the registers of a 16-bit row.
template <int K>
__device__ __forceinline__ void keep_packed(u32x4 (&v)[K]) {
#pragma unroll
  for (int k = 0; k < K; ++k) asm volatile("" : "+v"(v[k]));
}

// x as a rounded value of its own: the compiler may otherwise fold the product
// that made it into later sums, in one place and not in another, and the
// correction of the mean would then correct a different number than is used.
__device__ __forceinline__ float rounded(float x) {
  asm volatile("" : "+v"(x));
  return x;
}

// 1 / sqrt(v + eps), where rounding may leave v a little below zero.  NaN stays
// NaN: v is infinity less infinity where the squares of the deviations and of the
// mean's correction are beyond binary32, and no finite value may come of that
// (the maximum of v and 0 would be 0).
__device__ __forceinline__ float norm_rstd(float v, float eps) {
  return 1.f / sqrtf((v < 0.f ? 0.f : v) + eps);
}

// Sum over the wave's 64 lanes, the same bits in every lane: within the quads,
// eights and rows of 16 by data-parallel moves, then across the four rows.
__device__ __forceinline__ float wave_sum(float v) {
  auto move = [](float x, auto ctrl) {
    return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), ctrl.value, 0xF, 0xF, true));
  };
  v += move(v, std::integral_constant<int, 0xB1>{});   // quad lanes 1 0 3 2
  v += move(v, std::integral_constant<int, 0x4E>{});   // quad lanes 2 3 0 1
  v += move(v, std::integral_constant<int, 0x141>{});  // mirror of 8 lanes
  v += move(v, std::integral_constant<int, 0x140>{});  // mirror of 16 lanes
  v += __shfl_xor(v, 16);
  v += __shfl_xor(v, 32);
  return v;
}

// Sums of N values over the W waves of a row.  W > 1: the waves meet in LDS,
// in the slots of `buf` from `first` on (two turns used alternately, so one
// barrier a turn suffices: a wave writes a turn's slots again only after the
// next turn's barrier, which every wave reaches with its reads of the first
// turn done).  Every wave of the workgroup calls it.
template <int W, int N>
__device__ __forceinline__ void row_sums(float (&v)[N], float (*buf)[16][4], int& turn, int wave,
                                         int first) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if constexpr (W > 1) {
    static_assert(W <= 16 && N <= 4, "one slot per wave and value");
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) buf[turn][first + wave][i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float s = buf[turn][first][i];
#pragma unroll
      for (int w = 1; w < W; ++w) s += buf[turn][first + w][i];
      v[i] = s;
    }
    turn ^= 1;
  }
}

// Threads of a workgroup whose rows are W waves wide, and its rows at a time.
template <int W>
struct NormShape {
  static constexpr int THREADS = W == 1 ? 256 : 64 * W;
  static constexpr int GROUPS = THREADS / (64 * W);
};

// KEEP: gamma and beta stay in registers over the rows (rows of more than 32
// KiB have none left for them and read them again, from the L2).
template <int DT, int PDT, int W, int K>
__global__ __launch_bounds__(NormShape<W>::THREADS) void layernorm_kernel(NormArgs a) {
  using C = RowChunk<DT>;
  constexpr int VEC = C::VEC, LANES = 64 * W, GROUPS = NormShape<W>::GROUPS;
  constexpr bool KEEP = K <= 3;
  __shared__ float buf[2][16][4];
  // the wave's index in a scalar register: row addresses are then scalar too
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wave = w % W, grp = w / W;
  const int me = 64 * wave + (threadIdx.x & 63);
  const int n = a.cols;
  const float inv = 1.f / (float)a.cols;
  const int64_t step = (int64_t)gridDim.x * GROUPS;
  int64_t r = (int64_t)blockIdx.x * GROUPS + grp;
  int turn = 0;

  auto col = [&](int k) { return VEC * (me + k * LANES); };
  auto load = [&](u32x4 (&v)[K], int64_t row) {
    const char* p = static_cast<const char*>(a.x) + row * a.ldx * (int64_t)sizeof(typename C::Elem);
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = col(k) < n ? C::load(p, col(k), n) : u32x4{0u, 0u, 0u, 0u};
  };

  u32x4 next[K];
  if (r < a.rows) load(next, r);
  float gamma[KEEP ? K : 1][VEC], beta[KEEP ? K : 1][VEC];
  auto params = [&](int k, int to) {
    load_params<PDT>(a.gamma, col(k), n, 1.f, gamma[to]);
    load_params<PDT>(a.beta, col(k), n, 0.f, beta[to]);
  };
  if constexpr (KEEP)
#pragma unroll
    for (int k = 0; k < K; ++k) params(k, k);
  for (; r < a.rows; r += step) {
    u32x4 x[K];
#pragma unroll
    for (int k = 0; k < K; ++k) x[k] = next[k];
    if (r + step < a.rows) load(next, r + step);
    float s[1] = {0.f};
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < VEC; ++e) s[0] += C::elem(x[k], e);
    row_sums<W, 1>(s, buf, turn, wave, W * grp);
    keep_packed(x);
    const float m = rounded(s[0] * inv);
    float q[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < K; ++k)
      for_elems<VEC>(n - col(k), [&](int e) {
        const float d = C::elem(x[k], e) - m;
        q[0] += d;
        q[1] += d * d;
      });
    row_sums<W, 2>(q, buf, turn, wave, W * grp);
    keep_packed(x);
    const float dbar = q[0] * inv;
    const float rstd = norm_rstd(q[1] * inv - dbar * dbar, a.eps);
    char* p = static_cast<char*>(a.out) + r * a.ldo * (int64_t)sizeof(typename C::Elem);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (col(k) >= n) continue;
      if constexpr (!KEEP) params(k, 0);
      float y[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        y[e] = ((C::elem(x[k], e) - m) - dbar) * rstd * gamma[KEEP ? k : 0][e] + beta[KEEP ? k : 0][e];
      C::store(p, col(k), n, y);
    }
  }
}

// The backward pass.  The row's four sums after the mean -- d, d^2, u and u d
// -- come in one round: with dbar as above, sum(u h) = r (sum(u d) - dbar
// sum(u)).  Every lane keeps the partial sums of dgamma and dbeta of its own
// columns in registers over all its rows, in row order; the workgroup writes
// them to its slice of `part` at the end, and norm_params_kernel adds the
// slices in order.  The grid is fixed by the sizes (norm_slices), so the sums'
// order is too: the results repeat bit for bit.
// A workgroup is 16 or 8 waves, a row to each W of them, and there is one to a
// compute unit: the fewer slices, the fewer bytes beside the rows' own (with
// workgroups of one row, two to a unit, the slices were 8 % of the traffic of
// 16384 rows of 8192, and 8 % of the time).
// AHEAD, KEPT: the next row is loaded ahead, and gamma kept in registers, where
// a lane's packed row and sums leave room for it (2000 rows of 16384 bf16
// elements: 87 us without, 66 with).
// (Too few rows to give every unit one of 16 waves take the forward pass's
// smaller ones.)
template <int DT, int PDT, int W, int K, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void layernorm_bwd_kernel(NormArgs a) {
  using C = RowChunk<DT>;
  constexpr int VEC = C::VEC, LANES = 64 * W, GROUPS = WAVES / W;
  constexpr int ROOM = WAVES == 16 ? 84 : 176;   // of 128 and 256 registers
  constexpr int HELD = K * (8 + 2 * VEC);        // x, dy and the sums
  constexpr bool AHEAD = HELD + 8 * K <= ROOM, KEPT = AHEAD && HELD + 8 * K + VEC * K <= ROOM;
  __shared__ float buf[2][16][4];
  __shared__ float fold[GROUPS > 1 ? GROUPS : 1][GROUPS > 1 ? LANES * VEC * K : 1];
  // the wave's index in a scalar register: row addresses are then scalar too
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wave = w % W, grp = w / W;
  int me = 64 * wave + (threadIdx.x & 63);
  const int n = a.cols;
  const float inv = 1.f / (float)a.cols;
  const int64_t step = (int64_t)gridDim.x * GROUPS;
  int64_t r = (int64_t)blockIdx.x * GROUPS + grp;
  int turn = 0;

  auto col = [&](int k) { return VEC * (me + k * LANES); };
  auto load = [&](u32x4 (&v)[K], const void* base, int64_t ld, int64_t row) {
    const char* p = static_cast<const char*>(base) + row * ld * (int64_t)sizeof(typename C::Elem);
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = col(k) < n ? C::load(p, col(k), n) : u32x4{0u, 0u, 0u, 0u};
  };

  u32x4 nx[AHEAD ? K : 1], ny[AHEAD ? K : 1];
  float kept[KEPT ? K : 1][VEC];
  if constexpr (AHEAD) {
#pragma unroll
    for (int k = 0; k < K; ++k) nx[k] = ny[k] = u32x4{0u, 0u, 0u, 0u};
    if (r < a.rows) {
      load(nx, a.x, a.ldx, r);
      load(ny, a.dy, a.lddy, r);
    }
  }
  if constexpr (KEPT) {
#pragma unroll
    for (int k = 0; k < K; ++k) load_params<PDT>(a.gamma, col(k), n, 1.f, kept[k]);
  }
  float dg[K][VEC], db[K][VEC];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int e = 0; e < VEC; ++e) dg[k][e] = db[k][e] = 0.f;

  // every wave takes as many turns as the workgroup's first row needs; one
  // past the last row works on zeros and keeps nothing
  for (int64_t r0 = (int64_t)blockIdx.x * GROUPS; r0 < a.rows; r0 += step, r += step) {
    // addresses and column tests made anew for each pass over a row: kept they
    // would take a third of the registers
    if constexpr (K * VEC > 32) asm volatile("" : "+v"(me));
    const bool live = r < a.rows;
    u32x4 x[K], y[K];
    if constexpr (AHEAD) {
#pragma unroll
      for (int k = 0; k < K; ++k) x[k] = nx[k], y[k] = ny[k];
      if (r + step < a.rows) {
        load(nx, a.x, a.ldx, r + step);
        load(ny, a.dy, a.lddy, r + step);
      }
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) x[k] = y[k] = u32x4{0u, 0u, 0u, 0u};
      if (live) {
        load(x, a.x, a.ldx, r);
        load(y, a.dy, a.lddy, r);
      }
    }
    float s[1] = {0.f};
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < VEC; ++e) s[0] += C::elem(x[k], e);
    row_sums<W, 1>(s, buf, turn, wave, W * grp);
    keep_packed(x);
    const float m = rounded(s[0] * inv);
    auto gamma_of = [&](int k, float (&g)[VEC]) {
      if constexpr (KEPT) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) g[e] = kept[k][e];
      } else {
        load_params<PDT>(a.gamma, col(k), n, 1.f, g);
      }
    };
    if constexpr (K * VEC > 32) asm volatile("" : "+v"(me));
    float q[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float g[VEC];
      gamma_of(k, g);
      for_elems<VEC>(n - col(k), [&](int e) {
        const float d = C::elem(x[k], e) - m;
        const float u = C::elem(y[k], e) * g[e];
        q[0] += d;
        q[1] += d * d;
        q[2] += u;
        q[3] += u * d;
      });
    }
    row_sums<W, 4>(q, buf, turn, wave, W * grp);
    keep_packed(x);
    keep_packed(y);
    const float dbar = q[0] * inv;
    const float rstd = norm_rstd(q[1] * inv - dbar * dbar, a.eps);
    const float c1 = q[2] * inv;
    const float c2 = rstd * (q[3] * inv - dbar * c1);   // mean(u h)
    if (!live) continue;
    if constexpr (K * VEC > 32) asm volatile("" : "+v"(me));
    char* p = static_cast<char*>(a.out) + r * a.ldo * (int64_t)sizeof(typename C::Elem);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float g[VEC], dx[VEC];
      gamma_of(k, g);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float dy = C::elem(y[k], e);
        const float h = ((C::elem(x[k], e) - m) - dbar) * rstd;
        dx[e] = rstd * ((dy * g[e] - c1) - h * c2);
        dg[k][e] += dy * h;
        db[k][e] += dy;
      }
      if (col(k) < n) C::store(p, col(k), n, dx);
    }
  }
  if (!a.part) return;
  float* mine = a.part + (int64_t)blockIdx.x * 2 * n;
#pragma unroll
  for (int what = 0; what < 2; ++what) {
    float (&acc)[K][VEC] = what ? db : dg;
    if constexpr (GROUPS > 1) {
      // the groups' sums of a column, added in group order
      __syncthreads();
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < VEC; ++e) fold[grp][VEC * (me + k * LANES) + e] = acc[k][e];
      __syncthreads();
      for (int c = threadIdx.x; c < n; c += 64 * WAVES) {
        float t = fold[0][c];
#pragma unroll
        for (int q = 1; q < GROUPS; ++q) t += fold[q][c];
        mine[what * n + c] = t;
      }
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (col(k) + e < n) mine[what * n + col(k) + e] = acc[k][e];
    }
  }
}

// dgamma and dbeta from the workgroups' partial sums.  A workgroup adds 64
// columns of one of the two: each of its 16 waves takes every 16th slice, in
// order, and the waves' sums are added in wave order.
struct NormParamsArgs {
  const float* part;
  void *dgamma, *dbeta;   // either may be null
  int32_t slices, cols;
};

constexpr int kNormParamsWaves = 16;

template <int PDT>
__global__ __launch_bounds__(64 * kNormParamsWaves) void norm_params_kernel(NormParamsArgs a) {
  __shared__ float sum[kNormParamsWaves][64];
  void* out = blockIdx.y ? a.dbeta : a.dgamma;
  if (!out) return;   // the whole workgroup
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  float s = 0.f;
  if (c < a.cols) {
    const float* p = a.part + (int64_t)blockIdx.y * a.cols + c;
#pragma unroll 8
    for (int i = wave; i < a.slices; i += kNormParamsWaves) s += p[(int64_t)i * 2 * a.cols];
  }
  sum[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < a.cols) {
    float t = sum[0][lane];
#pragma unroll
    for (int w = 1; w < kNormParamsWaves; ++w) t += sum[w][lane];
    Out<PDT>::st(out, c, t);
  }
}

}  // namespace trt
