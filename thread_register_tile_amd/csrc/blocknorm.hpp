// blocknorm.hpp -- what lies between two blocks of a residual model in one pass,
// and its gradients, for gfx950.
//
//   N(x) = (x - mu) rstd  (mu: the row's mean, or 0 for the root mean square
//   norm), rstd = 1 / sqrt(mean((x - mu)^2) + eps)
//   u  = N(y) post_gamma + post_beta, or y itself
//   r' = alpha r + gate u
//   h  = N(r') gamma + beta
// backward, with rhat = N(r'), yhat = N(y):
//   t = dh gamma,   e = dr' + rstd_r (t - mean(t) - rhat mean(t rhat))
//   dr = alpha e,   s = gate post_gamma e
//   dy = rstd_y (s - mean(s) - yhat mean(s yhat)), or gate e without the norm
//   dgate = sum of e u,  dpost_gamma = sum of gate e yhat,  dpost_beta = sum of gate e,
//   dgamma = sum of dh rhat,  dbeta = sum of dh
// (mean(t) and mean(s) only where the mean was taken out).
//
// What bounds it: memory.  The forward pass reads r and y and writes r' and h, the
// backward pass reads dh, dr', r' and y and writes dr and dy, each once: a row
// lives in registers from its load to its store, as in the layer norm
// (layernorm.hpp, whose row cutting, sums and corrected mean this uses).  The
// stream is kept in binary32 between the sum and the second norm, so h has one
// rounding.  Backward, r' and y may be 8-bit rows (act8.hpp): they are restored
// in registers, 33/32 bytes an element instead of two.
//
// A gate row covers `span` rows.  Its gradient, and post_gamma's and post_beta's,
// all come of two sums over its rows, E0 of e and E1 of e yhat:
//   dgate = post_gamma E1 + post_beta E0,  dpost_gamma = sum of gate E1, ...
// so a lane keeps four running sums per column whatever there is to return, in
// row order; a workgroup's rows lie in one gate row, it writes its four sums at
// the end, and block_params_kernel adds the workgroups' in order: results repeat
// bit for bit.  A gate of its own for every row has its gradient written with
// the row, and is multiplied into the sums.
#pragma once

#include "act8.hpp"
#include "blocknorm_args.hpp"
#include "layernorm.hpp"

namespace trt {

// VEC values from element i of p, binary32 or of the rows' type.
template <int DT, int VEC>
__device__ __forceinline__ void load_values(const void* p, bool wide, int i, int n, float absent, float (&v)[VEC]) {
  if (DT == DT_F32 || wide) load_params<DT_F32>(p, i, n, absent, v);
  else load_params<DT>(p, i, n, absent, v);
}

__device__ __forceinline__ const void* row_of(const void* p, bool wide, int64_t row, int64_t ld, int narrow) {
  return static_cast<const char*>(p) + row * ld * (wide ? 4 : narrow);
}

// Sums of several values at once.  Each step that halves the lanes of one value's
// sum takes two values into one register, so N values cost as many moves as two
// or three alone: lanes 32 apart (permlane32_swap(x, y) leaves both halves of x in
// the lower lanes and both of y in the upper), then 16, then 8; and four steps
// within the lanes that are left.  Every step's order is fixed, so all waves have
// the same bits.
__device__ __forceinline__ float swap_add32(float x, float y) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(y), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float swap_add16(float x, float y) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(y), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
template <int CTRL>
__device__ __forceinline__ float dpp_add(float x) {
  return x + __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), CTRL, 0xF, 0xF, true));
}
constexpr int kRowRor = 0x120;   // rotation within 16 lanes

// Lanes 64 / N i .. 64 / N (i + 1) - 1 get the wave's sum of v[i]; N: 1, 2, 4 or 8.
template <int N>
__device__ __forceinline__ float wave_fold(const float (&v)[N]) {
  static_assert(N == 1 || N == 2 || N == 4 || N == 8, "halves of the lanes");
  float x;
  if constexpr (N == 8) {
    float h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = swap_add32(v[i], v[i + 4]);
    const float a = swap_add16(h[0], h[2]), b = swap_add16(h[1], h[3]);
    const float a8 = dpp_add<kRowRor + 8>(a), b8 = dpp_add<kRowRor + 8>(b);
    x = threadIdx.x & 8 ? b8 : a8;
  } else {
    if constexpr (N == 4) x = swap_add16(swap_add32(v[0], v[2]), swap_add32(v[1], v[3]));
    else if constexpr (N == 2) x = swap_add32(v[0], v[1]);
    else x = swap_add32(v[0], v[0]);
    if constexpr (N < 4) x = swap_add16(x, x);
    x = dpp_add<kRowRor + 8>(x);
  }
  x = dpp_add<0x141>(x);    // mirror of 8 lanes
  x = dpp_add<0x4E>(x);     // quad lanes 2 3 0 1
  return dpp_add<0xB1>(x);  // quad lanes 1 0 3 2
}

__device__ __forceinline__ float lane_value(float x, int lane) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), lane));
}

// Sums of N values over the W waves of a row.  W > 1: the waves meet in LDS, in
// the slots of `buf` from wave `first` on (two turns used alternately, so one
// barrier a turn suffices: see row_sums).  Every wave of the workgroup calls it.
template <int W, int N>
__device__ __forceinline__ void meet(float (&v)[N], float (*buf)[128], int& turn, int wave, int first) {
  static_assert(W <= 16 && N <= 8, "one slot per wave and value");
  constexpr int M = N <= 2 ? N : N <= 4 ? 4 : 8, EACH = 64 / M;
  const int lane = threadIdx.x & 63;
  float all[M];
#pragma unroll
  for (int i = 0; i < M; ++i) all[i] = i < N ? v[i] : 0.f;
  float x = wave_fold<M>(all);
  if constexpr (W == 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lane_value(x, EACH * i);
  } else {
    if (lane % EACH == 0) buf[turn][(first + wave) * M + lane / EACH] = x;
    __syncthreads();
    // lane l: value l mod M of wave l div M
    const float* from = &buf[turn][first * M];
    x = 0.f;
    if (W * M >= 64 || lane < W * M) x = from[lane];
    if constexpr (W * M > 64)
      if (lane < W * M - 64) x += from[64 + lane];
    if constexpr (M <= 8) x = dpp_add<kRowRor + 8>(x);
    if constexpr (M <= 4) x = dpp_add<kRowRor + 4>(x);
    if constexpr (M <= 2) x = dpp_add<kRowRor + 2>(x);
    if constexpr (M <= 1) x = dpp_add<kRowRor + 1>(x);
    x = swap_add16(x, x);
    x = swap_add32(x, x);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = lane_value(x, i);
    turn ^= 1;
  }
}

// EACH: a gate of its own for every row, loaded with it; otherwise gate and
// post norm's parameters are one product, made again when the gate row changes.
// KEEP: the vectors stay in registers (of 16 waves to a row none are left).
template <int DT, int W, int K, bool EACH>
__global__ __launch_bounds__(NormShape<W>::THREADS) void block_norm_kernel(BlockNormArgs a) {
  using C = RowChunk<DT>;
  constexpr int VEC = C::VEC, LANES = 64 * W, GROUPS = NormShape<W>::GROUPS, E = sizeof(typename C::Elem);
  constexpr bool KEEP = W < 16;
  __shared__ float buf[2][128];
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
  auto load = [&](u32x4 (&v)[K], const SavedRows& x, int64_t row) {
    const char* p = static_cast<const char*>(x.x) + row * x.ld * (int64_t)E;
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = col(k) < n ? C::load(p, col(k), n) : u32x4{0u, 0u, 0u, 0u};
  };

  // u1 yhat + u0 is what the gate multiplies (EACH) or what joins the stream
  float u1[KEEP ? K : 1][VEC], u0[KEEP ? K : 1][VEC], gamma[KEEP ? K : 1][VEC], beta[KEEP ? K : 1][VEC];
  auto post = [&](int k, int to, int64_t gate_row) {
    load_values<DT>(a.post ? a.post_gamma : nullptr, a.wide_params, col(k), n, 1.f, u1[to]);
    load_values<DT>(a.post ? a.post_beta : nullptr, a.wide_params, col(k), n, 0.f, u0[to]);
    if (!EACH && a.gate) {
      float g[VEC];
      load_values<DT>(row_of(a.gate, a.wide_gate, gate_row, a.ldg, E), a.wide_gate, col(k), n, 1.f, g);
#pragma unroll
      for (int e = 0; e < VEC; ++e) u1[to][e] *= g[e], u0[to][e] *= g[e];
    }
  };
  auto pre = [&](int k, int to) {
    load_values<DT>(a.gamma, a.wide_params, col(k), n, 1.f, gamma[to]);
    load_values<DT>(a.beta, a.wide_params, col(k), n, 0.f, beta[to]);
  };

  u32x4 nr[K], ny[K];
  if (r < a.rows) {
    load(nr, a.r, r);
    load(ny, a.y, r);
  }
  if constexpr (KEEP)
#pragma unroll
    for (int k = 0; k < K; ++k) pre(k, k);
  int64_t gate_row = -1;
  for (; r < a.rows; r += step) {
    u32x4 x[K], y[K];
#pragma unroll
    for (int k = 0; k < K; ++k) x[k] = nr[k], y[k] = ny[k];
    float g[EACH ? K : 1][VEC];
    if constexpr (EACH)
#pragma unroll
      for (int k = 0; k < K; ++k)
        load_values<DT>(row_of(a.gate, a.wide_gate, r, a.ldg, E), a.wide_gate, col(k), n, 1.f, g[k]);
    if (r + step < a.rows) {
      load(nr, a.r, r + step);
      load(ny, a.y, r + step);
    }
    const int64_t at = EACH ? 0 : (int64_t)((uint32_t)r / (uint32_t)a.span);
    if constexpr (KEEP)
      if (at != gate_row) {
#pragma unroll
        for (int k = 0; k < K; ++k) post(k, k, at);
      }
    gate_row = at;

    float m = 0.f, dbar = 0.f, rstd = 1.f;
    if (a.post) {
      if (!a.rms) {
        float s[1] = {0.f};
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int e = 0; e < VEC; ++e) s[0] += C::elem(y[k], e);
        meet<W, 1>(s, buf, turn, wave, W * grp);
        keep_packed(y);
        m = rounded(s[0] * inv);
      }
      float q[2] = {0.f, 0.f};
#pragma unroll
      for (int k = 0; k < K; ++k)
        for_elems<VEC>(n - col(k), [&](int e) {
          const float d = C::elem(y[k], e) - m;
          q[0] += d;
          q[1] += d * d;
        });
      meet<W, 2>(q, buf, turn, wave, W * grp);
      keep_packed(y);
      dbar = a.rms ? 0.f : q[0] * inv;
      rstd = norm_rstd(q[1] * inv - dbar * dbar, a.eps);
    }
    // the stream, zero past the columns
    float z[K][VEC];
    float s[1] = {0.f};
    char* p = static_cast<char*>(a.out_r) + r * a.ld_r * (int64_t)E;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int to = KEEP ? k : 0;
      if constexpr (!KEEP) post(k, 0, at);
#pragma unroll
      for (int e = 0; e < VEC; ++e) z[k][e] = 0.f;
      for_elems<VEC>(n - col(k), [&](int e) {
        float u = ((C::elem(y[k], e) - m) - dbar) * rstd * u1[to][e] + u0[to][e];
        if constexpr (EACH) u *= g[k][e];
        z[k][e] = rounded(a.alpha * C::elem(x[k], e) + u);
        s[0] += z[k][e];
      });
      if (col(k) < n) C::store(p, col(k), n, z[k]);
    }
    if (!a.out_y) continue;
    m = dbar = 0.f;
    if (!a.rms) {
      meet<W, 1>(s, buf, turn, wave, W * grp);
      m = rounded(s[0] * inv);
    }
    float q[2] = {0.f, 0.f};
#pragma unroll
    for (int k = 0; k < K; ++k)
      for_elems<VEC>(n - col(k), [&](int e) {
        const float d = z[k][e] - m;
        q[0] += d;
        q[1] += d * d;
      });
    meet<W, 2>(q, buf, turn, wave, W * grp);
    dbar = a.rms ? 0.f : q[0] * inv;
    rstd = norm_rstd(q[1] * inv - dbar * dbar, a.eps);
    p = static_cast<char*>(a.out_y) + r * a.ld_y * (int64_t)E;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (col(k) >= n) continue;
      const int to = KEEP ? k : 0;
      if constexpr (!KEEP) pre(k, 0);
      float h[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) h[e] = ((z[k][e] - m) - dbar) * rstd * gamma[to][e] + beta[to][e];
      C::store(p, col(k), n, h);
    }
  }
}

// The backward pass over the rows: workgroup `slice` of a gate row's `slices`
// takes that row's rows in turn, GROUPS at a time.  Three rounds of sums: the
// means of r' and y; the spreads, mean(t), mean(t rhat); mean(s), mean(s yhat).
// RMS: without the means, two rounds of four and one (a third of the arithmetic,
// which with 8-bit rows takes as long as the memory).
// AHEAD: the next row is loaded ahead, KEPT: gamma and post_gamma stay in
// registers, where the sums leave room for them.
template <int DT, int W, int K, int WAVES, bool RMS>
__global__ __launch_bounds__(64 * WAVES) void block_norm_bwd_kernel(BlockNormArgs a) {
  using C = RowChunk<DT>;
  using Q = Act8Chunk<DT>;
  constexpr int VEC = C::VEC, LANES = 64 * W, GROUPS = WAVES / W, E = sizeof(typename C::Elem);
  constexpr int ROOM = WAVES <= 8 ? 216 : 0;         // of 256 registers (168 and 128 of 12 and 16 waves)
  constexpr int HELD = K * (16 + 5 * VEC);           // the rows, e and the sums
  constexpr bool AHEAD = HELD + 16 * K <= ROOM, KEPT = AHEAD && HELD + 16 * K + 2 * VEC * K <= ROOM;
  __shared__ float buf[2][128];
  __shared__ float fold[GROUPS > 1 ? GROUPS : 1][GROUPS > 1 ? LANES * VEC * K : 1];
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wave = w % W, grp = w / W;
  int me = 64 * wave + (threadIdx.x & 63);
  const int n = a.cols;
  const float inv = 1.f / (float)a.cols;
  // the gate row's rows
  const int gate_row = blockIdx.x / (uint32_t)a.slices, slice = blockIdx.x % (uint32_t)a.slices;
  const bool each = a.gate && a.span == 1;
  const int begin = each ? 0 : gate_row * a.span;
  const int end = each || a.rows - begin < a.span ? a.rows : begin + a.span;
  const int step = a.slices * GROUPS;
  int r = begin + slice * GROUPS + grp;
  int turn = 0;

  auto col = [&](int k) { return VEC * (me + k * LANES); };
  const u32x4 none = {0u, 0u, 0u, 0u};
  auto load = [&](u32x4 (&v)[K], const void* base, int64_t ld, int64_t row) {
    const char* p = static_cast<const char*>(base) + row * ld * (int64_t)E;
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = base && col(k) < n ? C::load(p, col(k), n) : none;
  };
  // 8-bit rows wait as their bytes and the scale's
  auto load_saved = [&](u32x4 (&v)[K], const SavedRows& x, int64_t row) {
    if (!x.scale) return load(v, x.x, x.ld, row);
    const int8_t* p = static_cast<const int8_t*>(x.x) + row * x.ld;
    const uint8_t* s = x.scale + row * x.lds;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      v[k] = none;
      if (col(k) >= n) continue;
      const u32x2 q = Q::load(p, col(k), n);
      v[k] = u32x4{q[0], q[1], s[col(k) / kAct8Block], 0u};
    }
  };
  auto open = [&](u32x4 (&v)[K], const SavedRows& x) {
    if (!x.scale) return;
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = Q::restore(u32x2{v[k][0], v[k][1]}, Q::step(v[k][2]));
  };
  auto load_row = [&](u32x4 (&dh)[K], u32x4 (&dr)[K], u32x4 (&x)[K], u32x4 (&y)[K], int64_t row) {
    load(dh, a.dh, a.lddh, row);
    load(dr, a.dr, a.lddr, row);
    load_saved(x, a.r, row);
    load_saved(y, a.y, row);
  };

  // gamma and gate post_gamma, zero past the columns: what they multiply adds
  // nothing to a sum there
  float g1[KEPT ? K : 1][VEC], gp[KEPT ? K : 1][VEC];
  auto cut = [&](int k, float (&v)[VEC]) {
    if (col(k) + VEC > n)
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = col(k) + e < n ? v[e] : 0.f;
  };
  auto get_gamma = [&](int k, float (&v)[VEC]) {
    load_values<DT>(a.gamma, a.wide_params, col(k), n, 1.f, v);
    cut(k, v);
  };
  auto get_post = [&](int k, float (&v)[VEC]) {
    load_values<DT>(a.post ? a.post_gamma : nullptr, a.wide_params, col(k), n, 1.f, v);
    cut(k, v);
    if (!a.gate || each) return;
    float g[VEC];
    load_values<DT>(row_of(a.gate, a.wide_gate, gate_row, a.ldg, E), a.wide_gate, col(k), n, 1.f, g);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] *= g[e];
  };
  u32x4 nh[AHEAD ? K : 1], nd[AHEAD ? K : 1], nx[AHEAD ? K : 1], ny[AHEAD ? K : 1];
  if constexpr (AHEAD) {
#pragma unroll
    for (int k = 0; k < K; ++k) nh[k] = nd[k] = nx[k] = ny[k] = none;
    if (r < end) load_row(nh, nd, nx, ny, r);
  }
  if constexpr (KEPT)
#pragma unroll
    for (int k = 0; k < K; ++k) {
      get_gamma(k, g1[k]);
      get_post(k, gp[k]);
    }

  float e0[K][VEC], e1[K][VEC], b0[K][VEC], b1[K][VEC];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int e = 0; e < VEC; ++e) e0[k][e] = e1[k][e] = b0[k][e] = b1[k][e] = 0.f;

  // every wave takes as many turns as the workgroup's first row needs; one past
  // the last row works on zeros and keeps nothing
  for (int first = begin + slice * GROUPS; first < end; first += step, r += step) {
    const bool live = r < end;
    u32x4 dh[K], dr[K], x[K], y[K];
    if constexpr (AHEAD) {
#pragma unroll
      for (int k = 0; k < K; ++k) dh[k] = nh[k], dr[k] = nd[k], x[k] = nx[k], y[k] = ny[k];
      if (r + step < end) load_row(nh, nd, nx, ny, r + step);
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) dh[k] = dr[k] = x[k] = y[k] = none;
      if (live) load_row(dh, dr, x, y, r);
    }
    open(x, a.r);
    open(y, a.y);
    // addresses and column tests made anew for each pass over a long row: kept
    // they would take a third of the registers
    if constexpr (K * VEC > 8) asm volatile("" : "+v"(me));
    float mx = 0.f, my = 0.f;
    if constexpr (!RMS) {
      float s[2] = {0.f, 0.f};
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          s[0] += C::elem(x[k], e);
          s[1] += C::elem(y[k], e);
        }
      meet<W, 2>(s, buf, turn, wave, W * grp);
      mx = rounded(s[0] * inv);
      my = a.post ? rounded(s[1] * inv) : 0.f;
    }
    keep_packed(x);
    keep_packed(y);
    // d = x - mx, f = y - my: d^2, t d, f^2; with the means d, t, f too
    float q[RMS ? 3 : 6];
#pragma unroll
    for (float& v : q) v = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float gm[VEC];
      if constexpr (!KEPT) get_gamma(k, gm);
      auto add = [&](int e) __attribute__((always_inline)) {
        const float d = RMS ? C::elem(x[k], e) : C::elem(x[k], e) - mx;
        const float f = RMS ? C::elem(y[k], e) : C::elem(y[k], e) - my;
        const float t = C::elem(dh[k], e) * (KEPT ? g1[KEPT ? k : 0][e] : gm[e]);
        q[0] += d * d;
        q[1] += t * d;
        q[2] += f * f;
        if constexpr (!RMS) {
          q[3] += d;
          q[4] += t;
          q[5] += f;
        }
      };
      if constexpr (RMS) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) add(e);
      } else {
        for_elems<VEC>(n - col(k), add);
      }
    }
    meet<W, RMS ? 3 : 6>(q, buf, turn, wave, W * grp);
    keep_packed(x);
    keep_packed(y);
    keep_packed(dh);
    keep_packed(dr);
    // (the mean's correction: see layernorm.hpp)
    float bx = 0.f, by = 0.f, tbar = 0.f;
    if constexpr (!RMS) {
      bx = q[3] * inv;
      tbar = q[4] * inv;
      by = a.post ? q[5] * inv : 0.f;
    }
    const float rx = norm_rstd(q[0] * inv - bx * bx, a.eps);
    const float ry = a.post ? norm_rstd(q[2] * inv - by * by, a.eps) : 1.f;
    // e = dr + rx t - rx mean(t) - rhat rx mean(t rhat)
    const float c1 = rx * tbar, c2 = rx * (rx * (q[1] * inv - bx * tbar));
    if constexpr (K * VEC > 8) asm volatile("" : "+v"(me));
    float ev[K][VEC];
    float s[RMS ? 1 : 2];
#pragma unroll
    for (float& v : s) v = 0.f;
    char* p = static_cast<char*>(a.out_r) + r * a.ld_r * (int64_t)E;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float gm[VEC], pm[VEC];
      if constexpr (!KEPT) {
        get_gamma(k, gm);
        get_post(k, pm);
      }
      float out[VEC];
      if (a.dh) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float h = C::elem(dh[k], e), t = h * (KEPT ? g1[KEPT ? k : 0][e] : gm[e]);
          const float xh = (RMS ? C::elem(x[k], e) : (C::elem(x[k], e) - mx) - bx) * rx;
          float v = C::elem(dr[k], e) + rx * t;
          if constexpr (!RMS) v -= c1;
          ev[k][e] = v - xh * c2;
          if (live) {
            b0[k][e] += h;
            b1[k][e] += h * xh;
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) ev[k][e] = C::elem(dr[k], e);
      }
      if (live && col(k) < n) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) out[e] = a.alpha * ev[k][e];
        C::store(p, col(k), n, out);
      }
      if (each) {
        // the gate's own gradient, and the gate into e
        float gate[VEC];
        load_values<DT>(row_of(a.gate, a.wide_gate, live ? r : 0, a.ldg, E), a.wide_gate, col(k), n, 1.f, gate);
        if (a.dgate && live && col(k) < n) {
          float pg[VEC], pb[VEC];
          load_values<DT>(a.post ? a.post_gamma : nullptr, a.wide_params, col(k), n, 1.f, pg);
          load_values<DT>(a.post ? a.post_beta : nullptr, a.wide_params, col(k), n, 0.f, pb);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float yh = ((C::elem(y[k], e) - my) - by) * ry;
            out[e] = ev[k][e] * (yh * pg[e] + pb[e]);
          }
          if (a.wide_gate && DT != DT_F32) {
            float* to = static_cast<float*>(a.dgate) + r * a.lddg;
#pragma unroll
            for (int e = 0; e < VEC; e += 4) {
              const float four[4] = {out[e], out[e + 1], out[e + 2], out[e + 3]};
              if (col(k) + e < n) RowChunk<DT_F32>::store(to, col(k) + e, n, four);
            }
          } else {
            C::store(static_cast<char*>(a.dgate) + r * a.lddg * (int64_t)E, col(k), n, out);
          }
        }
#pragma unroll
        for (int e = 0; e < VEC; ++e) ev[k][e] *= gate[e];
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float f = RMS ? C::elem(y[k], e) : C::elem(y[k], e) - my;
        const float sv = ev[k][e] * (KEPT ? gp[KEPT ? k : 0][e] : pm[e]);
        s[0] += sv * f;
        if constexpr (!RMS) s[1] += sv;
      }
    }
    if (a.post) meet<W, RMS ? 1 : 2>(s, buf, turn, wave, W * grp);
    keep_packed(y);
    if (!live) continue;
    // dy = ry s - ry mean(s) - yhat ry mean(s yhat)
    float s1 = 0.f, s2 = 0.f;
    if (a.post) {
      const float sbar = RMS ? 0.f : s[RMS ? 0 : 1] * inv;
      s1 = ry * sbar;
      s2 = ry * (ry * (s[0] * inv - by * sbar));
    }
    p = static_cast<char*>(a.out_y) + r * a.ld_y * (int64_t)E;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float pm[VEC], out[VEC];
      if constexpr (!KEPT) get_post(k, pm);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float yh = (RMS ? C::elem(y[k], e) : (C::elem(y[k], e) - my) - by) * ry, v = ev[k][e];
        float o = ry * (v * (KEPT ? gp[KEPT ? k : 0][e] : pm[e]));
        if constexpr (!RMS) o -= s1;
        out[e] = o - yh * s2;
        e0[k][e] += v;
        e1[k][e] += v * yh;
      }
      if (col(k) < n) C::store(p, col(k), n, out);
    }
  }
  if (!a.part) return;
  float* mine = a.part + (int64_t)blockIdx.x * 4 * n;
  auto keep = [&](float (&acc)[K][VEC], int what) {
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
        mine[what * (int64_t)n + c] = t;
      }
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (col(k) + e < n) mine[what * (int64_t)n + col(k) + e] = acc[k][e];
    }
  };
  keep(e0, 0);
  keep(e1, 1);
  keep(b0, 2);
  keep(b1, 3);
}

}  // namespace trt
