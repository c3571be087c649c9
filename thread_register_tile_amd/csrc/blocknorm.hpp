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
// rounding.  Backward, r' and y may be 8-bit rows (act8.hpp), 33/32 bytes an
// element instead of two: the sums are those of the integers, each chunk's times
// its step.
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

__device__ __forceinline__ const char* row_of(const void* p, bool wide, int64_t row, int64_t ld, int narrow) {
  return static_cast<const char*>(p) + row * ld * (wide ? 4 : narrow);
}

// A row's chunks without a branch: with memory operations under a condition the
// compiler counts the fewest that may be in flight, and a wait for the row at
// work then waits for the next one's loads or the last one's stores too (16384 x
// 8192 bf16 backward from 8-bit rows 398 us, 266 without).  A row of n >= VEC
// elements is read VEC at a time from no further than its last VEC, and `fix`
// shifts out what lies before the chunk (all of it, where the chunk lies past the
// row): zeros take its place.  (The gradient of a gate for every row is stored under
// a condition all the same, and its gate read in the middle of the row.)  Stores go through a descriptor of the row, at an
// offset beyond it where the chunk is not whole; the cut chunk of a row whose
// length VEC does not divide follows in pieces.
// TINY: rows of fewer than VEC elements, read one by one.
template <int DT, bool TINY>
struct RowIO {
  using C = RowChunk<DT>;
  using Q = Act8Chunk<DT>;
  static constexpr int VEC = C::VEC, E = sizeof(typename C::Elem), BITS = 8 * E;

  // where a chunk is read (an offset without a sign: the loads then add it to a
  // scalar base by themselves)
  __device__ static uint32_t at(int i, int n) { return (uint32_t)(i < n - VEC ? i : n - VEC); }
  __device__ static u32x4 load(const char* row, int i, int n) {
    if constexpr (TINY) return i < n ? C::load(row, i, n) : u32x4{0u, 0u, 0u, 0u};
    return __builtin_nontemporal_load(reinterpret_cast<const typename C::Word4*>(row + at(i, n) * E));
  }
  __device__ static u32x4 load_shared(const char* row, int i, int n) {
    if constexpr (TINY) return i < n ? C::load_shared(row, i, n) : u32x4{0u, 0u, 0u, 0u};
    return *reinterpret_cast<const typename C::Word4*>(row + at(i, n) * E);
  }
  __device__ static u32x2 load8(const int8_t* row, int i, int n) {
    if constexpr (TINY) return i < n ? Q::load(row, i, n) : u32x2{0u, 0u};
    const int8_t* p = row + at(i, n);
    if constexpr (VEC == 8) return __builtin_nontemporal_load(reinterpret_cast<const u32x2_at1*>(p));
    else return u32x2{__builtin_nontemporal_load(reinterpret_cast<const u32_at1*>(p)), 0u};
  }

  // The chunk's own elements, of `over` (0 to VEC) that came before it.
  __device__ static int over(int i, int n) {
    const int o = i + VEC - n;
    return o < 0 ? 0 : o < VEC ? o : VEC;
  }
  __device__ static u32x4 fix(u32x4 v, int i, int n) {
    if constexpr (TINY) return v;
    const int bits = over(i, n) * BITS, b = bits & 63;
    const uint64_t lo = v[0] | (uint64_t)v[1] << 32, hi = v[2] | (uint64_t)v[3] << 32;
    const uint64_t l = bits & 64 ? hi : lo, h = bits & 64 ? 0 : hi;
    uint64_t a = l >> b | h << 1 << (63 - b), c = h >> b;
    if (bits == 128) a = c = 0;
    return u32x4{(uint32_t)a, (uint32_t)(a >> 32), (uint32_t)c, (uint32_t)(c >> 32)};
  }
  __device__ static u32x2 fix8(u32x2 v, int i, int n) {
    if constexpr (TINY) return v;
    const int bits = over(i, n) * 8;   // of VEC bytes: 64, or 32 with nothing above them
    const uint64_t q = v[0] | (uint64_t)v[1] << 32, a = bits == 64 ? 0 : q >> bits;
    return u32x2{(uint32_t)a, (uint32_t)(a >> 32)};
  }

  // whole: no chunk of the wave is cut.  live: store at all.
  __device__ static void store(char* row, int i, int n, bool whole, bool live, const float (&y)[VEC]) {
    const auto rs = __builtin_amdgcn_make_buffer_rsrc((void*)row, (short)0, live ? n * E : 0, kBufferFormat);
    u32x4 v;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if constexpr (DT == DT_F32) v[w] = __float_as_uint(y[w]);
      else v[w] = pack2_f32<DT>(y[2 * w], y[2 * w + 1]);
    }
    const uint32_t off = (uint32_t)i * E;
    __builtin_amdgcn_raw_buffer_store_b128(v, rs, (int)(off | (i + VEC <= n ? 0u : 0x80000000u)), 0, kNonTemporal);
    const int left = n % VEC;   // of the cut chunk, in pieces of 4, 2 and 1: three more operations at most
    if (whole || left == 0) return;
    const uint32_t to = off | (i < n && i + VEC > n ? 0u : 0x80000000u);
    if constexpr (DT == DT_F32) {
      if (left & 2) __builtin_amdgcn_raw_buffer_store_b64(u32x2{v[0], v[1]}, rs, (int)to, 0, 0);
      if (left & 1) __builtin_amdgcn_raw_buffer_store_b32(left & 2 ? v[2] : v[0], rs, (int)(to + (left & 2) * E), 0, 0);
    } else {
      if (left & 4) __builtin_amdgcn_raw_buffer_store_b64(u32x2{v[0], v[1]}, rs, (int)to, 0, 0);
      const uint32_t second = left & 4 ? v[2] : v[0], third = left & 4 ? v[3] : v[1];
      if (left & 2) __builtin_amdgcn_raw_buffer_store_b32(second, rs, (int)(to + (left & 4) * E), 0, 0);
      if (left & 1)
        __builtin_amdgcn_raw_buffer_store_b16((short)(left & 2 ? third : second), rs, (int)(to + (left & 6) * E), 0, 0);
    }
  }
};

// VEC values of a vector or of a gate's row, of the rows' type or binary32;
// `absent` where there is none, else zero past n.  (Read by many workgroups.)
template <int DT, bool TINY>
__device__ __forceinline__ void load_values(const void* p, bool wide, int i, int n, bool whole, float absent,
                                            float (&v)[RowChunk<DT>::VEC]) {
  using F = RowIO<DT_F32, TINY>;
  using IO = RowIO<DT, TINY>;
  constexpr int VEC = RowChunk<DT>::VEC;
  if (!p) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = absent;
  } else if (DT == DT_F32 || wide) {
#pragma unroll
    for (int c = 0; c < VEC; c += 4) {
      u32x4 x = F::load_shared(static_cast<const char*>(p), i + c, n);
      if (!whole) x = F::fix(x, i + c, n);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[c + e] = __uint_as_float(x[e]);
    }
  } else {
    u32x4 x = IO::load_shared(static_cast<const char*>(p), i, n);
    if (!whole) x = IO::fix(x, i, n);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = RowChunk<DT>::elem(x, e);
  }
}

// 1 / sqrt(v + eps) as norm_rstd gives it (NaN stays NaN, a v that rounding left
// below zero counts as zero) but by the reciprocal square root instruction, which
// is off by at most one unit in the last place where its argument is not below
// the normal numbers: those are scaled by 2^100.  (The two square roots and
// divisions of a row took a twentieth of the backward pass's instructions.)
__device__ __forceinline__ float block_rstd(float v, float eps) {
  const float x = (v < 0.f ? 0.f : v) + eps;
  const bool small = x < 0x1p-100f;
  const float y = __builtin_amdgcn_rsqf(small ? x * 0x1p100f : x);
  return small ? y * 0x1p50f : y;
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

// The gate row of a workgroup and its slice of that row's rows.  Neighbours in the grid
// are on different dies: up to 32 gate rows are dealt to them in turn, so that of 8 each
// die walks one (8 gate rows of 2048 rows of 8192 bf16 forward 185 to 188 us against 215
// with neighbours on one gate row, backward 335 and 370; of 4096 97 and 105, 157 and 170;
// but 64 of 256 rows 100 and 94 forward).
struct BlockPlace {
  int gate_row, slice;
};
__device__ __forceinline__ BlockPlace place_of(int slices) {
  const uint32_t b = blockIdx.x, groups = gridDim.x / (uint32_t)slices;
  if (groups <= 32) return {(int)(b % groups), (int)(b / groups)};
  return {(int)(b / (uint32_t)slices), (int)(b % (uint32_t)slices)};
}

// EACH: gate rows of few rows, loaded with each of them; otherwise a workgroup's
// rows lie in one gate row, and gate and post norm's parameters are one product.
// KEEP: the vectors stay in registers; of 16 waves to a row none are left, and LDS
// holds the factors, the summands (where there are any) are read with each row.
// Measured: 16384 x 8192 bf16 178 to 190 us (5.7 to 6.0 TB/s), 8192 x 16384 185 to 204 (8 to 23
// spilled registers), 4000 x 5000 f16 33 (160 MB), one row of 4096 3.8 to 4.
template <int DT, int W, int K, bool EACH, bool TINY>
__global__ __launch_bounds__(NormShape<W>::THREADS) void block_norm_kernel(BlockNormArgs a) {
  using C = RowChunk<DT>;
  using IO = RowIO<DT, TINY>;
  constexpr int VEC = C::VEC, LANES = 64 * W, GROUPS = NormShape<W>::GROUPS, E = sizeof(typename C::Elem);
  constexpr bool KEEP = W < 16;
  __shared__ float buf[2][128];
  // the wave's index in a scalar register: row addresses are then scalar too
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wave = w % W, grp = w / W;
  const int me = 64 * wave + (threadIdx.x & 63);
  const int n = a.cols;
  const float inv = 1.f / (float)a.cols;
  // the workgroup's rows: every `slices`-th GROUPS of one gate row's
  const auto [gate_row, slice] = place_of(a.slices);
  const int begin = EACH ? 0 : gate_row * a.span;
  const int end = EACH || a.rows - begin < a.span ? a.rows : begin + a.span;
  const int step = a.slices * GROUPS;
  int r = begin + slice * GROUPS + grp;
  int turn = 0;

  auto col = [&](int k) { return VEC * (me + k * LANES); };
  auto whole = [&](int k) { return VEC * (64 * (wave + 1) + k * LANES) <= n; };   // a scalar

  // u1 yhat + u0 is what the gate multiplies (EACH) or what joins the stream
  float u1[KEEP ? K : 1][VEC], u0[KEEP ? K : 1][VEC], gamma[KEEP ? K : 1][VEC], beta[KEEP ? K : 1][VEC];
  __shared__ f32x4 kept[2][KEEP ? 1 : K * VEC / 4][KEEP ? 1 : LANES];   // a lane's own entries
  auto gated = [&](int k, float (&v)[VEC]) __attribute__((always_inline)) {
    if (EACH || !a.gate) return;
    float g[VEC];
    load_values<DT, TINY>(row_of(a.gate, a.wide_gate, gate_row, a.ldg, E), a.wide_gate, col(k), n, whole(k), 1.f, g);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] *= g[e];
  };
  auto factors = [&](int k, float (&u)[VEC], float (&g)[VEC]) __attribute__((always_inline)) {
    load_values<DT, TINY>(a.post ? a.post_gamma : nullptr, a.wide_params, col(k), n, whole(k), 1.f, u);
    load_values<DT, TINY>(a.gamma, a.wide_params, col(k), n, whole(k), 1.f, g);
    gated(k, u);
  };
  const void* const post_beta = a.post ? a.post_beta : nullptr;
  auto post_summand = [&](int k, float (&v)[VEC]) __attribute__((always_inline)) {
    load_values<DT, TINY>(post_beta, a.wide_params, col(k), n, whole(k), 0.f, v);
    if (post_beta) gated(k, v);
  };
  auto summand = [&](int k, float (&v)[VEC]) __attribute__((always_inline)) {
    load_values<DT, TINY>(a.beta, a.wide_params, col(k), n, whole(k), 0.f, v);
  };
  auto factor_of = [&](int what, int k, float (&v)[VEC]) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < VEC / 4; ++q) {
      const f32x4 x = kept[what][k * (VEC / 4) + q][KEEP ? 0 : threadIdx.x];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * q + e] = x[e];
    }
  };

  // two rows' registers, used in turn: the one at work and the one on its way
  struct Row {
    u32x4 x[K], y[K];
  };
  Row rows[2];
  auto load_row = [&](Row& q, int row) __attribute__((always_inline)) {
    row = row < end ? row : end - 1;
    const char *x = row_of(a.r.x, false, row, a.r.ld, E), *y = row_of(a.y.x, false, row, a.y.ld, E);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      q.x[k] = IO::load(x, col(k), n);
      q.y[k] = IO::load(y, col(k), n);
    }
  };
  load_row(rows[0], r);
  if constexpr (KEEP)
#pragma unroll
    for (int k = 0; k < K; ++k) {
      factors(k, u1[k], gamma[k]);
      post_summand(k, u0[k]);
      summand(k, beta[k]);
    }
  else
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float v[2][VEC];
      factors(k, v[0], v[1]);
#pragma unroll
      for (int q = 0; q < VEC / 4; ++q)
#pragma unroll
        for (int what = 0; what < 2; ++what)
          kept[what][k * (VEC / 4) + q][threadIdx.x] = f32x4{v[what][4 * q], v[what][4 * q + 1], v[what][4 * q + 2], v[what][4 * q + 3]};
    }
  auto body = [&](Row& row, Row& next) __attribute__((always_inline)) {
    auto &x = row.x, &y = row.y;
    float g[EACH ? K : 1][VEC];
    const int at = (uint32_t)r / (uint32_t)a.span;
    if constexpr (EACH)
#pragma unroll
      for (int k = 0; k < K; ++k)
        load_values<DT, TINY>(row_of(a.gate, a.wide_gate, at, a.ldg, E), a.wide_gate, col(k), n, whole(k), 1.f, g[k]);
    load_row(next, r + step);
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (!whole(k)) x[k] = IO::fix(x[k], col(k), n), y[k] = IO::fix(y[k], col(k), n);
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
      rstd = block_rstd(q[1] * inv - dbar * dbar, a.eps);
    }
    // the stream, zero past the columns
    float z[K][VEC];
    float s[1] = {0.f};
    char* p = static_cast<char*>(a.out_r) + r * a.ld_r * (int64_t)E;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int to = KEEP ? k : 0;
      if constexpr (!KEEP) {
        factor_of(0, k, u1[0]);
        post_summand(k, u0[0]);
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) z[k][e] = 0.f;
      for_elems<VEC>(n - col(k), [&](int e) {
        float u = ((C::elem(y[k], e) - m) - dbar) * rstd * u1[to][e] + u0[to][e];
        if constexpr (EACH) u *= g[k][e];
        z[k][e] = rounded(a.alpha * C::elem(x[k], e) + u);
        s[0] += z[k][e];
      });
      IO::store(p, col(k), n, whole(k), true, z[k]);
    }
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
    rstd = block_rstd(q[1] * inv - dbar * dbar, a.eps);
    // (no h asked for: a descriptor of no bytes)
    p = static_cast<char*>(a.out_y) + r * a.ld_y * (int64_t)E;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int to = KEEP ? k : 0;
      if constexpr (!KEEP) {
        factor_of(1, k, gamma[0]);
        summand(k, beta[0]);
      }
      float h[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) h[e] = ((z[k][e] - m) - dbar) * rstd * gamma[to][e] + beta[to][e];
      IO::store(p, col(k), n, whole(k), a.out_y, h);
    }
  };
  for (; r < end; r += step) {
    body(rows[0], rows[1]);
    r += step;
    if (r >= end) break;
    body(rows[1], rows[0]);
  }
}

// keep_packed for saved rows of either form.
template <class V, int K>
__device__ __forceinline__ void keep_saved(V (&v)[K]) {
#pragma unroll
  for (int k = 0; k < K; ++k) asm volatile("" : "+v"(v[k]));
}

// The backward pass over the rows: workgroup `slice` of a gate row's `slices`
// takes that row's rows in turn, GROUPS at a time.  Three rounds of sums: the
// means of r' and y; the spreads, mean(t), mean(t rhat); mean(s), mean(s yhat).
// RMS: without the means, two rounds, of three sums and one (16384 x 8192 bf16 from
// 8-bit rows 250 to 265 us a call against 310: the arithmetic, 40 instructions an element
// and a fifth more with the means, takes over half the memory's time).
// AHEAD: the next row is loaded ahead, KEPT: gamma and post_gamma stay in
// registers, where the sums leave room for them.
// Measured (this kernel alone): 16384 x 8192 bf16 from 8-bit rows 250 us in a long run of
// calls (5.5 TB/s of 1386 MB), up to 304 in its tenth to twentieth call, before the part's clock
// has settled (5.0 TB/s over the first 20; the vector units issue 54 % of the time);
// 4001 x 1023 binary32 23.9 (four turns of rows that are not aligned), 128 x 1024 f16 7.
template <int DT, bool BYTES, int W, int K, int WAVES, bool RMS, bool TINY>
__global__ __launch_bounds__(64 * WAVES) void block_norm_bwd_kernel(BlockNormArgs a) {
  using C = RowChunk<DT>;
  using Q = Act8Chunk<DT>;
  using IO = RowIO<DT, TINY>;
  constexpr int VEC = C::VEC, LANES = 64 * W, GROUPS = WAVES / W, E = sizeof(typename C::Elem);
  // of 256, 168 and 128 registers; HELD: the rows, e and the sums.  (Workgroups of 12
  // and 16 waves spill 1 to 30 registers all the same: an estimate that counted the
  // addresses and constants would drop the next row or the vectors instead.)
  constexpr int ROOM = WAVES <= 8 ? 216 : WAVES <= 12 ? 118 : 78;
  // of long rows LDS holds what the registers do not: gamma and post_gamma, or of
  // 16 waves of 16-bit rows dgamma's and dbeta's sums
  constexpr bool LONG = WAVES > 8 && K > 1, PART = LONG && WAVES > 12 && VEC == 8, VECTORS = LONG && !PART;
  constexpr int HELD = K * (16 + (PART ? 3 : 5) * VEC);
  constexpr bool AHEAD = !(LONG && VEC == 8) && HELD + 16 * K <= ROOM, KEPT = AHEAD && !VECTORS && HELD + 16 * K + 2 * VEC * K <= ROOM;
  __shared__ float buf[2][128];
  __shared__ float fold[GROUPS > 1 ? GROUPS : 1][4][GROUPS > 1 ? LANES * VEC * K : 1];
  __shared__ f32x4 kept[2][LONG ? K * VEC / 4 : 1][LONG ? 64 * WAVES : 1];   // a lane's own entries
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wave = w % W, grp = w / W;
  int me = 64 * wave + (threadIdx.x & 63);
  const int n = a.cols;
  const float inv = 1.f / (float)a.cols;
  // the gate row's rows
  const auto [gate_row, slice] = place_of(a.slices);
  const bool each = a.gate && a.span == 1;
  const int begin = each ? 0 : gate_row * a.span;
  const int end = each || a.rows - begin < a.span ? a.rows : begin + a.span;
  const int step = a.slices * GROUPS;
  int r = begin + slice * GROUPS + grp;
  int turn = 0;

  auto col = [&](int k) { return VEC * (me + k * LANES); };
  auto whole = [&](int k) { return VEC * (64 * (wave + 1) + k * LANES) <= n; };   // a scalar
  using Saved = std::conditional_t<BYTES, u32x2, u32x4>;
  struct Row {
    u32x4 dh[K], dr[K];
    Saved x[K], y[K];
    uint32_t xb[K], yb[K];   // BYTES: the scales' bytes
  };
  // The operations are as many whatever there is to load: without dh or dr the
  // other stands for it, and for r'.
  const u32x4 none = {0u, 0u, 0u, 0u};
  const char *dhp = static_cast<const char*>(a.dh ? a.dh : a.dr), *drp = static_cast<const char*>(a.dr ? a.dr : a.dh);
  const int64_t lddh = a.dh ? a.lddh : a.lddr, lddr = a.dr ? a.lddr : a.lddh;
  const SavedRows xs = a.dh ? a.r : a.y, ys = a.y;
  auto load_saved = [&](Saved (&v)[K], uint32_t (&b)[K], const SavedRows& x, int row) __attribute__((always_inline)) {
    const char* p = static_cast<const char*>(x.x) + row * x.ld * (int64_t)(BYTES ? 1 : E);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if constexpr (BYTES) {
        const int at = col(k) < n ? col(k) : n - 1;
        v[k] = IO::load8(reinterpret_cast<const int8_t*>(p), col(k), n);
        b[k] = (x.scale + row * x.lds)[at / kAct8Block];
      } else {
        v[k] = IO::load(p, col(k), n);
      }
    }
  };
  auto load_up = [&](Row& q, int row) __attribute__((always_inline)) {
    row = row < end ? row : end - 1;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      q.dh[k] = IO::load(dhp + row * lddh * (int64_t)E, col(k), n);
      q.dr[k] = IO::load(drp + row * lddr * (int64_t)E, col(k), n);
    }
  };
  auto load_x = [&](Row& q, int row) __attribute__((always_inline)) { load_saved(q.x, q.xb, xs, row < end ? row : end - 1); };
  auto load_y = [&](Row& q, int row) __attribute__((always_inline)) { load_saved(q.y, q.yb, ys, row < end ? row : end - 1); };
  auto load_row = [&](Row& q, int row) __attribute__((always_inline)) {
    load_up(q, row);
    load_x(q, row);
    load_y(q, row);
  };
  // An element of a saved row is raw() times the chunk's step: the integer of an
  // 8-bit row, of which a sum takes the step out, or the element itself and 1.
  auto open_saved = [&](Saved (&v)[K], float (&step)[K], const uint32_t (&b)[K]) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if constexpr (BYTES) {
        step[k] = Q::step(b[k]);
        if (!whole(k)) v[k] = IO::fix8(v[k], col(k), n);
      } else {
        step[k] = 1.f;
        if (!whole(k)) v[k] = IO::fix(v[k], col(k), n);
      }
    }
  };
  auto raw = [](const Saved& v, int e) __attribute__((always_inline)) {
    if constexpr (BYTES) return (float)(int8_t)(v[e / 4] >> (8 * (e & 3)));
    else return C::elem(v, e);
  };

  // of 8-bit rows a chunk's sum of u v, an exact integer
  auto dot = [](const Saved& u, const Saved& v) __attribute__((always_inline)) {
    int c = 0;
#pragma unroll
    for (int w = 0; w < VEC / 4; ++w) c = __builtin_amdgcn_sdot4((int)u[w], (int)v[w], c, false);
    return (float)c;
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
    load_values<DT, TINY>(a.gamma, a.wide_params, col(k), n, whole(k), 1.f, v);
    cut(k, v);
  };
  auto get_post = [&](int k, float (&v)[VEC]) {
    load_values<DT, TINY>(a.post ? a.post_gamma : nullptr, a.wide_params, col(k), n, whole(k), 1.f, v);
    cut(k, v);
    if (!a.gate || each) return;
    float g[VEC];
    load_values<DT, TINY>(row_of(a.gate, a.wide_gate, gate_row, a.ldg, E), a.wide_gate, col(k), n, whole(k), 1.f, g);
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] *= g[e];
  };
  // a vector's part of a chunk, where it is not in registers
  auto vector = [&](int what, int k, float (&v)[VEC]) __attribute__((always_inline)) {
    if constexpr (VECTORS) {
#pragma unroll
      for (int q = 0; q < VEC / 4; ++q) {
        const f32x4 x = kept[what][k * (VEC / 4) + q][threadIdx.x];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * q + e] = x[e];
      }
    } else if (what == 0) {
      get_gamma(k, v);
    } else {
      get_post(k, v);
    }
  };
  if constexpr (VECTORS)
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float v[2][VEC];
      get_gamma(k, v[0]);
      get_post(k, v[1]);
#pragma unroll
      for (int q = 0; q < VEC / 4; ++q)
#pragma unroll
        for (int what = 0; what < 2; ++what)
          kept[what][k * (VEC / 4) + q][threadIdx.x] = f32x4{v[what][4 * q], v[what][4 * q + 1], v[what][4 * q + 2], v[what][4 * q + 3]};
    }
  // two rows' registers, used in turn: the one at work and the one on its way; or
  // one, each part of which is loaded again as soon as it has been used
  Row rows[AHEAD ? 2 : 1];
  load_row(rows[0], r);
  if constexpr (KEPT)
#pragma unroll
    for (int k = 0; k < K; ++k) {
      get_gamma(k, g1[k]);
      get_post(k, gp[k]);
    }

  float e0[K][VEC], e1[K][VEC], b0[PART ? 1 : K][VEC], b1[PART ? 1 : K][VEC];
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int e = 0; e < VEC; ++e) e0[k][e] = e1[k][e] = b0[PART ? 0 : k][e] = b1[PART ? 0 : k][e] = 0.f;
  if constexpr (PART)
#pragma unroll
    for (int v = 0; v < K * VEC / 4; ++v) kept[0][v][threadIdx.x] = kept[1][v][threadIdx.x] = f32x4{0.f, 0.f, 0.f, 0.f};

  // One row; a wave whose row lies past the end (in its last turn) works on zeros,
  // with rstd = 0, and stores nothing.  Gamma and the gate are zero for it too, or one
  // that is not finite would make NaN of them.
  static_assert(GROUPS == 1 || KEPT, "a wave without a row clears its gamma");
  auto body = [&](Row& row, Row& next) __attribute__((always_inline)) {
    const bool live = GROUPS == 1 || r < end;
    if constexpr (AHEAD) load_row(next, r + step);
    u32x4 (&dh)[K] = row.dh, (&dr)[K] = row.dr;
    Saved x[K], y[K];
    float xstep[K], ystep[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (!whole(k)) dh[k] = IO::fix(dh[k], col(k), n), dr[k] = IO::fix(dr[k], col(k), n);
      x[k] = row.x[k], y[k] = row.y[k];
    }
    open_saved(x, xstep, row.xb);
    open_saved(y, ystep, row.yb);
    if constexpr (!AHEAD && BYTES) {
      load_x(row, r + step);
      load_y(row, r + step);
    }
    if (!a.dr)
#pragma unroll
      for (int k = 0; k < K; ++k) dr[k] = none;
    if (!live)
#pragma unroll
      for (int k = 0; k < K; ++k) {
        dh[k] = dr[k] = none;
        x[k] = y[k] = Saved{};
        xstep[k] = ystep[k] = 0.f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          g1[KEPT ? k : 0][e] = 0.f;
          asm volatile("" : "+v"(g1[KEPT ? k : 0][e]));   // keeps the branch
        }
      }
    // addresses and column tests made anew for each pass over a long row: kept
    // they would take a third of the registers
    if constexpr (K * VEC > 8) asm volatile("" : "+v"(me));
    float mx = 0.f, my = 0.f;
    float xsum[K], ysum[K];   // BYTES: each chunk's
    if constexpr (!RMS) {
      float s[2] = {0.f, 0.f};
#pragma unroll
      for (int k = 0; k < K; ++k) {
        float c[2] = {0.f, 0.f};
        if constexpr (BYTES) {
          const Saved ones = {0x01010101u, 0x01010101u};
          c[0] = dot(x[k], ones);
          c[1] = dot(y[k], ones);
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            c[0] += raw(x[k], e);
            c[1] += raw(y[k], e);
          }
        }
        xsum[k] = xstep[k] * c[0];
        ysum[k] = ystep[k] * c[1];
        s[0] += xsum[k];
        s[1] += ysum[k];
      }
      meet<W, 2>(s, buf, turn, wave, W * grp);
      mx = rounded(s[0] * inv);
      my = a.post ? rounded(s[1] * inv) : 0.f;
    }
    keep_saved(x);
    keep_saved(y);
    // d = x - mx, f = y - my: d^2, t d, f^2; with the means d, t, f too
    float q[RMS ? 3 : 6];
#pragma unroll
    for (float& v : q) v = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float gm[VEC];
      if constexpr (!KEPT) vector(0, k, gm);
      if constexpr (RMS) {
        float c[3] = {0.f, 0.f, 0.f};
        if constexpr (BYTES) c[0] = dot(x[k], x[k]), c[2] = dot(y[k], y[k]);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float d = raw(x[k], e), f = raw(y[k], e);
          const float t = C::elem(dh[k], e) * (KEPT ? g1[KEPT ? k : 0][e] : gm[e]);
          if constexpr (!BYTES) c[0] += d * d;
          c[1] += t * d;
          if constexpr (!BYTES) c[2] += f * f;
        }
        q[0] += xstep[k] * (xstep[k] * c[0]);
        q[1] += xstep[k] * c[1];
        q[2] += ystep[k] * (ystep[k] * c[2]);
      } else {
        for_elems<VEC>(n - col(k), [&](int e) __attribute__((always_inline)) {
          const float d = raw(x[k], e) * xstep[k] - mx, f = raw(y[k], e) * ystep[k] - my;
          const float t = C::elem(dh[k], e) * (KEPT ? g1[KEPT ? k : 0][e] : gm[e]);
          q[0] += d * d;
          q[1] += t * d;
          q[2] += f * f;
          if constexpr (!BYTES) q[3] += d;
          q[4] += t;
          if constexpr (!BYTES) q[5] += f;
        });
        if constexpr (BYTES) {
          const int left = n - col(k);
          const float of = (float)(left < 0 ? 0 : left < VEC ? left : VEC);
          q[3] += xsum[k] - of * mx;
          q[5] += ysum[k] - of * my;
        }
      }
    }
    meet<W, RMS ? 3 : 6>(q, buf, turn, wave, W * grp);
    keep_saved(x);
    keep_saved(y);
    keep_packed(dh);
    keep_packed(dr);
    // (the mean's correction: see layernorm.hpp)
    float bx = 0.f, by = 0.f, tbar = 0.f;
    if constexpr (!RMS) {
      bx = q[3] * inv;
      tbar = q[4] * inv;
      by = a.post ? q[5] * inv : 0.f;
    }
    const float rx = live ? block_rstd(q[0] * inv - bx * bx, a.eps) : 0.f;
    const float ry = !live ? 0.f : a.post ? block_rstd(q[2] * inv - by * by, a.eps) : 1.f;
    // e = dr + rx (t - mean(t)) - rhat rx mean(t rhat), rhat = d rx - bx rx
    const float c2 = rx * (rx * (q[1] * inv - bx * tbar)), xo = -bx * rx, yo = -by * ry;
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
        vector(0, k, gm);
        vector(1, k, pm);
      }
      float out[VEC];
      f32x4 part[2];
      const float xr = xstep[k] * rx;
      if (a.dh) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float h = C::elem(dh[k], e);
          float t = h * (KEPT ? g1[KEPT ? k : 0][e] : gm[e]);
          if constexpr (!RMS) t -= tbar;
          const float xh = RMS ? raw(x[k], e) * xr : (raw(x[k], e) * xstep[k] - mx) * rx + xo;
          ev[k][e] = (C::elem(dr[k], e) + rx * t) - xh * c2;
          if constexpr (!PART) {
            b0[k][e] += h;
            b1[k][e] += h * xh;
          } else {
            // (one after the other: four sums at a time go through registers)
            if (e % 4 == 0) part[0] = kept[0][(VEC * k + e) / 4][threadIdx.x], part[1] = kept[1][(VEC * k + e) / 4][threadIdx.x];
            part[0][e % 4] += h;
            part[1][e % 4] += h * xh;
            if (e % 4 == 3) kept[0][(VEC * k + e) / 4][threadIdx.x] = part[0], kept[1][(VEC * k + e) / 4][threadIdx.x] = part[1];
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) ev[k][e] = C::elem(dr[k], e);
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) out[e] = a.alpha * ev[k][e];
      IO::store(p, col(k), n, whole(k), live, out);
      if (each) {
        // the gate's own gradient, and the gate into e
        float gate[VEC];
        load_values<DT, TINY>(row_of(a.gate, a.wide_gate, live ? r : 0, a.ldg, E), a.wide_gate, col(k), n, whole(k), 1.f, gate);
        if (!live)
#pragma unroll
          for (int e = 0; e < VEC; ++e) gate[e] = 0.f;
        if (a.dgate && live && col(k) < n) {
          float pg[VEC], pb[VEC];
          load_values<DT, TINY>(a.post ? a.post_gamma : nullptr, a.wide_params, col(k), n, whole(k), 1.f, pg);
          load_values<DT, TINY>(a.post ? a.post_beta : nullptr, a.wide_params, col(k), n, whole(k), 0.f, pb);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float yh = (raw(y[k], e) * ystep[k] - my) * ry + yo;
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
      float c = 0.f;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float f = RMS ? raw(y[k], e) : raw(y[k], e) * ystep[k] - my;
        const float sv = ev[k][e] * (KEPT ? gp[KEPT ? k : 0][e] : pm[e]);
        c += sv * f;
        if constexpr (!RMS) s[1] += sv;
      }
      s[0] += RMS ? ystep[k] * c : c;
    }
    if constexpr (!AHEAD) {
      load_up(row, r + step);
      if constexpr (!BYTES) load_x(row, r + step);
    }
    if (a.post) meet<W, RMS ? 1 : 2>(s, buf, turn, wave, W * grp);
    keep_saved(y);
    // dy = ry (s - mean(s)) - yhat ry mean(s yhat)
    float sbar = 0.f, s2 = 0.f;
    if (a.post) {
      if constexpr (!RMS) sbar = s[1] * inv;
      s2 = ry * (ry * (s[0] * inv - by * sbar));
    }
    p = static_cast<char*>(a.out_y) + r * a.ld_y * (int64_t)E;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float pm[VEC], out[VEC];
      if constexpr (!KEPT) vector(1, k, pm);
      const float yr = ystep[k] * ry;
      float yh[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        yh[e] = RMS ? raw(y[k], e) * yr : (raw(y[k], e) * ystep[k] - my) * ry + yo;
        out[e] = ev[k][e] * (KEPT ? gp[KEPT ? k : 0][e] : pm[e]);
        e0[k][e] += ev[k][e];
        e1[k][e] += ev[k][e] * yh[e];
      }
      // (without the norm y is no part of it, whatever it holds)
      if (a.post)
#pragma unroll
        for (int e = 0; e < VEC; ++e) out[e] = ry * (RMS ? out[e] : out[e] - sbar) - yh[e] * s2;
      IO::store(p, col(k), n, whole(k), live, out);
    }
    if constexpr (!AHEAD && !BYTES) load_y(row, r + step);
  };
  // every wave takes as many turns as the workgroup's first row needs
  int first = begin + slice * GROUPS;
  if constexpr (AHEAD) {
    for (; first < end; first += step, r += step) {
      body(rows[0], rows[1]);
      first += step, r += step;
      if (first >= end) break;
      body(rows[1], rows[0]);
    }
  } else {
    for (; first < end; first += step, r += step) body(rows[0], rows[0]);
  }
  if (!a.part) return;
  float* mine = a.part + ((int64_t)gate_row * a.slices + slice) * 4 * n;
  // of several groups: their sums of a column, added in group order
  auto keep = [&](float (&acc)[K][VEC], int what) {
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        if constexpr (GROUPS > 1) fold[grp][what][VEC * (me + k * LANES) + e] = acc[k][e];
        else if (col(k) + e < n) mine[what * (int64_t)n + col(k) + e] = acc[k][e];
      }
  };
  keep(e0, 0);
  keep(e1, 1);
  if constexpr (PART) {
#pragma unroll
    for (int what = 0; what < 2; ++what)
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (col(k) + e < n) mine[(2 + what) * (int64_t)n + col(k) + e] = kept[what][(VEC * k + e) / 4][threadIdx.x][e % 4];
  } else {
    keep(b0, 2);
    keep(b1, 3);
  }
  if constexpr (GROUPS > 1) {
    __syncthreads();
    for (int c = threadIdx.x; c < n; c += 64 * WAVES)
#pragma unroll
      for (int what = 0; what < 4; ++what) {
        float t = fold[0][what][c];
#pragma unroll
        for (int q = 1; q < GROUPS; ++q) t += fold[q][what][c];
        mine[what * (int64_t)n + c] = t;
      }
  }
}

}  // namespace trt
