// xent.hpp -- the vocabulary head's softmax cross entropy without its logits:
// what the GEMM kernels do around their products for it, and the small
// kernels beside them, for gfx950.
//
//   z = X W^T (tokens x vocabulary),  lse_t = log sum_v exp z_tv,
//   loss_t = lse_t - z_t,target
//   g_tv = exp(z_tv - lse_t) (dloss_t + dlse_t) - [v = target_t] dloss_t
//   dX = G W,  dW = G^T X
//
// Forward: the GEMM kernel's tile of z never leaves the registers.  Its
// epilogue takes each row's maximum over the tile's columns and the sum of
// exp(z - maximum) over all of them but the target, one pair per row and tile (8
// bytes for 256 logits), and the target's logit where the tile holds it;
// xent_combine_kernel joins a row's pairs.  With R the sum over the others,
// loss = log(1 + R / exp(z_target)): a well predicted token's small loss keeps
// its relative accuracy, which lse - z_target would lose to cancellation.
// Backward, in pieces of the vocabulary: the same product again, whose epilogue
// turns z into g in the registers and rounds it once to the inputs' type; then
// the two products of that piece of G.  Bound by the matrix cores from a few
// hundred tokens on, by reading W below.
//
// Tokens whose target is the ignored one take no part: xent_prep_kernel lists
// the others, the products' row counts are read from device memory, and A's
// rows are reached through that list, so a batch that is half prompt costs
// half, and whatever X holds at an ignored token (NaN included) reaches
// nothing.
//
// Roundings to 16 bits beside the results' own: G, to the inputs' type.  With c
// = max_t max(|dloss_t|, |dloss_t + dlse_t|) taken out and put back in
// binary32, |g| <= 2, and under a mean or a sum the entry that dominates a row,
// p_target - 1, loses nothing where p_target is small.  A gradient sums terms of
// either sign, so the terms' rounding errors stay one rounding's size against it
// however many they are: bf16 gradients are off by 2.2e-3 to 2.4e-3 of their
// norm for 77 tokens (16384 x 1024) and 1.9e-3 for 8192 (131072 x 4096), where a
// binary32 G would leave 1.7e-3, their own rounding; with binary16 the results'
// loss below 2^-14 weighs more (1.2e-3 either way for 4097 tokens, 32003 x 2560).  Without
// that rounding dX's and dW's products would be twice as long.  For few tokens,
// where they wait for memory, they may be: G is held as two rows of 16-bit
// numbers, the rounded value and what the rounding left, which is off by half a
// step of half a step (kXentHalvesTokens).  binary16 would lose small
// probabilities (its smallest value is 2^-24): G is held times 2^14 there,
// which keeps all bits of a g down to 2^-28 of c.
#pragma once

#include "gemm_dma.hpp"
#include "xent_args.hpp"

namespace trt {

// A's rows through the list of live tokens (ALWAYS: there is one; else all rows
// in place without one).  rows > 0.
template <bool ALWAYS>
struct LiveRows {
  const int32_t* list;
  int32_t rows;
  __device__ int operator()(int r) const {
    int at = r;
    if (ALWAYS || list) at = list[r < rows ? r : rows - 1];
    return r < rows ? at : -1;
  }
};

// A value that is the same for the whole workgroup, in a scalar register: the
// copies' descriptors are scalar arithmetic on it.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

// Copies 1 KiB of an array of `rows` entries of `each` bytes, from entry m0 on,
// to LDS address lds (one wave); 16-byte words past the last entry's read as
// zero.  (A descriptor drops a copy that its end cuts, so the end is rounded
// up: the arrays are padded in the workspace.)
__device__ __forceinline__ void copy_rows(const void* base, int rows, int each, uint32_t lds,
                                          int m0, int lane) {
  const auto rs = __builtin_amdgcn_make_buffer_rsrc((void*)base, (short)0, (rows * each + 15) & ~15,
                                                    kBufferFormat);
  // (five wait states after whatever wrote the descriptor: see dma_one)
  asm volatile("s_nop 4\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :: "{m0}"(uniform((int)lds)), "v"((uint32_t)(m0 * each + 16 * lane)), "s"(rs));
}

// Maximum and sum over the four lanes l, l + 16, l + 32, l + 48 that share a
// row of a fragment, in each of them.  Exchanging the odd rows of 16 lanes (then
// the upper 32 lanes) of a value with the even ones (lower 32) of its copy
// leaves both halves' values side by side in every lane.
template <class F>
__device__ __forceinline__ float over_row(float v, F&& f) {
  const uint32_t u = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  v = f(__uint_as_float(a[0]), __uint_as_float(a[1]));
  const uint32_t w = __float_as_uint(v);
  const auto b = __builtin_amdgcn_permlane32_swap(w, w, false, false);
  return f(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float row_max(float v) {
  return over_row(v, [](float a, float b) { return __builtin_fmaxf(a, b); });
}
__device__ __forceinline__ float row_sum(float v) {
  return over_row(v, [](float a, float b) { return a + b; });
}

// Sets the problem's row count to the number of live tokens; false for the
// workgroups past the last tile that leaves.
template <int BM, class P>
__device__ __forceinline__ bool live_rows(P& p) {
  if (p.live) p.M = uniform(*p.live);
  p.tiles_m = (p.M + BM - 1) / BM;
  return (int)blockIdx.x < p.tiles_m * p.tiles_n;
}

// ---- the forward product's epilogue -----------------------------------------

template <class TL_, bool PIPELINED>
struct XentStats {
  using Args = XentStatsArgs;
  __device__ static int tile(const Args&) { return blockIdx.x; }
  __device__ static bool begin(Args& p) { return live_rows<TL_::BM>(p); }
  static constexpr bool LISTED = TL_::BM == 256;   // tiles of 128 serve few tokens too, in place
  __device__ static LiveRows<LISTED> rows(const Args& p) { return {p.list, p.M}; }
  // finish() needs 8 bytes of LDS for each row and wave beside it
  static constexpr bool STREAMS = true;
  template <class TL>
  static constexpr int SCRATCH = TL::WN * TL::BM * 8;
  // the tile's targets, 4 bytes a row
  template <class TL>
  static constexpr int KEPT = 1024;
  template <class TL>
  __device__ static void fetch(const Args& p, uint32_t lds, int m0, int wave, int lane) {
    // (by every wave, the same bytes to the same place: a branch on the wave
    // costs more)
    if (LISTED || p.want) copy_rows(p.want, p.M, 4, lds, m0, lane);
  }

  // A lane holds, for each of its FM rows, FN runs of four columns; the four
  // lanes l, l+16, l+32, l+48 share a row.  Row sums therefore take two
  // exchanges, then LDS joins the waves side by side in the tile.
  template <class TL, int DT>
  __device__ __forceinline__ static void finish(const Args& p, f32x4 (&acc)[TL::FM][TL::FN],
                                                char* lds, char* kept, int m0, int n0, int t) {
    const int lane = t & 63, wave = t >> 6;
    f32x2* pairs = reinterpret_cast<f32x2*>(lds);   // [WN][BM]
    const int wn = wave % TL::WN;
    const int c0 = TL::owner_col(0, lane, wave);
    auto rows = [&]<bool EDGE>() __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < TL::FM; ++i) {
        int left = p.N - n0 - c0;   // columns from the lane's first one on
        // (made anew for each row: the 32 comparisons with it, kept from row to
        // row, would take 64 scalar registers)
        if (EDGE) asm volatile("" : "+v"(left));
        float v[4 * TL::FN];
#pragma unroll
        for (int j = 0; j < TL::FN; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[4 * j + e] = EDGE && 16 * j + e >= left ? -__builtin_inff() : acc[i][j][e];
        float top = v[0];
#pragma unroll
        for (int c = 1; c + 1 < 4 * TL::FN; c += 2) top = __builtin_fmaxf(__builtin_fmaxf(top, v[c]), v[c + 1]);
        top = row_max(__builtin_fmaxf(top, v[4 * TL::FN - 1]));
        // a row of -inf only: exp(-inf - 0) = 0
        const float base = top == -__builtin_inff() ? 0.f : -top * kLog2E;
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 4 * TL::FN; ++c)
          sum[c & 3] += __builtin_amdgcn_exp2f(__builtin_fmaf(v[c], kLog2E, base));
        const float all = row_sum((sum[0] + sum[1]) + (sum[2] + sum[3]));
        if (lane < 16) pairs[wn * TL::BM + TL::owner_row(4 * i * TL::FN, lane, wave)] = f32x2{top, all};
      }
    };
    if (n0 + TL::BN > p.N) rows.template operator()<true>();
    else rows.template operator()<false>();
    // The rows whose target lies in the wave's columns (few waves have any):
    // the target's logit apart, and the sum again without its term.  (In the
    // loop above, as a choice between every column and -inf, the wide tile
    // would spill a third of a row: 8192 x 131072 x 4096 6.35 ms, this way 5.95.)
#pragma unroll
    for (int i = 0; i < TL::FM; ++i) {
      const int row = TL::owner_row(4 * i * TL::FN, lane, wave), m = m0 + row;
      int64_t at = -1;
      if (PIPELINED && (LISTED || p.want)) at = reinterpret_cast<const int32_t*>(kept)[row];
      else if (m < p.M) at = p.want ? p.want[m] : p.target[m];
      at -= p.col0 + n0 + c0;   // from the lane's first column on
      const int want = m < p.M && at >= 0 && at < 16 * TL::FN && (at & 15) < 4 ? (int)at : -1;
      if (__any(want >= 0)) {
        int left = p.N - n0 - c0;
        asm volatile("" : "+v"(left));
        f32x2& pair = pairs[wn * TL::BM + row];
        const float top = pair[0], base = top == -__builtin_inff() ? 0.f : -top * kLog2E;
        float z = 0.f, sum = 0.f;
#pragma unroll
        for (int j = 0; j < TL::FN; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float v = acc[i][j][e], term = __builtin_amdgcn_exp2f(__builtin_fmaf(v, kLog2E, base));
            const bool it = want == 16 * j + e;
            z = it ? v : z;
            sum += it || 16 * j + e >= left ? 0.f : term;
          }
        if (want >= 0) p.at[m] = z;
        sum = row_sum(sum);
        if (lane < 16) pair[1] = sum;
      }
    }
    __syncthreads();
    if (t < TL::BM && m0 + t < p.M) {
      float top = -__builtin_inff();
#pragma unroll
      for (int w = 0; w < TL::WN; ++w) top = __builtin_fmaxf(top, pairs[w * TL::BM + t][0]);
      const float base = top == -__builtin_inff() ? 0.f : top;
      float sum = 0.f;
#pragma unroll
      for (int w = 0; w < TL::WN; ++w) {
        const f32x2 q = pairs[w * TL::BM + t];
        sum += q[1] * __builtin_amdgcn_exp2f((q[0] - base) * kLog2E);
      }
      p.part[(int64_t)(p.tile0 + n0 / TL::BN) * p.ldp + m0 + t] = f32x2{top, sum};
    }
  }
};

// ---- the backward products' epilogues -----------------------------------------

// Stores a tile of the pipelined kernel, `fast` as in epilogue_lds.
template <class TL, int OT, bool ADD>
__device__ __forceinline__ void store_tile(const GemmArgs& p, const f32x4 (&acc)[TL::FM][TL::FN],
                                           char* lds, int m0, int n0, int t, bool fast) {
  float none[EpiShape<TL>::PANELS][4];
#pragma unroll
  for (int q = 0; q < EpiShape<TL>::PANELS; ++q)
#pragma unroll
    for (int e = 0; e < 4; ++e) none[q][e] = -0.f;
  float* stage = reinterpret_cast<float*>(lds);
  if (fast) epilogue_passes<TL, OT, ADD ? EPI_FAST_RES : EPI_FAST>(p, acc, stage, m0, n0, t, none);
  else epilogue_passes<TL, OT, EPI_MASKED>(p, acc, stage, m0, n0, t, none);
}

// Stores a tile of 16-bit elements straight from the accumulators.  A lane
// holds four columns of a row in each fragment; exchanging them between the
// lanes 16 apart over two neighbouring fragments gives each lane eight
// consecutive columns of one fragment, 16 bytes.  The four stores that fill a
// 128-byte line follow each other, and the L2 joins them.  C through a descriptor
// that ends at row M; N and ldc are multiples of 8 and C is 16-byte aligned.
template <class TL, int DT>
__device__ __forceinline__ void store_rows(const GemmArgs& p, const f32x4 (&acc)[TL::FM][TL::FN],
                                           int m0, int n0, int lane, int wave) {
  const int rows = p.M - m0 < TL::BM ? p.M - m0 : TL::BM;
  const auto rs = __builtin_amdgcn_make_buffer_rsrc(
      (void*)(static_cast<uint16_t*>(p.C) + (int64_t)m0 * p.ldc), (short)0,
      (int)((uint32_t)rows * (uint32_t)p.ldc * 2u), kBufferFormat);
  const int odd = (lane >> 4) & 1;
  // after the exchange: columns of fragment 2 jj + odd, from its run 2 (lane / 32) on
  const int c0 = n0 + TL::owner_col(0, 0, wave) + 16 * odd + 8 * (lane >> 5);
  static_assert(TL::FN % 2 == 0, "fragments in pairs");
#pragma unroll
  for (int i = 0; i < TL::FM; ++i) {
    const uint32_t row = (uint32_t)TL::owner_row(4 * i * TL::FN, lane, wave) * (uint32_t)p.ldc;
#pragma unroll
    for (int j = 0; j < TL::FN; j += 2) {
      u32x4 v;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t lo = pack2_f32<DT>(acc[i][j][2 * h], acc[i][j][2 * h + 1]);
        const uint32_t hi = pack2_f32<DT>(acc[i][j + 1][2 * h], acc[i][j + 1][2 * h + 1]);
        const auto x = __builtin_amdgcn_permlane16_swap(lo, hi, false, false);
        v[h] = x[0];
        v[2 + h] = x[1];
      }
      const int c = c0 + 16 * j;
      const uint32_t off = (row + (uint32_t)c) * 2u | (c < p.N ? 0u : 0x80000000u);
      __builtin_amdgcn_raw_buffer_store_b128(v, rs, (int)off, 0, 0);
    }
  }
}

template <class TL_, bool PIPELINED>
struct XentGrad {
  using Args = XentGradArgs;
  __device__ static int tile(const Args&) { return blockIdx.x; }
  __device__ static bool begin(Args& p) { return live_rows<TL_::BM>(p); }
  __device__ static LiveRows<true> rows(const Args& p) { return {p.list, p.M}; }
  // finish() needs no LDS
  static constexpr bool STREAMS = true;
  template <class TL>
  static constexpr int SCRATCH = 0;
  // the tile's row entries, 64 to a wave's copy
  template <class TL>
  static constexpr int KEPT = TL::BM * (int)sizeof(XentRow);
  template <class TL>
  __device__ static void fetch(const Args& p, uint32_t lds, int m0, int wave, int lane) {
    static_assert(sizeof(XentRow) == 16 && TL::WAVES % (TL::BM / 64) == 0, "one copy a wave");
    const int w = wave % (TL::BM / 64);
    copy_rows(p.info, p.M, 16, lds + 1024 * w, m0 + 64 * w, lane);
  }

  template <class TL, int DT>
  __device__ __forceinline__ static void finish(const Args& p, f32x4 (&acc)[TL::FM][TL::FN],
                                                char* lds, char* kept, int m0, int n0, int t) {
    const int lane = t & 63, wave = t >> 6;
    const int c0 = n0 + TL::owner_col(0, lane, wave);
#pragma unroll
    for (int i = 0; i < TL::FM; ++i) {
      const int row = TL::owner_row(4 * i * TL::FN, lane, wave), m = m0 + row;
      XentRow q = {0.f, 0.f, 0.f, -1};
      if constexpr (PIPELINED) q = reinterpret_cast<const XentRow*>(kept)[row];
      else if (m < p.M) q = p.info[m];
      const float a = q.a * kGradScale<DT>, b = q.b * kGradScale<DT>;
#pragma unroll
      for (int j = 0; j < TL::FN; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[i][j][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(acc[i][j][e], kLog2E, -q.lse2)) * a;
      const int64_t rel = (int64_t)q.target - p.col0 - c0;
      const int want = rel >= 0 && rel < 16 * TL::FN ? (int)rel : -1;
      if (__any(want >= 0)) {   // few waves hold any of their rows' targets
#pragma unroll
        for (int j = 0; j < TL::FN; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] -= want == 16 * j + e ? b : 0.f;
      }
    }
    if (n0 + TL::BN > p.cols) {
#pragma unroll
      for (int j = 0; j < TL::FN; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (c0 + 16 * j + e >= p.cols)
#pragma unroll
            for (int i = 0; i < TL::FM; ++i) acc[i][j][e] = 0.f;
    }
    Args q = p;
    // (few tokens: not on tiles of 256)
    const bool halves = TL::BM < 256 && p.halves;
    if (halves) q.ldc = 2 * p.ldc;   // rows 2m and 2m + 1 of G
    auto store = [&]() __attribute__((always_inline)) {
      if constexpr (PIPELINED) store_rows<TL, DT>(q, acc, m0, n0, lane, wave);
      else epilogue_store<TL>(q, acc, m0, n0, lane, wave);
    };
    store();
    if (halves) {
#pragma unroll
      for (int i = 0; i < TL::FM; ++i)
#pragma unroll
        for (int j = 0; j < TL::FN; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] -= to_f32<DT>(from_f32<DT>(acc[i][j][e]));
      q.C = static_cast<uint16_t*>(p.C) + p.ldc;
      store();
    }
  }
};

// dX += G W over one piece: binary32 sums in the workspace, one buffer for
// each of the slices that K is cut into where tiles are few (xent_plan.hpp).
template <class TL_, bool PIPELINED>
struct XentInput {
  using Args = XentInputArgs;
  // Workgroups in order of their slice, then of their tile.
  __device__ static bool begin(Args& p) {
    const int slice = uniform(p.head->slice);
    p.M = uniform(p.head->live) << p.halves;
    p.tiles_m = (p.M + TL_::BM - 1) / TL_::BM;
    const int tiles = p.tiles_m * p.tiles_n;
    const int at = tiles > 0 ? blockIdx.x / (uint32_t)tiles : 0;
    if (tiles == 0 || (int64_t)at * slice >= p.K) return false;
    const int k0 = at * slice;
    p.A += k0;
    p.B += k0 * p.ldb;
    p.b_bytes -= k0 * p.ldb * 2;
    p.K = p.K - k0 < slice ? p.K - k0 : slice;
    // (32 bits suffice where the pipelined kernel runs, and only it asks)
    p.a_bytes = uniform(((p.M - 1) * (int)p.lda + p.K) * 2);
    p.C = static_cast<float*>(p.C) + at * (xent_sum_rows(p.M) * p.ldc);
    p.R = p.add ? p.C : nullptr;
    return true;
  }
  __device__ static int tile(const Args& p) { return (int)(blockIdx.x % (uint32_t)(p.tiles_m * p.tiles_n)); }
  __device__ static SameRows rows(const Args&) { return {}; }
  static constexpr bool STREAMS = false;
  template <class TL>
  static constexpr int KEPT = 0;
  template <class TL>
  __device__ static void fetch(const Args&, uint32_t, int, int, int) {}
  template <class TL, int DT>
  __device__ __forceinline__ static void finish(const Args& p, f32x4 (&acc)[TL::FM][TL::FN],
                                                char* lds, char*, int m0, int n0, int t) {
    if constexpr (PIPELINED) {
      // in place: a thread reads just the elements that it stores
      if (p.add) store_tile<TL, DT_F32, true>(p, acc, lds, m0, n0, t, true);
      else store_tile<TL, DT_F32, false>(p, acc, lds, m0, n0, t, true);
    } else {
      epilogue_store<TL>(p, acc, m0, n0, t & 63, t >> 6);
    }
  }
};

// dW = c G^T X' over the live tokens: K is their number.
template <class TL_, bool PIPELINED>
struct XentWeight {
  using Args = XentWeightArgs;
  __device__ static int tile(const Args&) { return blockIdx.x; }
  __device__ static bool begin(Args& p) {
    p.K = uniform(*p.live) << p.halves;
    // in 32 bits: below 2^31 where the pipelined kernel runs, and only it asks
    const int rows = p.K > 0 ? p.K - 1 : 0;
    p.a_bytes = uniform((rows * (int)p.lda + p.g_cols) * 2);
    p.b_bytes = uniform(p.K * (int)p.ldb * 2);
    return true;
  }
  __device__ static SameRows rows(const Args&) { return {}; }
  static constexpr bool STREAMS = false;
  template <class TL>
  static constexpr int KEPT = 0;
  template <class TL>
  __device__ static void fetch(const Args&, uint32_t, int, int, int) {}
  template <class TL, int DT>
  __device__ __forceinline__ static void finish(const Args& p, f32x4 (&acc)[TL::FM][TL::FN],
                                                char* lds, char*, int m0, int n0, int t) {
    const float f = *p.factor;
#pragma unroll
    for (int i = 0; i < TL::FM; ++i)
#pragma unroll
      for (int j = 0; j < TL::FN; ++j) acc[i][j] *= f;
    if constexpr (PIPELINED) {
      const bool fast = p.epi_vec && (n0 + TL::BN <= p.N || p.N % 4 == 0) && p.ldc < kEpiFastMaxLd;
      with_out_type(p.out_dt, [&]<int OT>() { store_tile<TL, OT, false>(p, acc, lds, m0, n0, t, fast); });
    } else {
      epilogue_store<TL>(p, acc, m0, n0, t & 63, t >> 6);
    }
  }
};

}  // namespace trt
