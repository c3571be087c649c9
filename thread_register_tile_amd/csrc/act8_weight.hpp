// act8_weight.hpp -- the weight gradient from an input saved in 8 bits.
//
//   dW = dY^T X,  X = the values that the 8-bit rows stand for
//
// The library's product with the tokens as its K, both operands stored with
// their columns contiguous.  X is restored to dY's type first, exactly
// (act8.hpp), so the product is that of 16-bit operands and every sum is
// binary32.  Bound by the matrix cores from a few hundred tokens on.  Where
// outputs x inputs give few tiles the tokens are cut into slices with results of
// their own, which a second kernel adds in order.  Restoring inside the product
// would convert each element once for every tile that reads it, with the vector
// units' power that the matrix cores lack; apart it costs 4 % of a large product.
// Measured: 16384 tokens x 8192 x 8192 bf16 1534 us (1.43 PFLOP/s; 66 of it restoring x),
// 4097 x 5001 x 2560 f16 108 (26 laying out x and dY, whose rows of 5001 the copies do not
// take), 77 x 1024 x 1024 9.4 in its two kernels.
#pragma once

#include "act8_args.hpp"
#include "xent.hpp"

namespace trt {

template <class TL_, bool PIPELINED>
struct Act8Weight {
  static_assert(PIPELINED, "the operands are always laid out for the copies");
  using Args = Act8WeightArgs;
  // A slice to each row of the grid.
  __device__ static bool begin(Args& p) {
    const int64_t at = blockIdx.y, k0 = at * p.slice;
    p.A += k0 * p.lda;
    p.B += k0 * p.ldb;
    p.K = p.K - k0 < p.slice ? p.K - (int)k0 : p.slice;
    // the rows' extents, below 2^31 each (the plan's care); a whole last row of
    // dY, whose columns are whole chunks
    p.a_bytes = ((p.K - 1) * (int)p.lda + (p.M + 7) / 8 * 8) * 2;
    p.b_bytes = p.K * (int)p.ldb * 2;
    p.C = static_cast<float*>(p.C) + at * p.part;
    return true;
  }
  __device__ static int tile(const Args&) { return blockIdx.x; }
  __device__ static SameRows rows(const Args&) { return {}; }
  static constexpr bool STREAMS = false;
  template <class TL>
  static constexpr int KEPT = 0;
  template <class TL>
  __device__ static void fetch(const Args&, uint32_t, int, int, int) {}
  template <class TL, int DT>
  __device__ __forceinline__ static void finish(const Args& p, f32x4 (&acc)[TL::FM][TL::FN],
                                                char* lds, char*, int m0, int n0, int t) {
    const bool fast = p.epi_vec && (n0 + TL::BN <= p.N || p.N % 4 == 0) && p.ldc < kEpiFastMaxLd;
    with_out_type(p.out_dt, [&]<int OT>() { store_tile<TL, OT, false>(p, acc, lds, m0, n0, t, fast); });
  }
};

}  // namespace trt
