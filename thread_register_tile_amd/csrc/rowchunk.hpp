// rowchunk.hpp -- 16-byte chunks of a matrix row of any alignment.
#pragma once

#include "gemm_kernel.hpp"

namespace trt {

// 16-byte chunks of a row.  A chunk's address is only known to be aligned to
// its element (odd widths and strides): the target's unaligned access mode
// reads it in one instruction all the same.
typedef uint32_t u32x4_at2 __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x4_at4 __attribute__((ext_vector_type(4), aligned(4)));
template <int DT>
struct RowChunk {
  static constexpr int VEC = DT == DT_F32 ? 4 : 8;
  using Word4 = std::conditional_t<DT == DT_F32, u32x4_at4, u32x4_at2>;
  using Elem = std::conditional_t<DT == DT_F32, float, uint16_t>;

  // elements i .. i+VEC-1 of the row p, of which those at or past n read as zero
  __device__ static u32x4 load(const void* p, int i, int n) {
    const Elem* q = static_cast<const Elem*>(p) + i;
    if (i + VEC <= n) return __builtin_nontemporal_load(reinterpret_cast<const Word4*>(q));
    return partial(q, n - i);
  }
  // the same, for data that other workgroups read too
  __device__ static u32x4 load_shared(const void* p, int i, int n) {
    const Elem* q = static_cast<const Elem*>(p) + i;
    if (i + VEC <= n) return *reinterpret_cast<const Word4*>(q);
    return partial(q, n - i);
  }
  __device__ static u32x4 partial(const Elem* q, int left64) {
    u32x4 v = {0u, 0u, 0u, 0u};
    int left = left64;   // below VEC; hidden from the compiler as in for_elems
    asm volatile("" : "+v"(left));
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      uint32_t w = 0u;
      if (e < left) {
        if constexpr (DT == DT_F32) w = __float_as_uint(q[e]);
        else w = q[e];
      }
      if constexpr (DT == DT_F32) v[e] = w;
      else v[e / 2] |= w << (16 * (e & 1));
    }
    return v;
  }
  __device__ static float elem(u32x4 v, int e) {
    if constexpr (DT == DT_F32) {
      const uint32_t w = v[e];
      return __uint_as_float(w);
    } else {
      return to_f32<DT>((e & 1) ? v[e >> 1] >> 16 : v[e >> 1] & 0xFFFFu);
    }
  }
  __device__ static void store(void* p, int i, int n, const float (&y)[VEC]) {
    Elem* q = static_cast<Elem*>(p) + i;
    if (i + VEC <= n) {
      Word4 v;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        if constexpr (DT == DT_F32) v[w] = __float_as_uint(y[w]);
        else v[w] = pack2_f32<DT>(y[2 * w], y[2 * w + 1]);
      }
      __builtin_nontemporal_store(v, reinterpret_cast<Word4*>(q));
      return;
    }
    int left = n - i;
    asm volatile("" : "+v"(left));
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (e < left) {
        if constexpr (DT == DT_F32) q[e] = y[e];
        else q[e] = (uint16_t)from_f32<DT>(y[e]);
      }
  }
};

}  // namespace trt
