// act8.hpp -- activations saved in 8 bits and restored, for gfx950.
//
// Of every 32 columns of a row the largest magnitude's exponent field X (7 at
// least) is the scale's byte, and each element is held as an integer
//   q = round to nearest even (x / 2^(X-133)), |q| <= 127,
// that stands for q 2^(X-133): the MX format's 8-bit integers with 8-bit
// exponents.  With 2^(X-127) <= max |x| < 2^(X-126) the largest q is at least 64
// and an element is off by at most half a step, 2^-7 of that power, or a
// whole one where it rounds up to 128.  The step is a power of two, so the
// values are what they are whatever the order of any sum: packing is exact
// arithmetic but for its one rounding, and what is restored (7 bits) fits bf16,
// and binary16 where x was binary16.  A block that holds an infinity or NaN has
// X = 255 and stands for NaN throughout: what was not finite does not come back
// as a number.  Integers rather than 8-bit floats: at the same 8.25 bits an
// element they leave a normal distribution's rows off by 0.8 % of their norm where 3 bits
// of mantissa leave 2.7 %.
//
// What bounds it: memory, x once and 33/32 bytes an element.  A thread takes
// four chunks of 16 bytes of x, 256 chunks apart, all loaded before the first
// is used; a block's four (binary32: eight) chunks sit in neighbouring lanes,
// whose maximum takes two (three) data-parallel moves.  Measured: 16384 x 8192 bf16
// packed in 67 to 69 us (6.0 TB/s), restored in 67 (6.1); 4001 x 1023 binary32, whose
// rows are not aligned, in 6.5 and 8.5, among other work 7 and 11.
#pragma once

#include "act8_args.hpp"
#include "rowchunk.hpp"

namespace trt {

typedef uint32_t u32x2_at1 __attribute__((ext_vector_type(2), aligned(1)));
typedef uint32_t u32_at1 __attribute__((aligned(1)));

// The 8-bit chunk beside a chunk of DT: VEC bytes in one or two words.
template <int DT>
struct Act8Chunk {
  static constexpr int VEC = RowChunk<DT>::VEC;
  static constexpr int PER = kAct8Block / VEC;   // chunks to a scale

  // bytes i .. i+VEC-1 of the row q, of which those at or past n read as zero
  __device__ static u32x2 load(const int8_t* q, int i, int n) {
    if (i + VEC <= n) {
      if constexpr (VEC == 8)
        return __builtin_nontemporal_load(reinterpret_cast<const u32x2_at1*>(q + i));
      else
        return u32x2{__builtin_nontemporal_load(reinterpret_cast<const u32_at1*>(q + i)), 0u};
    }
    u32x2 v = {0u, 0u};
    int left = n - i;   // below VEC; hidden from the compiler as in RowChunk
    asm volatile("" : "+v"(left));
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (e < left) v[e / 4] |= (uint32_t)(uint8_t)q[i + e] << (8 * (e & 3));
    return v;
  }
  __device__ static void store(int8_t* q, int i, int n, u32x2 v) {
    if (i + VEC <= n) {
      if constexpr (VEC == 8) __builtin_nontemporal_store(v, reinterpret_cast<u32x2_at1*>(q + i));
      else __builtin_nontemporal_store(v[0], reinterpret_cast<u32_at1*>(q + i));
      return;
    }
    int left = n - i;
    asm volatile("" : "+v"(left));
#pragma unroll
    for (int e = 0; e < VEC; ++e)
      if (e < left) q[i + e] = (int8_t)(v[e / 4] >> (8 * (e & 3)));
  }

  // The step 2^(X-133) of a scale's byte: NaN for 255, a number below the
  // normal ones for less than 7 (pack makes none).
  __device__ static float step(uint32_t byte) {
    const uint32_t normal = (byte - 6u) << 23, below = 1u << (byte + 16u);
    const uint32_t bits = byte >= 7u ? normal : below;
    return __uint_as_float(byte == 255u ? 0x7FC00000u : bits);
  }
  __device__ static float value(u32x2 v, int e, float s) {
    return (float)(int8_t)(v[e / 4] >> (8 * (e & 3))) * s;
  }
  // The chunk of DT that it stands for.
  __device__ static u32x4 restore(u32x2 v, float s) {
    u32x4 o;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if constexpr (DT == DT_F32) o[w] = __float_as_uint(value(v, w, s));
      else o[w] = pack2_f32<DT>(value(v, 2 * w, s), value(v, 2 * w + 1, s));
    }
    return o;
  }
};

// The largest of v over the PER lanes of a block's chunks, in each of them.
template <int PER>
__device__ __forceinline__ uint32_t block_max(uint32_t v) {
  auto with = [&](auto ctrl) {
    const uint32_t o = __builtin_amdgcn_update_dpp(0, v, ctrl.value, 0xF, 0xF, true);
    v = v > o ? v : o;
  };
  with(std::integral_constant<int, 0xB1>{});                          // quad lanes 1 0 3 2
  with(std::integral_constant<int, 0x4E>{});                          // quad lanes 2 3 0 1
  if constexpr (PER == 8) with(std::integral_constant<int, 0x141>{});  // mirror of 8 lanes
  static_assert(PER == 4 || PER == 8, "lanes of a block");
  return v;
}

// The workgroup's chunks: `per` to a row (whole blocks), thread t's j-th is
// chunk 256 j + t of the group's.  The division of the group's first chunk is
// scalar and 64 bits wide, each thread's own is 32.
struct Act8Place {
  int64_t row0;
  uint32_t first, per;
  __device__ Act8Place(int64_t group, int32_t cols, int per_block) {
    per = ((uint32_t)cols + kAct8Block - 1) / kAct8Block * per_block;
    const int64_t c = group * kAct8Chunks;
    row0 = c / per;
    first = (uint32_t)(c - row0 * per);
  }
  __device__ int64_t at(int j, uint32_t& chunk) const {
    const uint32_t c = first + 256u * j + threadIdx.x, r = c / per;
    chunk = c - r * per;
    return row0 + r;
  }
};

template <int DT>
__global__ __launch_bounds__(256) void act8_pack_kernel(Act8Args a) {
  using C = RowChunk<DT>;
  using Q = Act8Chunk<DT>;
  constexpr int VEC = C::VEC, U = kAct8Chunks / 256;
  const Act8Place place(blockIdx.x, a.cols, Q::PER);
  const int n = a.cols;
  int64_t row[U];
  int col[U];
  u32x4 x[U];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    uint32_t c;
    row[j] = place.at(j, c);
    col[j] = VEC * (int)c;
    const char* p = static_cast<const char*>(a.x) + row[j] * a.ldx * (int64_t)sizeof(typename C::Elem);
    x[j] = row[j] < a.rows && col[j] < n ? C::load(p, col[j], n) : u32x4{0u, 0u, 0u, 0u};
  }
#pragma unroll
  for (int j = 0; j < U; ++j) {
    uint32_t top = 0;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const uint32_t m = __float_as_uint(C::elem(x[j], e)) & 0x7FFFFFFFu;
      top = top > m ? top : m;
    }
    uint32_t byte = block_max<Q::PER>(top) >> 23;
    byte = byte > 7u ? byte : 7u;
    const float inv = __uint_as_float((260u - (byte < 255u ? byte : 254u)) << 23);
    u32x2 v = {0u, 0u};
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      // adding 1.5 2^23 rounds to an integer, to nearest even, in the low byte
      const float f = __builtin_amdgcn_fmed3f(C::elem(x[j], e) * inv, -127.f, 127.f) + 12582912.f;
      v[e / 4] |= (__float_as_uint(f) & 0xFFu) << (8 * (e & 3));
    }
    if (byte == 255u) v = u32x2{0u, 0u};
    if (row[j] >= a.rows || col[j] >= n) continue;
    Q::store(a.q + row[j] * a.ldq, col[j], n, v);
    if (col[j] % kAct8Block == 0) a.scale[row[j] * a.lds + col[j] / kAct8Block] = (uint8_t)byte;
  }
}

// Chunks of group `group` of the rows a, restored; WHOLE: out's rows are whole
// aligned chunks of a workspace, zero past the columns.
template <int DT, bool WHOLE>
__device__ __forceinline__ void act8_restore(const Act8Args& a, int64_t ldo, int64_t group) {
  using C = RowChunk<DT>;
  using Q = Act8Chunk<DT>;
  constexpr int VEC = C::VEC, U = kAct8Chunks / 256;
  const Act8Place place(group, a.cols, Q::PER);
  const int n = a.cols;
  int64_t row[U];
  int col[U];
  u32x2 q[U];
  uint32_t byte[U];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    uint32_t c;
    row[j] = place.at(j, c);
    col[j] = VEC * (int)c;
    const bool in = row[j] < a.rows && col[j] < n;
    q[j] = in ? Q::load(a.q + row[j] * a.ldq, col[j], n) : u32x2{0u, 0u};
    byte[j] = in ? a.scale[row[j] * a.lds + col[j] / kAct8Block] : 7u;
  }
#pragma unroll
  for (int j = 0; j < U; ++j) {
    if (row[j] >= a.rows || col[j] >= n) continue;
    typename C::Elem* p = static_cast<typename C::Elem*>(a.out) + row[j] * ldo;
    const float s = Q::step(byte[j]);
    if (WHOLE || col[j] + VEC <= n) {
      using Word4 = std::conditional_t<WHOLE, u32x4, typename C::Word4>;
      *reinterpret_cast<Word4*>(p + col[j]) = Q::restore(q[j], s);
    } else {
      float y[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) y[e] = Q::value(q[j], e, s);
      C::store(p, col[j], n, y);
    }
  }
}

template <int DT>
__global__ __launch_bounds__(256) void act8_unpack_kernel(Act8Args a) {
  act8_restore<DT, false>(a, a.ldx, blockIdx.x);
}

// The weight gradient's operands in the workspace: x restored, and dy copied
// where its rows are not whole aligned chunks.
template <int DT>
__global__ __launch_bounds__(256) void act8_operands_kernel(Act8OperandArgs a) {
  if ((int)blockIdx.x < a.x_groups) {
    act8_restore<DT, true>(a.x, a.x.ldx, blockIdx.x);
    return;
  }
  using C = RowChunk<DT>;
  constexpr int U = kAct8Chunks / 256;
  const Act8Place place(blockIdx.x - a.x_groups, a.dy_cols, 4);
  int64_t row[U];
  int col[U];
  u32x4 v[U];
#pragma unroll
  for (int j = 0; j < U; ++j) {
    uint32_t c;
    row[j] = place.at(j, c);
    col[j] = 8 * (int)c;
    if (row[j] < a.x.rows && col[j] < a.dy_cols) v[j] = C::load(a.dy + row[j] * a.lddy, col[j], a.dy_cols);
  }
#pragma unroll
  for (int j = 0; j < U; ++j)
    if (row[j] < a.x.rows && col[j] < a.dy_cols)
      *reinterpret_cast<u32x4*>(a.dy_out + row[j] * a.dy_ld + col[j]) = v[j];
}

// dW from the slices' results: each thread four columns, the slices in order.
template <int OT>
__global__ __launch_bounds__(256) void act8_sum_kernel(Act8SumArgs a) {
  const int64_t runs = a.part_ld / 4, all = runs * a.rows;
  for (int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x; id < all; id += (int64_t)gridDim.x * 256) {
    const int64_t m = id / runs, c = 4 * (id - m * runs);
    const float* p = a.part + m * a.part_ld + c;
    f32x4 y = *reinterpret_cast<const f32x4*>(p);
#pragma unroll 8
    for (int s = 1; s < a.slices; ++s) y += *reinterpret_cast<const f32x4*>(p + s * a.step);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (c + e < a.cols) Out<OT>::st(a.dw, m * a.ld + c + e, y[e]);
  }
}

}  // namespace trt
