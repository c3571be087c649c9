// gemm_wide.hpp -- the cross entropy's product kernel on 256x256 tiles.
//
// The pipelined kernel's product (gemm_dma.hpp: direct-to-LDS copies through
// buffer descriptors, swizzled LDS, 16x16x32 fragments; the products of a tile
// element are added in the same order), cut differently in two places.
//
//   * Four waves of 128x128 instead of eight of 128x64.  A K step of 32 takes
//     the matrix cores 1024 cycles, in which the LDS moves 128 bytes each:
//     eight waves read 12 KiB of fragments apiece and the copies write 32 KiB,
//     1024 cycles of LDS time, all there is; four waves read 16 KiB apiece and
//     leave a quarter of it free.
//   * K steps of 64 instead of 32.  A k-contiguous row then gives a step 128
//     bytes, a whole cache line; with 64 bytes each line crosses from the L2
//     twice, half of it unused each time.
//
// With one wave to a SIMD nothing covers a wait, so a step has one place for
// all of them.  Two LDS stages of 64 KiB, two sets of fragment registers, a
// step in two halves of 32 k:
//   first half: the products of set 0, reading the second half's fragments
//     into set 1 after every third product;
//   wait for those reads and for the copies of step kt + 1; barrier: the
//     stage of step kt is read out, step kt + 1's is whole, for every wave;
//   second half: the products of set 1, reading step kt + 1's first fragments
//     into set 0, with the copies of step kt + 2 into the free stage between
//     the products.
//
// Bound by the matrix cores, and on large products by the power they may draw:
// 8192 x 131072 x 4096 bf16 in 6.0 ms with the statistics' epilogue (1.46
// PFLOP/s at 1.7 GHz), 6.55 on the pipelined kernel.
//
// An epilogue that leaves the stages alone (EPI::STREAMS) runs on a grid of one
// workgroup per compute unit that walks the tiles: the copies of the next
// tile's first two steps go out ahead of the epilogue, which covers their
// latency and the gap between two workgroups.
#pragma once

#include "gemm_dma.hpp"

namespace trt {

// acc += a . b as mfma16 does, with acc held in an accumulation register: the
// 256 of a lane are all there are, the fragments fill the ordinary ones, and
// left to choose the compiler mixes the two and moves half of them every step.
// The compiler does not see a product in it, so whoever reads an accumulator
// by other means waits for it first (accumulators_done); a product on the same
// accumulator follows 64 products later.
template <int DT>
__device__ __forceinline__ void mfma16_acc(f32x4& acc, u32x4 a, u32x4 b) {
  if constexpr (DT == DT_F16) asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
  else asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(b));
}
// A product's result may be read 18 wait states after it at the latest; these are 32.
__device__ __forceinline__ void accumulators_done() {
  asm volatile("s_nop 15\n\ts_nop 15");
  __builtin_amdgcn_sched_barrier(0);
}

// One 16-byte copy per lane to LDS address m0v + OFF + 16 * lane (see
// dma_block: the instruction offset is added on both sides).  The main loop's
// descriptors are scalar arithmetic on loop-carried registers; elsewhere a
// descriptor word may come from a vector instruction (a restored scalar), and
// the copy waits out the five states itself (NOPS = 4).
template <int OFF, int NOPS>
__device__ __forceinline__ void dma_one(__amdgpu_buffer_rsrc_t rs, uint32_t m0v, uint32_t v) {
  asm volatile("s_nop %4\n\tbuffer_load_dwordx4 %1, %2, 0 offen offset:%3 lds"
               :: "{m0}"(m0v), "v"(v), "s"(rs), "n"(OFF), "n"(NOPS));
}

// Swizzle of a k-contiguous stage, rows of 8 chunks: chunk (r, g) in slot
// 8r + (g XOR sw(r)), sw(r) = r1 | (r1 XOR r2) << 1 | (r0 XOR r3) << 2 in the
// bits of r; rows 16 apart swizzle alike.  A fragment read of 16 bytes a lane
// passes 16 lanes at a time: of two neighbouring lane groups, rows 0-3 and 12-15
// of one and 4-11 of the other (then the rest), and these read chunks that
// differ in both low bits (frag_kchunk).  Their 16 words fall on 16 distinct
// places of a 256-byte window.  (With r2 for r1 XOR r2 they met in pairs: four
// cycles more for each read of eight.)
TRT_HD int wide_swz(int r) {
  return ((r >> 1) & 1) | ((((r >> 1) ^ (r >> 2)) & 1) << 1) | (((r ^ (r >> 3)) & 1) << 2);
}
constexpr bool wide_swz_spreads() {
  for (int g = 0; g < 8; ++g)
    for (int first = 0; first < 2; ++first) {
      int places = 0;
      for (int r = 0; r < 16; ++r) {
        const bool inner = r >= 4 && r < 12;
        const int chunk = inner == (first != 0) ? g : g ^ 3;
        places |= 1 << ((r & 1) * 8 + (chunk ^ wide_swz(r)));
        if (wide_swz(r + 16) != wide_swz(r)) return false;
      }
      if (places != 0xFFFF) return false;
    }
  return true;
}
static_assert(wide_swz_spreads(), "fragment reads cover the banks evenly");

// One operand's copies: NCH to a lane and step, copy i of wave w into the 64
// slots from (w NCH + i) 64 on.  A rows-contiguous operand's stage is two
// stages of 32 k in the pipelined kernel's layout, one after the other.
template <class TL, int R, bool KC>
struct WideOperand {
  static constexpr int NCH = R * 8 / TL::THREADS;
  static constexpr int BYTES = R * 128;
  static constexpr uint32_t BIAS = 3 * 1024;
  static_assert(R * 8 % TL::THREADS == 0 && NCH == 8, "two M0 values, four instruction offsets");

  const char* cur;
  uint32_t rem, step_bytes;   // step_bytes: rows-contiguous
  uint32_t voff[NCH];
  uint32_t drop;          // k-contiguous: bit i, copy i lies past K on the last step

  // What every tile shares.
  __device__ __forceinline__ void setup(int64_t ld, int wave, int lane, int K) {
    step_bytes = (uint32_t)(128 * ld);
    drop = 0;
    const int last = (K + 63) / 64 * 64 - 64;
#pragma unroll
    for (int i = 0; KC && i < NCH; ++i) {
      const int s = (wave * NCH + i) * 64 + lane, g = (s & 7) ^ wide_swz(s >> 3);
      drop |= last + 8 * g >= K ? 1u << i : 0u;
    }
  }

  template <class Rows>
  __device__ __forceinline__ void init(const uint16_t* X, int64_t ld, int64_t ext, int row0,
                                       int wave, int lane, Rows rows) {
    cur = reinterpret_cast<const char*>(X) - BIAS;
    rem = (uint32_t)ext + BIAS;
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int s = (wave * NCH + i) * 64 + lane;
      uint32_t off;
      if (KC) {
        const int r = s >> 3, g = (s & 7) ^ wide_swz(r);
        const auto row = rows(row0 + r);
        off = (uint32_t)(((int64_t)row * ld + 8 * g) * 2);
        if constexpr (!std::is_same_v<Rows, SameRows>)
          if (row < 0) off = 0x80000000u;   // beyond every record count
      } else {
        const int h = s / (4 * R), u = s % (4 * R);
        const int k = 32 * h + TL::template mn_slot_k<R>(u), c = TL::template mn_slot_c<R>(u);
        off = (uint32_t)(((int64_t)k * ld + row0 + 8 * c) * 2);
      }
      voff[i] = off + BIAS - 1024u * (i & 3);
    }
  }

  // Copy I of K step `step` of nk to the wave's slots at m0v; CHECKED as in
  // DmaOperand.  The last of a step moves the descriptor on.
  template <bool CHECKED, int I>
  __device__ __forceinline__ void copy(int step, int nk, uint32_t m0v) {
    uint32_t v = voff[I];
    int records = (int)rem;
    if constexpr (CHECKED) {
      records = step < nk ? (int)rem : 0;
      if (KC && step == nk - 1) v |= (drop >> I) << 31;
    }
    const auto rs = __builtin_amdgcn_make_buffer_rsrc((void*)cur, (short)0, records, kBufferFormat);
    dma_one<1024 * (I & 3), CHECKED ? 4 : 0>(rs, m0v + 4096u * (I >> 2), v);
    if constexpr (I == NCH - 1) {
      const uint32_t bytes = KC ? 128 : step_bytes;
      cur += bytes;
      rem -= bytes;
    }
  }
};

// Fragment reads of one operand from either stage: FragReader's, with the
// addresses of both stages (the offset field holds less than a stage).
template <class TL, int R, bool KC, int F, int STAGE>
struct WideReader {
  int addr[2][KC ? 2 : F];

  __device__ __forceinline__ void init(int rbase, int lane, int region) {
    const int g = frag_kchunk(lane >> 4);
    if (KC) {
      const int r = rbase + (lane & 15);
#pragma unroll
      for (int half = 0; half < 2; ++half)
        addr[0][half] = region + 16 * (8 * r + ((4 * half + g) ^ wide_swz(r)));
    } else {
      const int j = lane & 15;
      const int k = 8 * g + (j >> 2);
#pragma unroll
      for (int f = 0; f < F; ++f) {
        const int c = (rbase + 16 * f) / 8 + ((j & 3) >> 1);
        addr[0][f] = region + 16 * (k * (R / 8) + (c ^ TL::template mn_swz<R>(k))) + 8 * (j & 1);
      }
    }
#pragma unroll
    for (int i = 0; i < (KC ? 2 : F); ++i) addr[1][i] = addr[0][i] + STAGE;
  }

  template <int STG, int HALF>
  __device__ __forceinline__ u32x4 read(TRT_LDS char* lds, int f) const {
    if constexpr (KC) {
      return *(TRT_LDS u32x4*)(lds + addr[STG][HALF] + 2048 * f);
    } else {
      TRT_LDS char* p = lds + addr[STG][f] + HALF * (64 * R);
      const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((TRT_LDS i16x4*)p);
      const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((TRT_LDS i16x4*)(p + 8 * R));
      const u32x2 l2 = __builtin_bit_cast(u32x2, lo), h2 = __builtin_bit_cast(u32x2, hi);
      return u32x4{l2[0], l2[1], h2[0], h2[1]};
    }
  }
};

// Workgroups of a grid that walks its tiles: one for each compute unit.
constexpr int kWideUnits = 256;

template <class EPI, class TL>
constexpr int wide_scratch() {
  if constexpr (EPI::STREAMS) return EPI::template SCRATCH<TL>;
  else return 0;
}

template <class TL, int DT, bool A_KC, bool B_KC, class EPI>
__global__ __launch_bounds__(TL::THREADS, 1) void gemm_wide_kernel(typename EPI::Args p) {
  static_assert(TL::MF == 16 && TL::WAVES == 4, "four waves, 16x16x32 fragments");
  constexpr int BM = TL::BM, BN = TL::BN, FM = TL::FM, FN = TL::FN;
  constexpr int PRODUCTS = FM * FN, READS = FM + FN;
  using Args = typename EPI::Args;
  using OpA = WideOperand<TL, BM, A_KC>;
  using OpB = WideOperand<TL, BN, B_KC>;
  constexpr int STAGE = OpA::BYTES + OpB::BYTES;
  constexpr int COPIES = OpA::NCH + OpB::NCH;
  static_assert(3 * READS <= PRODUCTS && 4 * COPIES <= PRODUCTS, "reads and copies fit between the products");
  constexpr int EPI_BYTES = EPI::STREAMS ? 0 : (BM / 2) * BN * 4;
  constexpr int LDS_BYTES = 2 * STAGE > EPI_BYTES ? 2 * STAGE : EPI_BYTES;
  constexpr int KEPT = EPI::template KEPT<TL>;
  static_assert(KEPT % 1024 == 0, "whole copies");
  // behind the stages: what the epilogue keeps (of this tile and the next),
  // and its scratch
  constexpr int KEPT_BYTES = EPI::STREAMS ? 2 * KEPT : KEPT;
  constexpr int SCRATCH = wide_scratch<EPI, TL>();
  __shared__ __attribute__((aligned(1024))) char lds_raw[LDS_BYTES + KEPT_BYTES + SCRATCH];
  TRT_LDS char* lds = (TRT_LDS char*)lds_raw;

  const int t = threadIdx.x;
  const int lane = t & 63, wave = t >> 6;
  if (!EPI::begin(p)) return;

  OpA a;
  OpB b;
  a.setup(p.lda, wave, lane, p.K);
  b.setup(p.ldb, wave, lane, p.K);
  const int nk = (p.K + 63) / 64;
  const uint32_t lds_base = (uint32_t)(uintptr_t)lds;
  const uint32_t m0a = __builtin_amdgcn_readfirstlane(lds_base + wave * OpA::NCH * 1024);
  const uint32_t m0b =
      __builtin_amdgcn_readfirstlane(lds_base + OpA::BYTES + wave * OpB::NCH * 1024);

  WideReader<TL, BM, A_KC, FM, STAGE> ra;
  WideReader<TL, BN, B_KC, FN, STAGE> rb;
  ra.init(TL::owner_row(0, 0, wave), lane, 0);
  rb.init(TL::owner_col(0, 0, wave), lane, OpA::BYTES);

  f32x4 acc[FM][FN];
  u32x4 fa[2][FM], fb[2][FN];
  // fragment f of half HALF of the step in stage STG, into set HALF
  auto read_frag = [&]<int STG, int HALF, int F>() __attribute__((always_inline)) {
    if constexpr (F < FM) fa[HALF][F] = ra.template read<STG, HALF>(lds, F);
    else fb[HALF][F - FM] = rb.template read<STG, HALF>(lds, F - FM);
  };
  auto copy = [&]<bool CHECKED, int C>(int step, int nk, uint32_t st) __attribute__((always_inline)) {
    if constexpr (C < OpA::NCH) a.template copy<CHECKED, C>(step, nk, m0a + st);
    else b.template copy<CHECKED, C - OpA::NCH>(step, nk, m0b + st);
  };
  auto each = [&]<int... I>(auto&& f, std::integer_sequence<int, I...>) __attribute__((always_inline)) {
    (f.template operator()<I>(), ...);
  };

  // The arguments, read again where they are needed (a tile's start and its
  // epilogue): kept, they would hold scalar registers through the main loop,
  // and a scalar spilled to a vector register may not feed a copy (dma_block).
  // Of what begin() changed, a streaming epilogue's is M and the tile rows.
  const int live_m = p.M, tiles_m = p.tiles_m;
  auto arguments = [&]() __attribute__((always_inline)) {
    typedef const __attribute__((address_space(4))) uint64_t* Words;
    static_assert(sizeof(Args) % 8 == 0 && alignof(Args) == 8, "whole words");
    Words from = (Words)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(from));
    uint64_t words[sizeof(Args) / 8];
#pragma unroll
    for (size_t i = 0; i < sizeof(Args) / 8; ++i) words[i] = from[i];
    Args q = __builtin_bit_cast(Args, words);
    q.M = live_m;
    q.tiles_m = tiles_m;
    return q;
  };

  // A tile's first copies: what the epilogue keeps, steps 0 and 1.
  int m0 = 0, n0 = 0;
  auto enter = [&](const Args& p, int tile, int turn) __attribute__((always_inline)) {
    int tm, tn;
    tile_of<8>(tile, p.tiles_m, p.tiles_n, tm, tn);
    m0 = tm * BM;
    n0 = tn * BN;
    // (the lane as a value of this tile's own: nothing made of it is kept from
    // tile to tile, where it would hold registers through the main loop)
    int l = lane, steps = nk;
    asm volatile("" : "+v"(l));
    asm volatile("" : "+s"(steps));
    a.init(p.A, p.lda, p.a_bytes, m0, wave, l, EPI::rows(p));
    b.init(p.B, p.ldb, p.b_bytes, n0, wave, l, SameRows{});
    EPI::template fetch<TL>(p, lds_base + LDS_BYTES + turn * KEPT, m0, wave, l);
    each([&]<int C>() __attribute__((always_inline)) { copy.template operator()<true, C>(0, steps, 0); },
         std::make_integer_sequence<int, COPIES>{});
    each([&]<int C>() __attribute__((always_inline)) { copy.template operator()<true, C>(1, steps, STAGE); },
         std::make_integer_sequence<int, COPIES>{});
  };

  // Step kt, whose stage is U = kt mod 2.
  auto step_body = [&]<bool CHECKED, int U>(int kt) __attribute__((always_inline)) {
    each([&]<int Q>() __attribute__((always_inline)) {
      constexpr int j = Q / FM, i = Q % FM;
      mfma16_acc<DT>(acc[i][j], fb[0][j], fa[0][i]);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (Q % 3 == 0 && Q / 3 < READS) read_frag.template operator()<U, 1, Q / 3>();
      __builtin_amdgcn_sched_barrier(0);
    }, std::make_integer_sequence<int, PRODUCTS>{});
    __builtin_amdgcn_s_waitcnt(waitcnt_lgkm(0));
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    each([&]<int Q>() __attribute__((always_inline)) {
      constexpr int j = Q / FM, i = Q % FM;
      mfma16_acc<DT>(acc[i][j], fb[1][j], fa[1][i]);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (Q % 3 == 0 && Q / 3 < READS) read_frag.template operator()<U ^ 1, 0, Q / 3>();
      if constexpr (Q % 4 == 1 && Q / 4 < COPIES) copy.template operator()<CHECKED, Q / 4>(kt + 2, nk, U * STAGE);
      __builtin_amdgcn_sched_barrier(0);
    }, std::make_integer_sequence<int, PRODUCTS>{});
  };

  int tile = EPI::tile(p), turn = 0;
  if constexpr (EPI::STREAMS) enter(arguments(), tile, turn);
  else enter(p, tile, turn);
  for (;;) {
    // step 0's copies are older than the 16 youngest operations in any case
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(COPIES));
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    each([&]<int F>() __attribute__((always_inline)) { read_frag.template operator()<0, 0, F>(); },
         std::make_integer_sequence<int, READS>{});
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    // Whole rounds of two steps; all but the last two copy live steps before
    // the last one only.
    int kt = 0;
    for (; kt + 4 < nk; kt += 2) {
      step_body.template operator()<false, 0>(kt);
      step_body.template operator()<false, 1>(kt + 1);
    }
    for (; kt + 2 <= nk; kt += 2) {
      step_body.template operator()<true, 0>(kt);
      step_body.template operator()<true, 1>(kt + 1);
    }
    if (kt < nk) step_body.template operator()<true, 0>(kt);
    // drain the copies issued past the end (zero records: they fetch nothing)
    // and the reads of the stage after the last
    __builtin_amdgcn_s_waitcnt(waitcnt_vm(0));
    __builtin_amdgcn_s_waitcnt(waitcnt_lgkm(0));
    accumulators_done();
    __syncthreads();

    char* kept = lds_raw + LDS_BYTES + turn * KEPT;
    if constexpr (EPI::STREAMS) {
      const int em = m0, en = n0;
      tile += kWideUnits;
      turn ^= 1;
      const Args q = arguments();
      const bool more = tile < q.tiles_m * q.tiles_n;
      if (more) enter(arguments(), tile, turn);
      int et = t;
      asm volatile("" : "+v"(et));
      EPI::template finish<TL, DT>(q, acc, lds_raw + LDS_BYTES + KEPT_BYTES, kept, em, en, et);
      if (!more) return;
    } else {
      EPI::template finish<TL, DT>(p, acc, lds_raw, kept, m0, n0, t);
      return;
    }
  }
}

}  // namespace trt
