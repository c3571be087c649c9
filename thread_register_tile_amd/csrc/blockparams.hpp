// blockparams.hpp -- the second kernel of the block norm's backward pass: the
// gradients of its parameters and gate rows from the workgroups' sums.
#pragma once

#include "blocknorm_args.hpp"
#include "gemm_kernel.hpp"

namespace trt {

constexpr int kBlockParamsWaves = 16;

// One value of a vector of type dt, `absent` where there is none.
__device__ __forceinline__ float value_at(const void* p, int dt, int64_t i, float absent) {
  if (!p) return absent;
  if (dt == DT_F32) return Out<DT_F32>::ld(p, i);
  return dt == DT_F16 ? Out<DT_F16>::ld(p, i) : Out<DT_BF16>::ld(p, i);
}
__device__ __forceinline__ void put_value(void* p, int dt, int64_t i, float v) {
  if (dt == DT_F32) Out<DT_F32>::st(p, i, v);
  else if (dt == DT_F16) Out<DT_F16>::st(p, i, v);
  else Out<DT_BF16>::st(p, i, v);
}

// The gradients of parameters and gate rows: 64 columns to a workgroup.  Rows 0
// to 3 of the grid add one of the four sums over every slice, each of the 16
// waves every 16th, in order; the others take the gate rows, a wave each, or the
// workgroup where a gate row has 16 slices or more.  Bound by the reads' latency: 34 MB of
// sums (16384 x 8192, 8 gate rows) take 15 us, 6 MB (4001 x 1023) 4.3; 16 loads in flight
// instead of 8 took 6.3 there, four columns to a lane 16.6 for the 34 MB.
__global__ __launch_bounds__(64 * kBlockParamsWaves) void block_params_kernel(BlockParamsArgs a) {
  __shared__ float sum[2][kBlockParamsWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
  const int64_t stride = 4 * (int64_t)a.cols;
  auto meet = [&](int which, float v) {
    sum[which][wave][lane] = v;
    __syncthreads();
    float t = sum[which][0][lane];
#pragma unroll
    for (int w = 1; w < kBlockParamsWaves; ++w) t += sum[which][w][lane];
    return t;
  };
  const int what = blockIdx.y;
  if (what < 4) {
    void* const outs[4] = {a.dpost_beta, a.dpost_gamma, a.dbeta, a.dgamma};
    void* out = outs[what];
    if (!out) return;   // the whole workgroup
    const bool gated = what < 2 && a.gate && !a.each;
    float s = 0.f;
    if (c < a.cols) {
      const float* p = a.part + what * (int64_t)a.cols + c;
      const int all = a.groups * a.slices;
      if (gated && a.groups > 1) {
#pragma unroll 4
        for (int i = wave; i < all; i += kBlockParamsWaves)
          s += p[i * stride] * value_at(a.gate, a.gdt, (int64_t)((uint32_t)i / (uint32_t)a.slices) * a.ldg + c, 1.f);
      } else {
#pragma unroll 8
        for (int i = wave; i < all; i += kBlockParamsWaves) s += p[i * stride];
        if (gated) s *= value_at(a.gate, a.gdt, c, 1.f);
      }
    }
    s = meet(0, s);
    if (wave == 0 && c < a.cols) put_value(out, a.pdt, c, s);
    return;
  }
  const bool shared = a.slices >= kBlockParamsWaves;
  const int64_t by = shared ? 1 : kBlockParamsWaves, turns = gridDim.y - 4;
  for (int64_t g0 = (what - 4) * by; g0 < a.groups; g0 += turns * by) {
    const int64_t g = g0 + (shared ? 0 : wave);
    float s0 = 0.f, s1 = 0.f;
    if (c < a.cols && g < a.groups) {
      const float* p = a.part + g * a.slices * stride + c;
#pragma unroll 4
      for (int i = shared ? wave : 0; i < a.slices; i += shared ? kBlockParamsWaves : 1) {
        s0 += p[i * stride];
        s1 += p[i * stride + a.cols];
      }
    }
    if (shared) {
      s0 = meet(0, s0);
      s1 = meet(1, s1);
    }
    if (c < a.cols && g < a.groups && (!shared || wave == 0)) {
      // (without post_beta the sum of e is no part of it, whatever it came to)
      float v = s1 * value_at(a.post_gamma, a.pdt, c, 1.f);
      if (a.post_beta) v += s0 * value_at(a.post_beta, a.pdt, c, 0.f);
      put_value(a.dgate, a.gdt, g * a.lddg + c, v);
    }
    if (shared) __syncthreads();
  }
}

}  // namespace trt
