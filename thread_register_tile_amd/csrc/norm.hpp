// norm.hpp -- the layer norm's launch entry points (kern_layernorm.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace trt {

struct NormArgs {
  const void* x;
  const void* dy;        // backward only
  const void* gamma;     // [cols] or null (ones)
  const void* beta;      // [cols] or null (zeros); forward only
  void* out;             // y, or dx
  float* part;           // backward: [gridDim.x][2][cols] partial sums of dgamma and dbeta, or null
  int64_t ldx, lddy, ldo;
  int32_t rows, cols;
  float eps;
};

// Longest row: 64 KiB, which one workgroup of 16 waves holds in registers.
constexpr int64_t kNormMaxRowBytes = 65536;

// Workgroups of the backward pass, each of which leaves one slice of
// 2 * cols binary32 partial sums (dt: the type of x).
int norm_slices(int64_t rows, int64_t cols, int dt);

hipError_t launch_layernorm(const NormArgs& a, int dt, int pdt, hipStream_t s);

// a.part: norm_slices(...) * 2 * cols floats, or null when neither parameter
// gradient is wanted.
hipError_t launch_layernorm_bwd(const NormArgs& a, void* dgamma, void* dbeta, int dt, int pdt,
                                hipStream_t s);

}  // namespace trt
