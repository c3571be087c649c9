// status.hpp -- the calling thread's last error, shared by the units that
// define entry points.
#pragma once

#include <hip/hip_runtime.h>

#include <string>

#include "../../include/trt.h"

namespace trt {

inline thread_local std::string g_err;

inline trt_status fail(trt_status s, const std::string& msg) {
  g_err = msg;
  return s;
}

// The status of one launch, as the runtime returned it for that launch.
inline trt_status launched(hipError_t e, const char* what) {
  if (e != hipSuccess)
    return fail(TRT_ERR_HIP, std::string(what) + ": " + hipGetErrorString(e));
  g_err.clear();
  return TRT_OK;
}

}  // namespace trt
