// buffers.hpp -- host-side checks of the callers' buffers, shared by the row
// operators' entry points.
#pragma once

#include "status.hpp"
#include "validate.hpp"

namespace trt {

// A caller's buffer: a rows x cols matrix with leading dimension ld, named
// for the messages.  A null base is an absent optional buffer.
struct Buf {
  const char* name;
  const void* base;
  int64_t rows, cols, ld, esize;
  Extent extent() const {
    int64_t bytes = 0;
    if (base) span_bytes(rows, cols, ld, bytes, esize);
    const uintptr_t lo = reinterpret_cast<uintptr_t>(base);
    return Extent{lo, lo + (uintptr_t)bytes};
  }
};

// Every buffer's alignment, stride and extent, then each written buffer
// against every other one.  The first n_out buffers are written.
template <size_t N>
trt_status check_buffers(const Buf (&b)[N], size_t n_out) {
  for (size_t i = 0; i < N; ++i) {
    if (!b[i].base) continue;
    if (i < n_out ? b[i].ld < b[i].cols : b[i].ld < 1)
      return fail(TRT_ERR_STRIDE, std::string(b[i].name) +
                                      (i < n_out ? ": rows written must not overlap (ld >= cols)"
                                                 : ": leading dimension must be >= 1"));
    if (reinterpret_cast<uintptr_t>(b[i].base) & (uintptr_t)(b[i].esize - 1))
      return fail(TRT_ERR_ALIGN, std::string(b[i].name) + " must be aligned to its element");
    int64_t bytes;
    if (!span_bytes(b[i].rows, b[i].cols, b[i].ld, bytes, b[i].esize))
      return fail(TRT_ERR_SIZE, std::string(b[i].name) + ": extent overflows");
  }
  for (size_t i = 0; i < n_out; ++i)
    for (size_t j = 0; j < N; ++j)
      if (i != j && overlaps(b[i].extent(), b[j].extent()))
        return fail(TRT_ERR_OVERLAP, std::string(b[i].name) + " overlaps " + b[j].name);
  return TRT_OK;
}

// A workspace of which a call needs `need` > 0 bytes.
inline trt_status check_workspace(const void* ws, int64_t bytes, int64_t need) {
  if (bytes < 0) return fail(TRT_ERR_SIZE, "workspace_bytes must be >= 0");
  if (!ws) return fail(TRT_ERR_NULL, "this call needs a workspace of " + std::to_string(need) + " bytes");
  if (bytes < need)
    return fail(TRT_ERR_SIZE, "the workspace must hold at least " + std::to_string(need) + " bytes");
  if (reinterpret_cast<uintptr_t>(ws) & 15u)
    return fail(TRT_ERR_ALIGN, "the workspace must be 16-byte aligned");
  return TRT_OK;
}

}  // namespace trt
