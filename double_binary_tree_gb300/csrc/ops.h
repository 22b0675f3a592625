// Host-side helpers shared by the training operators (internal): device
// properties, launches and buffer checks (ops.cc).
#pragma once

#include <cuda_runtime.h>

#include "../../include/vr.h"

namespace vr {

struct OpDevice {
  int device;
  int sms;
  unsigned* status;              // this device's status word
  unsigned long long timeoutNs;  // limit of every bounded wait
};

// The current device's properties (api.cc).
vr_result_t op_device(OpDevice* out);
// One kernel launch on the caller's stream (api.cc), counted in
// vr_launch_count.  Every kernel launched this way calls pdl_wait before it
// touches memory: it may start while the previous one on the stream drains.
vr_result_t op_launch(const void* fn, dim3 grid, dim3 block, void** args, size_t smem,
                      void* stream, int cluster = 1);

inline size_t op_elem_size(int dtype) {
  return dtype == VR_FLOAT32 ? 4 : dtype == VR_FLOAT16 || dtype == VR_BFLOAT16 ? 2 : 0;
}

// A buffer of `rows` rows of rowBytes bytes, strideBytes apart.
struct OpBuffer {
  const void* p;
  size_t rows, rowBytes, strideBytes;
  bool write;
};
// No written buffer may touch another one, except an identical input listed
// directly before it (in place).  Rows of equal stride may interleave.
bool op_buffers_ok(const OpBuffer* b, int n);

// The same for `count` inputs and outputs of one size and a workspace:
// dst[i] may be src[i].  Any count: sorted by address.
bool op_lists_ok(const void* const* src, void* const* dst, int count, size_t bytes,
                 const void* workspace, size_t workspaceBytes);

// The option VR_VALIDATE_POINTERS (api.cc): whether every buffer can be
// reached from the current device.
vr_result_t op_reachable(const OpBuffer* b, int n, int device);
vr_result_t op_reachable(const void* const* p, int n, int device);

// Bytes rounded up to the alignment of a workspace's parts.
constexpr size_t kOpAlign = 256;
inline size_t op_round(size_t n) { return (n + kOpAlign - 1) & ~(kOpAlign - 1); }
// Callers align a workspace to 16 bytes; kernels that access its parts 32
// bytes at a time take them from the first multiple of kOpAlign in it, for
// which the size that the caller was told has kOpSlack bytes.
constexpr size_t kOpSlack = kOpAlign - 16;
inline char* op_workspace(void* p) {
  return reinterpret_cast<char*>(op_round(reinterpret_cast<size_t>(p)));
}

}  // namespace vr
