// Buffer checks shared by the training operators.
#include "ops.h"

#include <algorithm>
#include <cstdint>
#include <vector>

namespace vr {
namespace {

// Whether any byte belongs to both buffers.
bool touch(const OpBuffer& a, const OpBuffer& b) {
  if (!a.rows || !b.rows || !a.rowBytes || !b.rowBytes) return false;
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  const size_t an = (a.rows - 1) * a.strideBytes + a.rowBytes;
  const size_t bn = (b.rows - 1) * b.strideBytes + b.rowBytes;
  if (x + an <= y || y + bn <= x) return false;
  // Rows of one stride: the columns may be disjoint although the extents
  // are not (slices of one wider matrix).
  if (a.strideBytes == b.strideBytes && a.rows > 1 && b.rows > 1) {
    const size_t s = a.strideBytes;
    const size_t d = x <= y ? (size_t)(y - x) % s : (s - (size_t)(x - y) % s) % s;
    return !(d >= a.rowBytes && s - d >= b.rowBytes);
  }
  return true;
}

}  // namespace

bool op_buffers_ok(const OpBuffer* b, int n) {
  for (int i = 0; i < n; ++i) {
    if (!b[i].write) continue;
    for (int j = 0; j < n; ++j) {
      if (j == i || (b[j].write && j < i) || !touch(b[i], b[j])) continue;
      const bool inPlace = j == i - 1 && !b[j].write && b[j].p == b[i].p &&
                           b[j].rowBytes == b[i].rowBytes && b[j].strideBytes == b[i].strideBytes;
      if (!inPlace) return false;
    }
  }
  return true;
}

bool op_lists_ok(const void* const* src, void* const* dst, int count, size_t bytes,
                 const void* workspace, size_t workspaceBytes) {
  try {
    struct Span {
      uintptr_t lo, hi;
      int i;  // list index; -1: the workspace
      bool write;
    };
    std::vector<Span> v;
    v.reserve(2 * (size_t)count + 1);
    for (int i = 0; i < count; ++i) {
      v.push_back({(uintptr_t)dst[i], (uintptr_t)dst[i] + bytes, i, true});
      if (src[i] != dst[i]) v.push_back({(uintptr_t)src[i], (uintptr_t)src[i] + bytes, i, false});
    }
    v.push_back({(uintptr_t)workspace, (uintptr_t)workspace + workspaceBytes, -1, true});
    std::sort(v.begin(), v.end(), [](const Span& a, const Span& b) { return a.lo < b.lo; });
    // the furthest end so far of any span, and of a written one
    uintptr_t any = 0, written = 0;
    for (const Span& s : v) {
      if (s.lo < written || (s.write && s.lo < any)) return false;
      any = std::max(any, s.hi);
      if (s.write) written = std::max(written, s.hi);
    }
    return true;
  } catch (...) {  // no host memory for the list
    return false;
  }
}

}  // namespace vr
