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
  // By address, only buffers whose extents overlap are compared: few or none.
  struct Span {
    uintptr_t lo, hi;
    int i;
  };
  constexpr int kMost = 4 * VR_MAX_RANKS + 3;
  Span v[kMost];
  if (n > kMost) return false;
  int m = 0;
  for (int i = 0; i < n; ++i)
    if (b[i].rows && b[i].rowBytes) {
      const uintptr_t lo = (uintptr_t)b[i].p;
      v[m++] = {lo, lo + (b[i].rows - 1) * b[i].strideBytes + b[i].rowBytes, i};
    }
  std::sort(v, v + m, [](const Span& x, const Span& y) { return x.lo < y.lo; });
  for (int x = 0; x < m; ++x)
    for (int y = x + 1; y < m && v[y].lo < v[x].hi; ++y) {
      const OpBuffer &p = b[v[x].i], &q = b[v[y].i];
      if ((!p.write && !q.write) || !touch(p, q)) continue;
      const int first = std::min(v[x].i, v[y].i), second = std::max(v[x].i, v[y].i);
      const bool inPlace = second == first + 1 && !b[first].write && b[second].write &&
                           p.p == q.p && p.rowBytes == q.rowBytes &&
                           p.strideBytes == q.strideBytes;
      if (!inPlace) return false;
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
