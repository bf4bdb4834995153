// mss_checks.hpp -- host-side argument checks shared by the C ABI's sources.
#pragma once

#include <algorithm>
#include <cstdint>

namespace mss {

struct Extent {
  uintptr_t lo = 0, hi = 0;  // byte range [lo, hi)
  bool valid = false;
};

inline Extent extent_of(const void* p, const int64_t* sizes, const int64_t* strides, int rank,
                 int64_t elem) {
  Extent e;
  if (p == nullptr) return e;
  int64_t span = 0;
  for (int i = 0; i < rank; ++i) span += (sizes[i] - 1) * strides[i];
  e.lo = reinterpret_cast<uintptr_t>(p);
  e.hi = e.lo + static_cast<uintptr_t>((span + 1) * elem);
  e.valid = true;
  return e;
}

inline bool overlaps(const Extent& a, const Extent& b) {
  return a.valid && b.valid && a.lo < b.hi && b.lo < a.hi;
}

inline bool aligned(const void* p, int64_t a) {
  return p == nullptr || (reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(a)) == 0;
}

inline bool strides_nonneg(const int64_t* st, int rank) {
  for (int i = 0; i < rank; ++i)
    if (st[i] < 0) return false;
  return true;
}

// Distinct indices map to distinct elements (needed for outputs only).
inline bool non_overlapping(const int64_t* sizes, const int64_t* strides, int rank) {
  int idx[3] = {0, 1, 2};
  std::sort(idx, idx + rank, [&](int a, int b) { return strides[a] < strides[b]; });
  int64_t need = 1;
  for (int k = 0; k < rank; ++k) {
    const int i = idx[k];
    if (sizes[i] == 1) continue;
    if (strides[i] < need) return false;
    need = strides[i] * sizes[i];
  }
  return true;
}

}  // namespace mss
