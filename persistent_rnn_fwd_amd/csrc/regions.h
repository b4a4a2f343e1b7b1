// Host side of the sequence operators: checks that their entry points share.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "prnn.h"

namespace prnn {

inline size_t size_of(prnnDataType_t t) { return t == PRNN_DATA_FLOAT ? 4 : 2; }
inline bool known(prnnDataType_t t) { return t == PRNN_DATA_FLOAT || t == PRNN_DATA_HALF || t == PRNN_DATA_BFLOAT; }
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// The bytes a buffer touches: rows of `row` bytes at multiples of the strides
// below (bytes; counts of 1 have no stride).
struct Region {
  uintptr_t base = 0;
  uint64_t row = 0;  // 0: touches nothing
  struct Axis {
    uint64_t stride, count;
  } axis[3] = {};
};

// `e` and the bytes from an axis' first row to its last.  No memory reaches
// kFar: what does counts as that, so that the sums stay in 64 bits.
constexpr uint64_t kFar = 1ull << 60;
inline uint64_t along(uint64_t e, const Region::Axis& x) {
  if (x.count <= 1) return e;
  const unsigned __int128 far = (unsigned __int128)x.stride * (x.count - 1) + e;
  return far < kFar ? (uint64_t)far : kFar;
}

inline uint64_t extent(const Region& r) {
  uint64_t e = r.row;
  for (const auto& x : r.axis) e = along(e, x);
  return e;
}

inline uint64_t gcd(uint64_t a, uint64_t b) {
  while (b != 0) {
    const uint64_t t = a % b;
    a = b;
    b = t;
  }
  return a;
}

// Whether two regions can share a byte.  Ranges that meet are still disjoint
// when both repeat with one period (slices of one fused buffer) and their
// places inside that period do not meet: the axes whose strides are at least
// the period only move by whole periods.
inline bool overlap(const Region& a, const Region& b) {
  if (a.row == 0 || b.row == 0) return false;
  if (a.base >= b.base + extent(b) || b.base >= a.base + extent(a)) return false;
  // candidate periods: the strides of either region
  for (int from = 0; from < 6; ++from) {
    const auto& pick = from < 3 ? a.axis[from] : b.axis[from - 3];
    if (pick.count <= 1 || pick.stride == 0) continue;
    uint64_t period = pick.stride;
    for (const Region* r : {&a, &b})
      for (const auto& x : r->axis)
        if (x.count > 1 && x.stride >= pick.stride) period = gcd(period, x.stride);
    uint64_t foot[2];
    int i = 0;
    for (const Region* r : {&a, &b}) {
      foot[i] = r->row;
      for (const auto& x : r->axis)
        if (x.stride < pick.stride) foot[i] = along(foot[i], x);
      ++i;
    }
    const uint64_t d = a.base <= b.base ? (b.base - a.base) % period : (period - (a.base - b.base) % period) % period;
    if (d >= foot[0] && d + foot[1] <= period) return false;
  }
  return true;
}

// Whether every element of a region lies apart from the others.
inline bool distinct(const Region& r) {
  Region::Axis x[3] = {r.axis[0], r.axis[1], r.axis[2]};
  std::sort(x, x + 3, [](const Region::Axis& p, const Region::Axis& q) { return p.stride < q.stride; });
  uint64_t e = r.row;
  for (const auto& y : x) {
    if (y.count <= 1) continue;
    if (y.stride < e) return false;
    e = along(e, y);
  }
  return true;
}

inline Region flat(const void* p, uint64_t bytes) {
  Region r;
  r.base = reinterpret_cast<uintptr_t>(p);
  r.row = p != nullptr ? bytes : 0;
  return r;
}

inline Region rows_of(const void* p, int64_t M, int N, int64_t ld, size_t e) {
  Region r = flat(p, p != nullptr && M > 0 ? (uint64_t)N * e : 0);
  r.axis[0] = {(uint64_t)ld * e, (uint64_t)M};
  return r;
}

// Strides beyond this cannot address memory.
constexpr int64_t kMaxStride = 1ll << 40;
inline bool ld_ok(int64_t ld, int N) { return ld >= N && ld <= kMaxStride; }

inline prnnStatus_t launched(hipError_t e) {
  if (e == hipSuccess) return PRNN_STATUS_SUCCESS;
  (void)hipGetLastError();
  return PRNN_STATUS_INTERNAL_ERROR;
}

}  // namespace prnn
