// Norms over rows of N: a row's vectors and sums, and the instance for a width.
#pragma once

#include "device_common.h"
#include "sequence.h"

namespace prnn {
namespace norm {

// V neighbouring elements of a row of N.  ODD: rows start at any element and the
// last vector of a row may overlap the one before it, since it ends where the row
// does; else every vector is aligned and the last one ends there by itself.
template <class E, int V, bool ODD>
struct Vec {
  typedef typename E::raw raw;
  typedef raw type __attribute__((ext_vector_type(V)));
  typedef raw any __attribute__((ext_vector_type(V), aligned(ODD ? sizeof(raw) : sizeof(type))));
  static __device__ __forceinline__ type load(const raw* p, bool live, raw absent) {
    return live ? *reinterpret_cast<const any*>(p) : type(absent);
  }
  static __device__ __forceinline__ void store(raw* p, bool live, const type& v) {
    if (live) *reinterpret_cast<any*>(p) = v;
  }
};

// Vector c of a row of N: its first column, whether it exists, and how many of
// its columns the vector before it has.
template <int V, bool ODD>
struct Columns {
  int n, again;
  bool in;
  __device__ __forceinline__ Columns(int c, int N) : n(c * V), again(0), in(c * V < N) {
    if (ODD && in && n + V > N) {
      again = n + V - N;
      n = N - V;
    }
  }
  __device__ __forceinline__ bool own(int e) const { return !ODD || e >= again; }
};

// Parameters: fp32 or the rows' own type; absent ones are a constant.
template <class P, int V, bool ODD>
__device__ __forceinline__ void load_param(const void* p, int n, bool in, float absent, float (&f)[V]) {
  const auto v = Vec<P, V, ODD>::load(static_cast<const typename P::raw*>(p) + n, p != nullptr && in, P::put(absent));
#pragma unroll
  for (int e = 0; e < V; ++e) f[e] = P::get(v[e]);
}

// Sums over the TPR threads of a row, the same value in each of them: within
// rows of 16 lanes, across them, and across the waves through `slot`, the
// row's LDS of TPR / 64 values (TPR > 64 only; every thread of the workgroup
// calls).
template <int TPR, int K>
__device__ __forceinline__ void row_sums(float (&x)[K], float* slot) {
#pragma unroll
  for (int i = 0; i < K; ++i) {
    x[i] = dpp_row_sum(x[i]);
    if constexpr (TPR >= 64) {
      float y = x[i];
      swap16_add(x[i], y);
      y = x[i];
      swap32_add(x[i], y);
    }
  }
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    const int w = threadIdx.x % TPR / 64;
    __syncthreads();  // the values of the sum before have been read
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < K; ++i) slot[w * K + i] = x[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < K; ++i) {
      x[i] = 0.f;
#pragma unroll
      for (int j = 0; j < W; ++j) x[i] += slot[j * K + i];
    }
  }
}

// Threads a row (TPR) and vectors a thread (NV) for rows of N: the fewest
// threads whose registers hold the row, so that most of a vector load's lanes
// are used; vectors of 16 bytes, up to `columns` elements a thread.
struct Shape {
  bool odd;
  int tpr, nv;  // tpr 0: the row does not fit
};
inline Shape shape_of(int N, int elems, bool odd, int columns) {
  static const int kShapes[][2] = {{16, 1},  {16, 2},  {64, 1},  {64, 2},  {64, 3},  {128, 2}, {128, 3},
                                   {256, 2}, {256, 3}, {256, 4}, {512, 3}, {512, 4}, {512, 6}};
  const int units = (N + elems - 1) / elems;
  if (N < elems) return {odd, 0, 0};  // (narrower than a vector: as the widest)
  for (const auto& p : kShapes)
    if (p[0] * p[1] >= units && p[1] * elems <= columns) return {odd, p[0], p[1]};
  return {odd, 0, 0};
}

// Workgroups of 1024 threads for `tasks`: a launch counts threads in 32 bits.
inline unsigned workgroups(int64_t tasks) { return (unsigned)(tasks < 1 << 20 ? tasks : 1 << 20); }

inline bool aligned16(const void* p) { return (uintptr_t)p % 16 == 0; }

constexpr int block_of(int tpr) { return tpr > 256 ? tpr : 256; }

// Calls f(E, P) as types.
template <class F>
hipError_t for_types(prnnDataType_t type, prnnDataType_t ptype, F f) {
  switch (type) {
    case PRNN_DATA_FLOAT: return f(F32(), F32());
    case PRNN_DATA_HALF: return ptype == PRNN_DATA_FLOAT ? f(F16(), F32()) : f(F16(), F16());
    default: return ptype == PRNN_DATA_FLOAT ? f(BF16(), F32()) : f(BF16(), BF16());
  }
}

template <int V, bool ODD, int TPR, int NV>
struct Config {
  static constexpr int v = V, tpr = TPR, nv = NV, block = block_of(TPR);
  static constexpr bool odd = ODD;
};

// Calls f(Config) for the shape; false when the row does not fit.  COLUMNS: as
// shape_of's.
template <int V, int COLUMNS, bool ODD, class F>
bool for_shape(const Shape& s, F f) {
#define PRNN_SHAPE(TPR, NV)                   \
  if constexpr (NV * V <= COLUMNS)            \
    if (s.tpr == TPR && s.nv == NV) {         \
      f(Config<V, ODD, TPR, NV>());           \
      return true;                            \
    }
  PRNN_SHAPE(16, 1) PRNN_SHAPE(16, 2) PRNN_SHAPE(64, 1) PRNN_SHAPE(64, 2) PRNN_SHAPE(64, 3) PRNN_SHAPE(128, 2)
  PRNN_SHAPE(128, 3) PRNN_SHAPE(256, 2) PRNN_SHAPE(256, 3) PRNN_SHAPE(256, 4) PRNN_SHAPE(512, 3) PRNN_SHAPE(512, 4)
  PRNN_SHAPE(512, 6)
#undef PRNN_SHAPE
  return false;
}
template <int V, int COLUMNS, class F>
bool for_shape(const Shape& s, F f) {
  return s.odd ? for_shape<V, COLUMNS, true>(s, f) : for_shape<V, COLUMNS, false>(s, f);
}

}  // namespace norm
}  // namespace prnn
