// Layer norm over rows of N, forward and backward.
//
//   y = (x - mean) rstd w + b
//   dx = rstd (g - mean(g) - n mean(g n)),  dw = sum_m dy n,  db = sum_m dy,
//   with n = (x - mean) rstd and g = dy w
//
// Both passes are bound by memory: x in and y out, or x and dy in and dx out.
// A row is read once into the registers of TPR threads, 16 bytes at a time (V
// elements a vector, NV vectors a thread), so mean and variance are sums over
// centred values without a second read.  The threads of a row set keep their
// columns from row to row: the parameters stay in registers, the next row's
// loads are in flight during this row's sums, and the parameters' gradients are
// sums in registers; each workgroup leaves one partial sum of them and a second
// kernel adds those in a fixed order.  Sums and statistics are fp32; y, dx and
// the parameters' gradients are rounded once.
//
// Rows whose width, stride or address no 16-byte vector divides use the same
// vectors unaligned, the last one moved back to end with the row: 50000 x 500
// bf16 backward takes 33 us against 100 with that vector read by elements, whose
// waits end the loads ahead.
//
// y and dx are stored plainly, for the next layer to find in the caches: a chain
// of norms of 4096 x 5760 bf16 takes 15.5 us each, with nontemporal stores 18.8.
//
// Measured: forward 16384 x 5760 bf16 71-75 us (5.2 TB/s; with the parameters
// read again for every row 90), backward 115 us (4.9 TB/s, a few percent of it
// the partial sums), 4099 x 1153 fp32 backward 18 us.
#include "device_common.h"
#include "sequence.h"

namespace prnn {
namespace {

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

// Forward.  The grid's row sets take rows r, r + R grid, ...; thread i of a set
// keeps the parameters of vectors i + j TPR.  The next row's loads are issued
// before this row's sums.
template <class E, class P, int V, bool ODD, int TPR, int NV, int BLOCK>
__global__ void __launch_bounds__(BLOCK) norm_kernel(NormArgs a) {
  typedef typename E::raw raw;
  typedef Vec<E, V, ODD> Row;
  typedef Columns<V, ODD> Cols;
  constexpr int R = BLOCK / TPR;
  __shared__ float slots[BLOCK / 64 + 1];
  const int i = threadIdx.x % TPR, r = threadIdx.x / TPR;
  float* slot = slots + r * (TPR / 64);
  typename Row::type xn[NV];
  auto fetch = [&](int64_t m) {
    const raw* x = static_cast<const raw*>(a.x) + m * a.ldx;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Cols c(i + j * TPR, a.N);
      xn[j] = Row::load(x + c.n, m < a.M && c.in, raw(0));
    }
  };
  fetch((int64_t)blockIdx.x * R + r);
  float w[NV][V], b[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const Cols c(i + j * TPR, a.N);
    load_param<P, V, ODD>(a.weight, c.n, c.in, 1.f, w[j]);
    load_param<P, V, ODD>(a.bias, c.n, c.in, 0.f, b[j]);
  }
  const int64_t step = (int64_t)gridDim.x * R;
  for (int64_t m0 = (int64_t)blockIdx.x * R; m0 < a.M; m0 += step) {
    const int64_t m = m0 + r;
    float x[NV][V], s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Cols c(i + j * TPR, a.N);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        x[j][e] = E::get(xn[j][e]);
        s[0] += c.own(e) ? x[j][e] : 0.f;
      }
    }
    fetch(m + step);
    row_sums<TPR>(s, slot);
    const float mean = s[0] / (float)a.N;
    s[0] = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Cols c(i + j * TPR, a.N);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        x[j][e] -= mean;
        s[0] += c.in && c.own(e) ? x[j][e] * x[j][e] : 0.f;
      }
    }
    row_sums<TPR>(s, slot);
    const float rstd = 1.f / sqrtf(s[0] / (float)a.N + a.eps);
    if (m < a.M) {
      raw* y = static_cast<raw*>(a.y) + m * a.ldy;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const Cols c(i + j * TPR, a.N);
        typename Row::type out;
#pragma unroll
        for (int e = 0; e < V; ++e) out[e] = E::put(__builtin_fmaf(x[j][e] * rstd, w[j][e], b[j][e]));
        Row::store(y + c.n, c.in, out);
      }
      if (i == 0) {
        if (a.mean != nullptr) a.mean[m] = mean;
        if (a.rstd != nullptr) a.rstd[m] = rstd;
      }
    }
  }
}

// Rows wider than the registers of a workgroup (or narrower than a vector): three
// reads of the row, the later two from the caches, element by element: 4096 x 16392
// bf16 takes 117 us (2.3 TB/s; x 16384, in registers, 46), and a row of 4 columns a
// workgroup of its own, 2^20 rows 3.3 ms (of 8 columns, in registers, 63 us).  A
// workgroup takes rows r, r + grid, ...
template <class E, class P>
__global__ void __launch_bounds__(1024) norm_wide_kernel(NormArgs a) {
  typedef typename E::raw raw;
  __shared__ float slots[16];
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    const raw* x = static_cast<const raw*>(a.x) + m * a.ldx;
    raw* y = static_cast<raw*>(a.y) + m * a.ldy;
    float s[1] = {0.f};
    for (int n = threadIdx.x; n < a.N; n += 1024) s[0] += E::get(x[n]);
    row_sums<1024>(s, slots);
    const float mean = s[0] / (float)a.N;
    s[0] = 0.f;
    for (int n = threadIdx.x; n < a.N; n += 1024) {
      const float c = E::get(x[n]) - mean;
      s[0] = __builtin_fmaf(c, c, s[0]);
    }
    row_sums<1024>(s, slots);
    const float rstd = 1.f / sqrtf(s[0] / (float)a.N + a.eps);
    for (int n = threadIdx.x; n < a.N; n += 1024) {
      float w[1], b[1];
      load_param<P, 1, false>(a.weight, n, true, 1.f, w);
      load_param<P, 1, false>(a.bias, n, true, 0.f, b);
      y[n] = E::put(__builtin_fmaf((E::get(x[n]) - mean) * rstd, w[0], b[0]));
    }
    if (threadIdx.x == 0) {
      if (a.mean != nullptr) a.mean[m] = mean;
      if (a.rstd != nullptr) a.rstd[m] = rstd;
    }
  }
}

// Backward, in the same way; what a vector has again counts in dx alone.
template <class E, class P, int V, bool ODD, int TPR, int NV, int BLOCK>
__global__ void __launch_bounds__(BLOCK) norm_backward_kernel(NormArgs a) {
  typedef typename E::raw raw;
  typedef Vec<E, V, ODD> Row;
  typedef typename Row::type vec;
  typedef Columns<V, ODD> Cols;
  constexpr int R = BLOCK / TPR;
  __shared__ float slots[2 * (BLOCK / 64) + 2];
  extern __shared__ float comb[];  // [R - 1][V NV][TPR]
  const int i = threadIdx.x % TPR, r = threadIdx.x / TPR;
  float* slot = slots + 2 * r * (TPR / 64);
  vec xn[NV], dn[NV];
  auto fetch = [&](int64_t m) {
    const raw* x = static_cast<const raw*>(a.x) + m * a.ldx;
    const raw* dy = static_cast<const raw*>(a.dy) + m * a.lddy;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Cols c(i + j * TPR, a.N);
      xn[j] = Row::load(x + c.n, m < a.M && c.in, raw(0));
      dn[j] = Row::load(dy + c.n, m < a.M && c.in, raw(0));
    }
  };
  fetch((int64_t)blockIdx.x * R + r);
  float dw[NV][V], db[NV][V], w[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const Cols c(i + j * TPR, a.N);
    load_param<P, V, ODD>(a.weight, c.n, c.in, 1.f, w[j]);
#pragma unroll
    for (int e = 0; e < V; ++e) dw[j][e] = db[j][e] = 0.f;
  }
  const int64_t step = (int64_t)gridDim.x * R;
  for (int64_t m0 = (int64_t)blockIdx.x * R; m0 < a.M; m0 += step) {
    const int64_t m = m0 + r;
    const bool live = m < a.M;
    const float mean = live ? a.mean_in[m] : 0.f, rstd = live ? a.rstd_in[m] : 0.f;
    vec xv[NV], dv[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      xv[j] = xn[j];
      dv[j] = dn[j];
    }
    fetch(m + step);
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      // (vectors that do not exist: dy is 0 there, and so is all that follows)
      const Cols k(i + j * TPR, a.N);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float d = k.own(e) ? E::get(dv[j][e]) : 0.f, c = (E::get(xv[j][e]) - mean) * rstd, g = d * w[j][e];
        dw[j][e] = __builtin_fmaf(d, c, dw[j][e]);
        db[j][e] += d;
        s[0] += g;
        s[1] = __builtin_fmaf(g, c, s[1]);
      }
    }
    row_sums<TPR>(s, slot);
    const float g0 = s[0] / (float)a.N, g1 = s[1] / (float)a.N;
    if (live && a.y != nullptr) {
      raw* dx = static_cast<raw*>(a.y) + m * a.ldy;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const Cols k(i + j * TPR, a.N);
        vec out;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float c = (E::get(xv[j][e]) - mean) * rstd, g = E::get(dv[j][e]) * w[j][e];
          out[e] = E::put(rstd * (g - g0 - c * g1));
        }
        Row::store(dx + k.n, k.in, out);
      }
    }
  }
  if (a.partial == nullptr) return;
  // The R row sets of the workgroup are added in order, dw and then db.
  float* out = a.partial + (size_t)blockIdx.x * 2 * a.N;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if constexpr (R > 1) {
      __syncthreads();
      if (r > 0)
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int e = 0; e < V; ++e) comb[((r - 1) * NV * V + j * V + e) * TPR + i] = which ? db[j][e] : dw[j][e];
      __syncthreads();
    }
    if (r == 0) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const Cols k(i + j * TPR, a.N);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float t = which ? db[j][e] : dw[j][e];
          for (int q = 0; q < R - 1; ++q) t += comb[(q * NV * V + j * V + e) * TPR + i];
          if (k.in && k.own(e)) out[(size_t)which * a.N + k.n + e] = t;
        }
      }
    }
  }
}

// dx of rows wider than the registers of a workgroup, or narrower than a vector; with
// the parameters' sums x and dy are read three times (4096 x 12296 bf16 148 us, 2.0
// TB/s; x 12288 67 us, 4.5 TB/s).
template <class E, class P>
__global__ void __launch_bounds__(1024) norm_backward_wide_kernel(NormArgs a) {
  typedef typename E::raw raw;
  __shared__ float slots[32];
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    const raw* x = static_cast<const raw*>(a.x) + m * a.ldx;
    const raw* dy = static_cast<const raw*>(a.dy) + m * a.lddy;
    raw* dx = static_cast<raw*>(a.y) + m * a.ldy;
    const float mean = a.mean_in[m], rstd = a.rstd_in[m];
    float s[2] = {0.f, 0.f};
    for (int n = threadIdx.x; n < a.N; n += 1024) {
      float w[1];
      load_param<P, 1, false>(a.weight, n, true, 1.f, w);
      const float g = E::get(dy[n]) * w[0];
      s[0] += g;
      s[1] = __builtin_fmaf(g, (E::get(x[n]) - mean) * rstd, s[1]);
    }
    row_sums<1024>(s, slots);
    const float g0 = s[0] / (float)a.N, g1 = s[1] / (float)a.N;
    for (int n = threadIdx.x; n < a.N; n += 1024) {
      float w[1];
      load_param<P, 1, false>(a.weight, n, true, 1.f, w);
      const float c = (E::get(x[n]) - mean) * rstd, g = E::get(dy[n]) * w[0];
      dx[n] = E::put(rstd * (g - g0 - c * g1));
    }
  }
}

// The parameters' partial sums of such rows: workgroup (x, y) sums 256 columns
// over every gridDim.y-th row.
template <class E>
__global__ void __launch_bounds__(256) norm_columns_kernel(NormArgs a) {
  typedef typename E::raw raw;
  const int n = blockIdx.x * 256 + threadIdx.x;
  if (n >= a.N) return;
  float dw = 0.f, db = 0.f;
  for (int64_t m = blockIdx.y; m < a.M; m += gridDim.y) {
    const float d = E::get(static_cast<const raw*>(a.dy)[m * a.lddy + n]);
    const float c = (E::get(static_cast<const raw*>(a.x)[m * a.ldx + n]) - a.mean_in[m]) * a.rstd_in[m];
    dw = __builtin_fmaf(d, c, dw);
    db += d;
  }
  a.partial[(size_t)blockIdx.y * 2 * a.N + n] = dw;
  a.partial[(size_t)blockIdx.y * 2 * a.N + a.N + n] = db;
}

// Adds `count` partial sums [count][2][N]: 64 of the 2 N columns a workgroup,
// 16 threads on each, each taking every 16th partial in order (512 of 5760
// columns, 24 MB, 5 us).
template <class P>
__global__ void __launch_bounds__(1024) norm_params_kernel(const float* partial, int count, int N, void* dweight,
                                                           void* dbias) {
  typedef typename P::raw raw;
  __shared__ float part[16][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  for (int64_t c0 = (int64_t)blockIdx.x * 64; c0 < 2ll * N; c0 += (int64_t)gridDim.x * 64) {
    const int64_t c = c0 + lane;
    float s = 0.f;
    if (c < 2ll * N) {
      constexpr int kAhead = 8;
      for (int g0 = w; g0 < count; g0 += 16 * kAhead) {
        float x[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int g = g0 + 16 * i;
          x[i] = g < count ? partial[(size_t)g * 2 * N + c] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) s += x[i];
      }
    }
    part[w][lane] = s;
    __syncthreads();
    if (w == 0 && c < 2ll * N) {
      s = 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j) s += part[j][lane];
      raw* out = static_cast<raw*>(c < N ? dweight : dbias);
      if (out != nullptr) out[c < N ? c : c - N] = P::put(s);
    }
    __syncthreads();  // before the next columns' sums
  }
}

// Threads a row (TPR) and vectors a thread (NV) for rows of N: the fewest
// threads whose registers hold the row, so that most of a vector load's lanes
// are used; vectors of 16 bytes, up to `columns` elements a thread.
struct Shape {
  bool odd;
  int tpr, nv;  // tpr 0: the row does not fit
};
Shape shape_of(int N, int elems, bool odd, int columns) {
  static const int kShapes[][2] = {{16, 1},  {16, 2},  {64, 1},  {64, 2},  {64, 3},  {128, 2}, {128, 3},
                                   {256, 2}, {256, 3}, {256, 4}, {512, 3}, {512, 4}, {512, 6}};
  const int units = (N + elems - 1) / elems;
  if (N < elems) return {odd, 0, 0};  // (narrower than a vector: as the widest)
  for (const auto& p : kShapes)
    if (p[0] * p[1] >= units && p[1] * elems <= columns) return {odd, p[0], p[1]};
  return {odd, 0, 0};
}

// Workgroups of 1024 threads for `tasks`: a launch counts threads in 32 bits.
unsigned workgroups(int64_t tasks) { return (unsigned)(tasks < 1 << 20 ? tasks : 1 << 20); }

bool aligned16(const void* p) { return (uintptr_t)p % 16 == 0; }

// (odd: not every row and parameter vector starts at a multiple of 16 bytes)
Shape shape_for(const NormArgs& a, prnnDataType_t type, bool backward) {
  const int elems = type == PRNN_DATA_FLOAT ? 4 : 8;
  bool whole = a.N % elems == 0 && a.ldx % elems == 0 && aligned16(a.x) && aligned16(a.weight) && aligned16(a.bias) &&
               (a.y == nullptr || (a.ldy % elems == 0 && aligned16(a.y)));
  if (backward) whole = whole && a.lddy % elems == 0 && aligned16(a.dy);
  return shape_of(a.N, elems, !whole, backward ? 24 : 32);  // (the backward pass holds five values a column)
}

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

}  // namespace

hipError_t launch_layer_norm(const NormArgs& a, prnnDataType_t type, prnnDataType_t ptype, hipStream_t stream) {
  const Shape s = shape_for(a, type, false);
  return for_types(type, ptype, [&](auto e, auto p) {
    typedef decltype(e) E;
    typedef decltype(p) P;
    constexpr int V = E::id == PRNN_DATA_FLOAT ? 4 : 8;
    const bool fits = for_shape<V, 32>(s, [&](auto c) {
      typedef decltype(c) C;
      const int64_t sets = (a.M + C::block / C::tpr - 1) / (C::block / C::tpr);
      // Four workgroups on a compute unit.  Measured (1 / 2 / 4 / 8 on each / one for every row set): 16384 x 5760
      // bf16 119 / 75 / 73 / 72 / 87 us, 50000 x 500 bf16 24 / 19 / 20 / 19 / 21, 3000 x 4096 fp32 21 / 17 / 16 / 16 / 16.
      const int64_t most = 4ll * a.compute_units, grid = sets < most ? sets : most;
      norm_kernel<E, P, C::v, C::odd, C::tpr, C::nv, C::block><<<(unsigned)grid, C::block, 0, stream>>>(a);
    });
    if (!fits) norm_wide_kernel<E, P><<<workgroups(a.M), 1024, 0, stream>>>(a);
    return hipGetLastError();
  });
}

int layer_norm_backward_grid(const NormArgs& a, prnnDataType_t type, int compute_units) {
  const Shape s = shape_for(a, type, true);
  if (s.tpr == 0) return (int)(a.M < 64 ? a.M : 64);
  const int R = block_of(s.tpr) / s.tpr;
  const int64_t sets = (a.M + R - 1) / R;
  // Two workgroups of 256 threads on a compute unit, one of 512: more leave
  // more partial sums than their loads in flight gain.  Measured (1 / 2 / 3 on
  // each): 16384 x 5760 bf16 140 / 115 / 133 us, 3000 x 12000 bf16 48 / 58 / 70.
  const int64_t most = (s.tpr > 256 ? 1ll : 2ll) * compute_units;
  return (int)(sets < most ? sets : most);
}

hipError_t launch_layer_norm_backward(const NormArgs& a, prnnDataType_t type, prnnDataType_t ptype, int grid,
                                      hipStream_t stream) {
  const Shape s = shape_for(a, type, true);
  return for_types(type, ptype, [&](auto e, auto p) {
    typedef decltype(e) E;
    typedef decltype(p) P;
    constexpr int V = E::id == PRNN_DATA_FLOAT ? 4 : 8;
    if (grid > 0) {
      const bool fits = for_shape<V, 24>(s, [&](auto c) {
        typedef decltype(c) C;
        constexpr int R = C::block / C::tpr;
        norm_backward_kernel<E, P, C::v, C::odd, C::tpr, C::nv, C::block>
            <<<grid, C::block, (R - 1) * C::v * C::nv * C::tpr * 4, stream>>>(a);
      });
      if (!fits) {
        // the columns first: dx may be written over x or dy
        if (a.partial != nullptr) norm_columns_kernel<E><<<dim3((a.N + 255) / 256, grid), 256, 0, stream>>>(a);
        if (a.y != nullptr) norm_backward_wide_kernel<E, P><<<workgroups(a.M), 1024, 0, stream>>>(a);
      }
    }
    if (a.dweight != nullptr || a.dbias != nullptr)
      norm_params_kernel<P><<<workgroups((2ll * a.N + 63) / 64), 1024, 0, stream>>>(a.partial, grid, a.N, a.dweight,
                                                                                   a.dbias);
    return hipGetLastError();
  });
}

}  // namespace prnn
