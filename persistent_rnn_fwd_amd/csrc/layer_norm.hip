// Layer norm over rows of N, forward and backward.
//
//   y = (x - mean) rstd w + b
//   dx = rstd (g - mean(g) - n mean(g n)),  dw = sum_m dy n,  db = sum_m dy,
//   with n = (x - mean) rstd and g = dy w
//
// Both passes are bound by memory: x in and y out, or x and dy in and dx out.
// A row is read once into the registers of TPR threads, 16 bytes at a time
// where width, strides and addresses allow it (V elements a vector, NV vectors
// a thread), so mean and variance are sums over centred values without a
// second read.  In the backward pass the threads of a row keep their columns
// from row to row, so the parameters' gradients are sums in registers; each
// workgroup leaves one partial sum and a second kernel adds those in a fixed
// order.
#include "device_common.h"
#include "sequence.h"

namespace prnn {
namespace {

template <class E, int V>
struct Vec {
  typedef typename E::raw raw;
  typedef raw type __attribute__((ext_vector_type(V)));
};

// Parameters: fp32 or the rows' own type; absent ones are a constant.
template <class P, int V>
__device__ __forceinline__ void load_param(const void* p, int n, bool in, float absent, float (&f)[V]) {
  typedef typename Vec<P, V>::type vec;
  if (p != nullptr && in) {
    const vec v = *reinterpret_cast<const vec*>(static_cast<const typename P::raw*>(p) + n);
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = P::get(v[e]);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = absent;
  }
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

template <class E, class P, int V, int TPR, int NV, int BLOCK>
__global__ void __launch_bounds__(BLOCK) norm_kernel(NormArgs a) {
  typedef typename E::raw raw;
  typedef typename Vec<E, V>::type vec;
  __shared__ float slots[BLOCK / 64 + 1];
  const int i = threadIdx.x % TPR, r = threadIdx.x / TPR;
  float* slot = slots + r * (TPR / 64);
  const int64_t m = (int64_t)blockIdx.x * (BLOCK / TPR) + r;
  const bool live = m < a.M;
  const raw* x = static_cast<const raw*>(a.x) + m * a.ldx;
  vec xv[NV];
  float s[1] = {0.f};
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int n = (i + j * TPR) * V;
    xv[j] = live && n < a.N ? *reinterpret_cast<const vec*>(x + n) : vec(raw(0));
  }
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < V; ++e) s[0] += E::get(xv[j][e]);
  row_sums<TPR>(s, slot);
  const float mean = s[0] / (float)a.N;
  s[0] = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const bool in = (i + j * TPR) * V < a.N;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const float c = E::get(xv[j][e]) - mean;
      s[0] += in ? c * c : 0.f;
    }
  }
  row_sums<TPR>(s, slot);
  const float rstd = 1.f / sqrtf(s[0] / (float)a.N + a.eps);
  if (!live) return;
  raw* y = static_cast<raw*>(a.y) + m * a.ldy;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int n = (i + j * TPR) * V;
    float w[V], b[V];
    load_param<P, V>(a.weight, n, n < a.N, 1.f, w);
    load_param<P, V>(a.bias, n, n < a.N, 0.f, b);
    vec out;
#pragma unroll
    for (int e = 0; e < V; ++e) out[e] = E::put(__builtin_fmaf((E::get(xv[j][e]) - mean) * rstd, w[e], b[e]));
    if (n < a.N) *reinterpret_cast<vec*>(y + n) = out;
  }
  if (i == 0) {
    if (a.mean != nullptr) a.mean[m] = mean;
    if (a.rstd != nullptr) a.rstd[m] = rstd;
  }
}

// Rows wider than the registers of a workgroup: three reads of the row, the
// later two from the caches.
template <class E, class P>
__global__ void __launch_bounds__(1024) norm_wide_kernel(NormArgs a) {
  typedef typename E::raw raw;
  __shared__ float slots[16];
  const int64_t m = blockIdx.x;
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
    load_param<P, 1>(a.weight, n, true, 1.f, w);
    load_param<P, 1>(a.bias, n, true, 0.f, b);
    y[n] = E::put(__builtin_fmaf((E::get(x[n]) - mean) * rstd, w[0], b[0]));
  }
  if (threadIdx.x == 0) {
    if (a.mean != nullptr) a.mean[m] = mean;
    if (a.rstd != nullptr) a.rstd[m] = rstd;
  }
}

// Backward.  The grid's row sets take rows r, r + R grid, ...; thread i of a
// set keeps columns V (i + j TPR) .. + V - 1.
template <class E, class P, int V, int TPR, int NV, int BLOCK>
__global__ void __launch_bounds__(BLOCK) norm_backward_kernel(NormArgs a) {
  typedef typename E::raw raw;
  typedef typename Vec<E, V>::type vec;
  constexpr int R = BLOCK / TPR;
  __shared__ float slots[2 * (BLOCK / 64) + 2];
  extern __shared__ float comb[];  // [R - 1][V NV][TPR]
  const int i = threadIdx.x % TPR, r = threadIdx.x / TPR;
  float* slot = slots + 2 * r * (TPR / 64);
  float dw[NV][V], db[NV][V], w[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int n = (i + j * TPR) * V;
    load_param<P, V>(a.weight, n, n < a.N, 1.f, w[j]);
#pragma unroll
    for (int e = 0; e < V; ++e) dw[j][e] = db[j][e] = 0.f;
  }
  vec xn[NV], dn[NV];
  auto fetch = [&](int64_t m) {
    const raw* x = static_cast<const raw*>(a.x) + m * a.ldx;
    const raw* dy = static_cast<const raw*>(a.dy) + m * a.lddy;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int n = (i + j * TPR) * V;
      const bool in = m < a.M && n < a.N;
      xn[j] = in ? *reinterpret_cast<const vec*>(x + n) : vec(raw(0));
      dn[j] = in ? *reinterpret_cast<const vec*>(dy + n) : vec(raw(0));
    }
  };
  // The next row's loads are issued before this row's sums where there are
  // registers for them.
  constexpr bool kAhead = V > 1 || NV <= 16;
  const int64_t step = (int64_t)gridDim.x * R;
  if (kAhead) fetch((int64_t)blockIdx.x * R + r);
  for (int64_t m0 = (int64_t)blockIdx.x * R; m0 < a.M; m0 += step) {
    const int64_t m = m0 + r;
    const bool live = m < a.M;
    const float mean = live ? a.mean_in[m] : 0.f, rstd = live ? a.rstd_in[m] : 0.f;
    vec xv[NV], dv[NV];
    if (!kAhead) fetch(m);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      xv[j] = xn[j];
      dv[j] = dn[j];
    }
    if (kAhead) fetch(m + step);
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      // (columns past N: dy is 0 there, and so is all that follows)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float d = E::get(dv[j][e]), c = (E::get(xv[j][e]) - mean) * rstd, g = d * w[j][e];
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
        const int n = (i + j * TPR) * V;
        vec out;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float c = (E::get(xv[j][e]) - mean) * rstd, g = E::get(dv[j][e]) * w[j][e];
          out[e] = E::put(rstd * (g - g0 - c * g1));
        }
        if (n < a.N) *reinterpret_cast<vec*>(dx + n) = out;
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
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) {
          float t = which ? db[j][e] : dw[j][e];
          for (int q = 0; q < R - 1; ++q) t += comb[(q * NV * V + j * V + e) * TPR + i];
          const int n = (i + j * TPR) * V + e;
          if (n < a.N) out[(size_t)which * a.N + n] = t;
        }
    }
  }
}

// dx of rows wider than the registers of a workgroup.
template <class E, class P>
__global__ void __launch_bounds__(1024) norm_backward_wide_kernel(NormArgs a) {
  typedef typename E::raw raw;
  __shared__ float slots[32];
  const int64_t m = blockIdx.x;
  const raw* x = static_cast<const raw*>(a.x) + m * a.ldx;
  const raw* dy = static_cast<const raw*>(a.dy) + m * a.lddy;
  raw* dx = static_cast<raw*>(a.y) + m * a.ldy;
  const float mean = a.mean_in[m], rstd = a.rstd_in[m];
  float s[2] = {0.f, 0.f};
  for (int n = threadIdx.x; n < a.N; n += 1024) {
    float w[1];
    load_param<P, 1>(a.weight, n, true, 1.f, w);
    const float g = E::get(dy[n]) * w[0];
    s[0] += g;
    s[1] = __builtin_fmaf(g, (E::get(x[n]) - mean) * rstd, s[1]);
  }
  row_sums<1024>(s, slots);
  const float g0 = s[0] / (float)a.N, g1 = s[1] / (float)a.N;
  for (int n = threadIdx.x; n < a.N; n += 1024) {
    float w[1];
    load_param<P, 1>(a.weight, n, true, 1.f, w);
    const float c = (E::get(x[n]) - mean) * rstd, g = E::get(dy[n]) * w[0];
    dx[n] = E::put(rstd * (g - g0 - c * g1));
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
// 16 threads on each, each taking every 16th partial in order.
template <class P>
__global__ void __launch_bounds__(1024) norm_params_kernel(const float* partial, int count, int N, void* dweight,
                                                           void* dbias) {
  typedef typename P::raw raw;
  __shared__ float part[16][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + lane;
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
  if (w != 0 || c >= 2ll * N) return;
  s = 0.f;
#pragma unroll
  for (int j = 0; j < 16; ++j) s += part[j][lane];
  raw* out = static_cast<raw*>(c < N ? dweight : dbias);
  if (out != nullptr) out[c < N ? c : c - N] = P::put(s);
}

// Threads a row (TPR) and vectors a thread (NV) for rows of N: the fewest
// threads whose registers hold the row, so that most of a vector load's lanes
// are used; vectors of 16 bytes, up to `columns` elements a thread, or single
// elements.
struct Shape {
  bool vec;
  int tpr, nv;  // tpr 0: the row does not fit
};
Shape shape_of(int N, int elems, bool vec, int columns) {
  Shape s = {vec, 0, 0};
  const int units = vec ? N / elems : N;
  if (vec) {
    static const int kShapes[][2] = {{16, 1}, {16, 2}, {16, 4}, {64, 2}, {64, 4}, {256, 2}, {256, 3}, {256, 4}, {512, 3}, {512, 4}, {512, 6}};
    for (const auto& p : kShapes)
      if (p[0] * p[1] >= units && p[1] * elems <= columns) {
        s.tpr = p[0];
        s.nv = p[1];
        return s;
      }
  } else {
    static const int kShapes[][2] = {{16, 8}, {64, 4}, {64, 8}, {256, 5}, {256, 8}, {512, 8}, {512, 16}, {512, 24}};
    for (const auto& p : kShapes)
      if (p[0] * p[1] >= units) {
        s.tpr = p[0];
        s.nv = p[1];
        return s;
      }
  }
  return s;
}

bool aligned16(const void* p) { return (uintptr_t)p % 16 == 0; }

// Whether every row and parameter vector starts at a multiple of 16 bytes.
Shape shape_for(const NormArgs& a, prnnDataType_t type, bool backward) {
  const int elems = type == PRNN_DATA_FLOAT ? 4 : 8;
  bool vec = a.N % elems == 0 && a.ldx % elems == 0 && aligned16(a.x) && aligned16(a.weight) && aligned16(a.bias) &&
             (a.y == nullptr || (a.ldy % elems == 0 && aligned16(a.y)));
  if (backward) vec = vec && a.lddy % elems == 0 && aligned16(a.dy);
  return shape_of(a.N, elems, vec, backward ? 24 : 32);  // (the backward pass holds five values a column)
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

template <int V, int TPR, int NV>
struct Config {
  static constexpr int v = V, tpr = TPR, nv = NV, block = block_of(TPR);
};

// Calls f(Config) for the shape; false when the row does not fit.  COLUMNS: as
// shape_of's.
template <int V, int COLUMNS, class F>
bool for_shape(const Shape& s, F f) {
#define PRNN_SHAPE(VV, TPR, NV)                 \
  if (s.tpr == TPR && s.nv == NV) {             \
    f(Config<VV, TPR, NV>());                   \
    return true;                                \
  }
  if (s.vec) {
    PRNN_SHAPE(V, 16, 1) PRNN_SHAPE(V, 16, 2) PRNN_SHAPE(V, 64, 2)
    if constexpr (V == 4 || COLUMNS == 32) {
      PRNN_SHAPE(V, 16, 4) PRNN_SHAPE(V, 64, 4)
    }
    PRNN_SHAPE(V, 256, 2) PRNN_SHAPE(V, 256, 3) PRNN_SHAPE(V, 512, 3)
    if constexpr (V == 4 || COLUMNS == 32) {
      PRNN_SHAPE(V, 256, 4) PRNN_SHAPE(V, 512, 4)
    }
    if constexpr (V == 4) {
      PRNN_SHAPE(V, 512, 6)
    }
  } else {
    PRNN_SHAPE(1, 16, 8) PRNN_SHAPE(1, 64, 4) PRNN_SHAPE(1, 64, 8) PRNN_SHAPE(1, 256, 5) PRNN_SHAPE(1, 256, 8)
    PRNN_SHAPE(1, 512, 8) PRNN_SHAPE(1, 512, 16) PRNN_SHAPE(1, 512, 24)
  }
#undef PRNN_SHAPE
  return false;
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
      const int64_t grid = (a.M + C::block / C::tpr - 1) / (C::block / C::tpr);
      norm_kernel<E, P, C::v, C::tpr, C::nv, C::block><<<(unsigned)grid, C::block, 0, stream>>>(a);
    });
    if (!fits) norm_wide_kernel<E, P><<<(unsigned)a.M, 1024, 0, stream>>>(a);
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
  // each): 16384 x 5760 bf16 137 / 125 / 139 us, 3000 x 12000 bf16 58 / 76 / 98.
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
        norm_backward_kernel<E, P, C::v, C::tpr, C::nv, C::block>
            <<<grid, C::block, (R - 1) * C::v * C::nv * C::tpr * 4, stream>>>(a);
      });
      if (!fits) {
        // the columns first: dx may be written over x or dy
        if (a.partial != nullptr) norm_columns_kernel<E><<<dim3((a.N + 255) / 256, grid), 256, 0, stream>>>(a);
        if (a.y != nullptr) norm_backward_wide_kernel<E, P><<<(unsigned)a.M, 1024, 0, stream>>>(a);
      }
    }
    if (a.dweight != nullptr || a.dbias != nullptr)
      norm_params_kernel<P><<<(unsigned)((2ll * a.N + 63) / 64), 1024, 0, stream>>>(a.partial, grid, a.N, a.dweight,
                                                                                   a.dbias);
    return hipGetLastError();
  });
}

}  // namespace prnn
