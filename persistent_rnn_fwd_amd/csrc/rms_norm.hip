// Rms norm over rows of N, with the residual's addition and an 8-bit output,
// and its gradients.
//
//   s = x + residual,  y = s rstd w,  rstd = 1 / sqrt(mean(s^2) + eps)
//   8 bits: scale = max(max |y| / 448, 2^-126) over a row or 128 columns, y / scale as e4m3
//   dx = rstd (g - n mean(g n)) + dsum,  dw = sum_m dy n,  with n = s rstd and g = dy w
//
// Built like layer norm (layer_norm.hip): bound by memory (measured: see the launch; gradients of
// 16384 x 5760 bf16 148 us, 5.1 TB/s, a large copy reaches 4.8), a row is read once into
// the registers of TPR threads, 16 bytes at a time, with the next row's loads in
// flight; the sum s stays in fp32 between its addition and the norm and is
// rounded once where it is stored, as y is.  The scale of 128 columns is a
// maximum over the 16 or 32 lanes that hold them; y / scale is rounded once in fp32
// before it is rounded to e4m3 (nearest, ties to even) and cannot pass 448 by as much as its
// last step, so nothing is clamped.
#include "norm_rows.h"
#include "rms_norm.h"

namespace prnn {
namespace {

using namespace norm;

// Maximum over rows of 16 lanes, the same in each of them (by exchanges through LDS's network).
__device__ __forceinline__ float max16(float x) {
#pragma unroll
  for (int m = 1; m < 16; m *= 2) x = fmaxf(x, __shfl_xor(x, m));
  return x;
}

// ... over the TPR threads of a row (see row_sums).
template <int TPR>
__device__ __forceinline__ float row_max(float x, float* slot) {
  x = max16(x);
  if constexpr (TPR >= 64) {
    x = fmaxf(x, __shfl_xor(x, 16));
    x = fmaxf(x, __shfl_xor(x, 32));
  }
  if constexpr (TPR > 64) {
    constexpr int W = TPR / 64;
    __syncthreads();
    if ((threadIdx.x & 63) == 0) slot[threadIdx.x % TPR / 64] = x;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < W; ++j) x = fmaxf(x, slot[j]);
  }
  return x;
}

__device__ __forceinline__ float scale_of(float most) { return fmaxf(most / 448.f, 0x1p-126f); }

// A group's scale as y is divided by it: y / scale is y times the reciprocal and one step
// of its residual, rounded once.  (An infinite scale is that of a row with an infinity:
// what is finite there becomes 0.)
struct Scale {
  float finite, inverse;
  __device__ __forceinline__ explicit Scale(float scale) : finite(fminf(scale, 0x1.fffffep127f)), inverse(1.f / scale) {}
  __device__ __forceinline__ float under(float y) const {
    const float q = y * inverse;
    return __builtin_fmaf(__builtin_fmaf(-q, finite, y), inverse, q);
  }
};

// V values in 8 bits.
template <int V>
__device__ __forceinline__ void eights(const float (&y)[V], const Scale& s, uint32_t (&out)[V / 4]) {
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(s.under(y[i]), s.under(y[i + 1]), 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(s.under(y[i + 2]), s.under(y[i + 3]), w, true);
    out[i / 4] = (uint32_t)w;
  }
}

// Forward; thread i of a row set keeps the weights of vectors i + j TPR.
template <class E, class P, int V, bool ODD, int TPR, int NV, int BLOCK, bool EIGHT>
__global__ void __launch_bounds__(BLOCK) rms_kernel(RmsArgs a) {
  typedef typename E::raw raw;
  typedef Vec<E, V, ODD> Row;
  typedef Columns<V, ODD> Cols;
  constexpr int R = BLOCK / TPR;
  __shared__ float slots[BLOCK / 64 + 1];
  const int i = threadIdx.x % TPR, r = threadIdx.x / TPR;
  float* slot = slots + r * (TPR / 64);
  typename Row::type xn[NV], rn[NV];
  auto fetch = [&](int64_t m) {
    const raw* x = static_cast<const raw*>(a.x) + m * a.ldx;
    const raw* res = static_cast<const raw*>(a.residual) + m * a.ldr;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Cols c(i + j * TPR, a.N);
      xn[j] = Row::load(x + c.n, m < a.M && c.in, raw(0));
      rn[j] = Row::load(res + c.n, a.residual != nullptr && m < a.M && c.in, raw(0));
    }
  };
  fetch((int64_t)blockIdx.x * R + r);
  float w[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const Cols c(i + j * TPR, a.N);
    load_param<P, V, ODD>(a.weight, c.n, c.in, 1.f, w[j]);
  }
  const int groups = EIGHT ? (a.group > 0 ? (a.N + kRmsGroup - 1) / kRmsGroup : 1) : 0;
  const int64_t step = (int64_t)gridDim.x * R;
  for (int64_t m0 = (int64_t)blockIdx.x * R; m0 < a.M; m0 += step) {
    const int64_t m = m0 + r;
    const bool live = m < a.M;
    float x[NV][V], s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Cols c(i + j * TPR, a.N);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        x[j][e] = E::get(xn[j][e]) + E::get(rn[j][e]);
        s[0] = c.own(e) ? __builtin_fmaf(x[j][e], x[j][e], s[0]) : s[0];
      }
    }
    fetch(m + step);
    row_sums<TPR>(s, slot);
    const float rstd = 1.f / sqrtf(s[0] / (float)a.N + a.eps);
    if (live && a.sum != nullptr) {
      raw* sum = static_cast<raw*>(a.sum) + m * a.lds;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const Cols c(i + j * TPR, a.N);
        typename Row::type out;
#pragma unroll
        for (int e = 0; e < V; ++e) out[e] = E::put(x[j][e]);
        Row::store(sum + c.n, c.in, out);
      }
    }
    if (live && i == 0 && a.rstd != nullptr) a.rstd[m] = rstd;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) x[j][e] = x[j][e] * rstd * w[j][e];
    if constexpr (!EIGHT) {
      if (live) {
        raw* y = static_cast<raw*>(a.y) + m * a.ldy;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const Cols c(i + j * TPR, a.N);
          typename Row::type out;
#pragma unroll
          for (int e = 0; e < V; ++e) out[e] = E::put(x[j][e]);
          Row::store(y + c.n, c.in, out);
        }
      }
    } else {
      float most[NV], all = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const Cols c(i + j * TPR, a.N);
        most[j] = 0.f;
#pragma unroll
        for (int e = 0; e < V; ++e) most[j] = c.in && c.own(e) ? fmaxf(most[j], fabsf(x[j][e])) : most[j];
        all = fmaxf(all, most[j]);
      }
      constexpr int kLanes = kRmsGroup / V;  // that hold a group
      if (a.group == 0 || TPR < kLanes) {    // (TPR < kLanes: a row has one group)
        all = row_max<TPR>(all, slot);
#pragma unroll
        for (int j = 0; j < NV; ++j) most[j] = all;
      } else {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          most[j] = max16(most[j]);
          if (kLanes == 32) most[j] = fmaxf(most[j], __shfl_xor(most[j], 16));
        }
      }
      if (live) {
        uint8_t* y = static_cast<uint8_t*>(a.y) + m * a.ldy;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const int k = i + j * TPR;
          const Cols c(k, a.N);
          if (!c.in) continue;
          const float scale = scale_of(most[j]);
          uint32_t out[V / 4];
          eights<V>(x[j], Scale(scale), out);
          if (groups == 1 ? k == 0 : k % kLanes == 0) a.scales[m * groups + k / kLanes] = scale;
          if (ODD && c.again > 0) {  // the columns before may be another scale's
#pragma unroll
            for (int e = 0; e < V; ++e)
              if (c.own(e)) y[c.n + e] = (uint8_t)(out[e / 4] >> (8 * (e % 4)));
          } else {
            typedef uint32_t words __attribute__((ext_vector_type(V / 4 == 1 ? 1 : 2), aligned(ODD ? 1 : V)));
            words z;
#pragma unroll
            for (int e = 0; e < V / 4; ++e) z[e] = out[e];
            *reinterpret_cast<words*>(y + c.n) = z;
          }
        }
      }
    }
  }
}

// Rows wider than the registers of a workgroup (16384 columns of 16 bits, 12288 of fp32), or
// narrower than a vector: read twice (8 bits: three times), the later times from the
// caches, element by element.  A wave takes the groups that have a scale in turn.  Simple,
// not fast: 4096 x 20480 bf16 with a residual 275 us (2.4 TB/s; 16384 columns, by vectors, 104
// us, 5.2 TB/s), in 8 bits 408, with a scale for 128 columns 459; 65536 x 4 bf16 180 us.
template <class E, class P, bool EIGHT>
__global__ void __launch_bounds__(1024) rms_wide_kernel(RmsArgs a) {
  typedef typename E::raw raw;
  __shared__ float slots[16];
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    const raw* x = static_cast<const raw*>(a.x) + m * a.ldx;
    const raw* res = a.residual != nullptr ? static_cast<const raw*>(a.residual) + m * a.ldr : nullptr;
    auto value = [&](int n) { return E::get(x[n]) + (res != nullptr ? E::get(res[n]) : 0.f); };
    float s[1] = {0.f};
    for (int n = threadIdx.x; n < a.N; n += 1024) {
      const float c = value(n);
      s[0] = __builtin_fmaf(c, c, s[0]);
    }
    row_sums<1024>(s, slots);
    const float rstd = 1.f / sqrtf(s[0] / (float)a.N + a.eps);
    auto normed = [&](int n) {
      float w[1];
      load_param<P, 1, false>(a.weight, n, true, 1.f, w);
      return value(n) * rstd * w[0];
    };
    if constexpr (!EIGHT) {
      raw* y = static_cast<raw*>(a.y) + m * a.ldy;
      for (int n = threadIdx.x; n < a.N; n += 1024) {
        const float f = normed(n), t = value(n);
        if (a.sum != nullptr) static_cast<raw*>(a.sum)[m * a.lds + n] = E::put(t);
        y[n] = E::put(f);
      }
    } else {
      uint8_t* y = static_cast<uint8_t*>(a.y) + m * a.ldy;
      const int groups = a.group > 0 ? (a.N + kRmsGroup - 1) / kRmsGroup : 1;
      auto put = [&](int n, const Scale& s8) {
        const float f = normed(n), t = value(n);
        if (a.sum != nullptr) static_cast<raw*>(a.sum)[m * a.lds + n] = E::put(t);
        y[n] = (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(s8.under(f), 0.f, 0, false);
      };
      if (a.group == 0) {
        float most = 0.f;
        for (int n = threadIdx.x; n < a.N; n += 1024) most = fmaxf(most, fabsf(normed(n)));
        const float scale = scale_of(row_max<1024>(most, slots));
        if (threadIdx.x == 0) a.scales[m] = scale;
        for (int n = threadIdx.x; n < a.N; n += 1024) put(n, Scale(scale));
      } else {
        const int lane = threadIdx.x & 63;
        for (int q = threadIdx.x >> 6; q < groups; q += 16) {
          const int n0 = q * kRmsGroup + lane, n1 = n0 + 64;
          float most = 0.f;
          if (n0 < a.N) most = fabsf(normed(n0));
          if (n1 < a.N) most = fmaxf(most, fabsf(normed(n1)));
#pragma unroll
          for (int d = 1; d < 64; d *= 2) most = fmaxf(most, __shfl_xor(most, d));
          const float scale = scale_of(most);
          if (lane == 0) a.scales[m * groups + q] = scale;
          if (n0 < a.N) put(n0, Scale(scale));
          if (n1 < a.N) put(n1, Scale(scale));
        }
      }
    }
    if (threadIdx.x == 0 && a.rstd != nullptr) a.rstd[m] = rstd;
  }
}

// Backward; what a vector has again counts in dx alone.
template <class E, class P, int V, bool ODD, int TPR, int NV, int BLOCK>
__global__ void __launch_bounds__(BLOCK) rms_backward_kernel(RmsArgs a) {
  typedef typename E::raw raw;
  typedef Vec<E, V, ODD> Row;
  typedef typename Row::type vec;
  typedef Columns<V, ODD> Cols;
  constexpr int R = BLOCK / TPR;
  constexpr bool kAhead = NV < 6;  // registers for the next row's loads
  __shared__ float slots[BLOCK / 64 + 1];
  extern __shared__ float comb[];  // [R - 1][V NV][TPR]
  const int i = threadIdx.x % TPR, r = threadIdx.x / TPR;
  float* slot = slots + r * (TPR / 64);
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
  if (kAhead) fetch((int64_t)blockIdx.x * R + r);
  float dw[NV][V], w[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const Cols c(i + j * TPR, a.N);
    load_param<P, V, ODD>(a.weight, c.n, c.in, 1.f, w[j]);
#pragma unroll
    for (int e = 0; e < V; ++e) dw[j][e] = 0.f;
  }
  const int64_t step = (int64_t)gridDim.x * R;
  for (int64_t m0 = (int64_t)blockIdx.x * R; m0 < a.M; m0 += step) {
    const int64_t m = m0 + r;
    const bool live = m < a.M;
    const float rstd = live ? a.rstd_in[m] : 0.f;
    if (!kAhead) fetch(m);
    vec xv[NV], dv[NV], tv[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      xv[j] = xn[j];
      dv[j] = dn[j];
      const Cols k(i + j * TPR, a.N);
      tv[j] = Row::load(static_cast<const raw*>(a.dsum) + m * a.lds + k.n, a.dsum != nullptr && live && k.in, raw(0));
    }
    if (kAhead) fetch(m + step);
    float s[1] = {0.f};
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      // (vectors that do not exist: dy is 0 there, and so is all that follows)
      const Cols k(i + j * TPR, a.N);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float d = k.own(e) ? E::get(dv[j][e]) : 0.f, c = E::get(xv[j][e]) * rstd;
        dw[j][e] = __builtin_fmaf(d, c, dw[j][e]);
        s[0] = __builtin_fmaf(d * w[j][e], c, s[0]);
      }
    }
    row_sums<TPR>(s, slot);
    const float along = s[0] / (float)a.N;
    if (live && a.y != nullptr) {
      raw* dx = static_cast<raw*>(a.y) + m * a.ldy;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const Cols k(i + j * TPR, a.N);
        vec out;
#pragma unroll
        for (int e = 0; e < V; ++e) {
          const float c = E::get(xv[j][e]) * rstd, g = E::get(dv[j][e]) * w[j][e];
          out[e] = E::put(__builtin_fmaf(rstd, __builtin_fmaf(-c, along, g), E::get(tv[j][e])));
        }
        Row::store(dx + k.n, k.in, out);
      }
    }
  }
  if (a.partial == nullptr) return;
  // The R row sets of the workgroup are added in order.
  float* out = a.partial + (size_t)blockIdx.x * a.N;
  if constexpr (R > 1) {
    if (r > 0)
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) comb[((r - 1) * NV * V + j * V + e) * TPR + i] = dw[j][e];
    __syncthreads();
  }
  if (r == 0) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const Cols k(i + j * TPR, a.N);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float t = dw[j][e];
        for (int q = 0; q < R - 1; ++q) t += comb[(q * NV * V + j * V + e) * TPR + i];
        if (k.in && k.own(e)) out[k.n + e] = t;
      }
    }
  }
}

// dx of rows wider than the registers of a workgroup (12288 columns), or narrower than a
// vector.  With the weight's sums, which read x and dy once more: 4096 x 16384 bf16 with
// the sum's gradient 259 us (2.1 TB/s; 12288 columns, by vectors, 83 us, 4.9 TB/s).
template <class E, class P>
__global__ void __launch_bounds__(1024) rms_backward_wide_kernel(RmsArgs a) {
  typedef typename E::raw raw;
  __shared__ float slots[16];
  for (int64_t m = blockIdx.x; m < a.M; m += gridDim.x) {
    const raw* x = static_cast<const raw*>(a.x) + m * a.ldx;
    const raw* dy = static_cast<const raw*>(a.dy) + m * a.lddy;
    const raw* ds = a.dsum != nullptr ? static_cast<const raw*>(a.dsum) + m * a.lds : nullptr;
    raw* dx = static_cast<raw*>(a.y) + m * a.ldy;
    const float rstd = a.rstd_in[m];
    float s[1] = {0.f};
    for (int n = threadIdx.x; n < a.N; n += 1024) {
      float w[1];
      load_param<P, 1, false>(a.weight, n, true, 1.f, w);
      s[0] = __builtin_fmaf(E::get(dy[n]) * w[0], E::get(x[n]) * rstd, s[0]);
    }
    row_sums<1024>(s, slots);
    const float along = s[0] / (float)a.N;
    for (int n = threadIdx.x; n < a.N; n += 1024) {
      float w[1];
      load_param<P, 1, false>(a.weight, n, true, 1.f, w);
      const float c = E::get(x[n]) * rstd, g = E::get(dy[n]) * w[0];
      dx[n] = E::put(__builtin_fmaf(rstd, __builtin_fmaf(-c, along, g), ds != nullptr ? E::get(ds[n]) : 0.f));
    }
  }
}

// The weight's partial sums of such rows: workgroup (x, y) sums 256 columns over
// every gridDim.y-th row.
template <class E>
__global__ void __launch_bounds__(256) rms_columns_kernel(RmsArgs a) {
  typedef typename E::raw raw;
  const int n = blockIdx.x * 256 + threadIdx.x;
  if (n >= a.N) return;
  float dw = 0.f;
  for (int64_t m = blockIdx.y; m < a.M; m += gridDim.y)
    dw = __builtin_fmaf(E::get(static_cast<const raw*>(a.dy)[m * a.lddy + n]), E::get(static_cast<const raw*>(a.x)[m * a.ldx + n]) * a.rstd_in[m], dw);
  a.partial[(size_t)blockIdx.y * a.N + n] = dw;
}

// Adds `count` partial sums [count][N]: 64 columns a workgroup, 16 threads on
// each, each taking every 16th partial in order.
template <class P>
__global__ void __launch_bounds__(1024) rms_params_kernel(const float* partial, int count, int N, void* dweight) {
  typedef typename P::raw raw;
  __shared__ float part[16][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  for (int64_t c0 = (int64_t)blockIdx.x * 64; c0 < N; c0 += (int64_t)gridDim.x * 64) {
    const int64_t c = c0 + lane;
    float s = 0.f;
    if (c < N) {
      constexpr int kAhead = 8;
      for (int g0 = w; g0 < count; g0 += 16 * kAhead) {
        float x[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int g = g0 + 16 * i;
          x[i] = g < count ? partial[(size_t)g * N + c] : 0.f;
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) s += x[i];
      }
    }
    part[w][lane] = s;
    __syncthreads();
    if (w == 0 && c < N) {
      s = 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j) s += part[j][lane];
      static_cast<raw*>(dweight)[c] = P::put(s);
    }
    __syncthreads();  // before the next columns' sums
  }
}

// (odd: not every row and parameter vector starts at a multiple of its size)
Shape rms_shape(const RmsArgs& a, prnnDataType_t type, bool backward, bool eight) {
  const int elems = type == PRNN_DATA_FLOAT ? 4 : 8;
  auto rows = [&](const void* p, int64_t ld, int size) { return p == nullptr || (ld % elems == 0 && (uintptr_t)p % (elems * size) == 0); };
  const int e = 16 / elems;
  bool whole = a.N % elems == 0 && rows(a.x, a.ldx, e) && aligned16(a.weight) && rows(a.y, a.ldy, eight ? 1 : e);
  if (backward)
    whole = whole && rows(a.dy, a.lddy, e) && rows(a.dsum, a.lds, e);
  else
    whole = whole && rows(a.residual, a.ldr, e) && rows(a.sum, a.lds, e);
  return shape_of(a.N, elems, !whole, backward ? 24 : 32);
}

}  // namespace

hipError_t launch_rms_norm(const RmsArgs& a, prnnDataType_t type, prnnDataType_t ptype, bool eight, hipStream_t stream) {
  const Shape s = rms_shape(a, type, false, eight);
  return for_types(type, ptype, [&](auto e, auto p) {
    typedef decltype(e) E;
    typedef decltype(p) P;
    constexpr int V = E::id == PRNN_DATA_FLOAT ? 4 : 8;
    const bool fits = for_shape<V, 32>(s, [&](auto c) {
      typedef decltype(c) K;
      const int64_t sets = (a.M + K::block / K::tpr - 1) / (K::block / K::tpr);
      // Workgroups with a row or two each: those at work then are on neighbouring rows.  With 4 /
      // 16 / 64 a unit: 16384 x 5760 bf16 with a residual, in 8 bits with a scale a row, 133 / 124 / 116
      // us; 8192 x 8192 fp32 with a residual 199 / 199 / 189; 100000 x 513 bf16 45 / 42 / 44; 40000 x 1153
      // fp16 in 8 bits with a scale for 128 columns 52 / 50 / 58 (1152 columns: 41 / 36 / 37).
      const int64_t most = 64ll * a.compute_units;
      const unsigned grid = (unsigned)(sets < most ? sets : most);
      if (eight)
        rms_kernel<E, P, K::v, K::odd, K::tpr, K::nv, K::block, true><<<grid, K::block, 0, stream>>>(a);
      else
        rms_kernel<E, P, K::v, K::odd, K::tpr, K::nv, K::block, false><<<grid, K::block, 0, stream>>>(a);
    });
    if (!fits) {
      if (eight)
        rms_wide_kernel<E, P, true><<<workgroups(a.M), 1024, 0, stream>>>(a);
      else
        rms_wide_kernel<E, P, false><<<workgroups(a.M), 1024, 0, stream>>>(a);
    }
    return hipGetLastError();
  });
}

int rms_norm_backward_grid(const RmsArgs& a, prnnDataType_t type, int compute_units) {
  const Shape s = rms_shape(a, type, true, false);
  if (s.tpr == 0) return (int)(a.M < 64 ? a.M : 64);
  const int R = block_of(s.tpr) / s.tpr;
  const int64_t sets = (a.M + R - 1) / R;
  // (each leaves a row of sums; 1 / 2 / 3 / 4 a unit: 16384 x 5760 bf16 158 / 147 / 160 / 156 us,
  // 100000 x 512 105 / 77 / 80 / 82)
  const int64_t most = (s.tpr > 256 ? 1ll : 2ll) * compute_units;
  return (int)(sets < most ? sets : most);
}

hipError_t launch_rms_norm_backward(const RmsArgs& a, prnnDataType_t type, prnnDataType_t ptype, int grid, hipStream_t stream) {
  const Shape s = rms_shape(a, type, true, false);
  return for_types(type, ptype, [&](auto e, auto p) {
    typedef decltype(e) E;
    typedef decltype(p) P;
    constexpr int V = E::id == PRNN_DATA_FLOAT ? 4 : 8;
    if (grid > 0) {
      const bool fits = for_shape<V, 24>(s, [&](auto c) {
        typedef decltype(c) K;
        constexpr int R = K::block / K::tpr;
        rms_backward_kernel<E, P, K::v, K::odd, K::tpr, K::nv, K::block>
            <<<grid, K::block, (R - 1) * K::v * K::nv * K::tpr * 4, stream>>>(a);
      });
      if (!fits) {
        // the columns first: dx may be written over x or dy
        if (a.partial != nullptr) rms_columns_kernel<E><<<dim3((a.N + 255) / 256, grid), 256, 0, stream>>>(a);
        if (a.y != nullptr) rms_backward_wide_kernel<E, P><<<workgroups(a.M), 1024, 0, stream>>>(a);
      }
    }
    if (a.dweight != nullptr) rms_params_kernel<P><<<workgroups((a.N + 63ll) / 64), 1024, 0, stream>>>(a.partial, grid, a.N, a.dweight);
    return hipGetLastError();
  });
}

}  // namespace prnn
