// Linear attention with a decay for each head: the sum over shared heads, and one
// token (the chunks are in attention_chunk.h, the plan in attention_plan.cpp).
//
//   S[t] = d S[t-1] + k[t] v[t]^T,  o[t] = scale S[t]^T q[t],  d = exp(log_decay)
#include <algorithm>

#include "attention_chunk.h"

namespace prnn {
namespace {

using attn::base_of;
using attn::decay_power;
using attn::divide;
using attn::Span;
using attn::span_of;

// The heads' gradients of k and of v, summed over each group in head order.
// grid: `blocks` workgroups for each sequence, 2; a thread 4 columns of one row
// and group at a time (VEC: D % 4 == 0), else one.  Bound by memory and, at this
// size, by its launch: 1024 rows of 18 fp32 heads of 64 on 9, twice, 14 MB, 5 us.
template <class E, bool VEC>
__global__ void __launch_bounds__(256) attention_reduce_kernel(AttnReduceArgs a) {
  typedef typename E::raw raw;
  constexpr int W = VEC ? 4 : 1;
  typedef float vec __attribute__((ext_vector_type(W)));
  typedef raw out __attribute__((ext_vector_type(W), aligned(sizeof(raw))));
  const auto& x = a.grad[blockIdx.y];
  const uint32_t per_row = (uint32_t)(a.groups * (x.D / W)), per_group = (uint32_t)(x.D / W);
  const int b = blockIdx.x / a.blocks;
  const Span s = span_of(a, b);
  raw* const dst = static_cast<raw*>(const_cast<void*>(x.dst.p)) +
                   (a.offsets != nullptr ? s.first * x.dst.token : (int64_t)b * x.dst.batch);
  const float* const from = static_cast<const float*>(x.src.p) +
                            (a.offsets != nullptr ? s.first * x.src.token : (int64_t)b * x.src.batch);
  const int rows = a.lengths != nullptr ? a.T : s.len;  // (padding: zeros)
  const uint32_t step = (uint32_t)a.blocks * 256u;
  uint32_t i = (blockIdx.x % a.blocks) * 256u + threadIdx.x;
  uint32_t t = i / per_row, at = i - t * per_row;
  const uint32_t dt = step / per_row, dat = step - dt * per_row;
  for (; t < (uint32_t)rows; t += dt, at += dat) {
    if (at >= per_row) {
      at -= per_row;
      if (++t >= (uint32_t)rows) break;
    }
    const uint32_t g = at / per_group;
    const int d = (int)(at - g * per_group) * W;
    vec sum = vec(0.f);
    if ((int)t < s.len) {
      const float* src = from + (int64_t)t * x.src.token + (int64_t)g * a.per_group * x.src.head + d;
      for (int j = 0; j < a.per_group; ++j, src += x.src.head) sum += *reinterpret_cast<const vec*>(src);
    }
    out y;
#pragma unroll
    for (int e = 0; e < W; ++e) y[e] = E::put(sum[e]);
    *reinterpret_cast<out*>(dst + (int64_t)t * x.dst.token + (int64_t)g * x.dst.head + d) = y;
  }
}

// Copies a state, 4 elements a thread at a time.  Bound by memory (134 MB in 39 us).
__global__ void __launch_bounds__(256) attention_keep_kernel(const float* from, float* to, int64_t n) {
  constexpr int U = 4;
  for (int64_t i0 = (int64_t)blockIdx.x * (256 * U) + threadIdx.x; i0 < n; i0 += (int64_t)gridDim.x * (256 * U)) {
    float x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) x[u] = i0 + u * 256 < n ? from[i0 + u * 256] : 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u * 256 < n) to[i0 + u * 256] = x[u];
  }
}

// One token: grid column tiles of 32 x B H.  Lane l of the workgroup owns W = 4
// columns, 4 (l % 8) .. + 3 of the tile, and rows l / 8 + 32 j, or one column, l
// % 32, and rows l / 32 + 8 j.  The state is read once and written once, which is
// all this call costs.  ODD: rows of the state start at any element, and the last
// lane's columns are moved back to end with the row; of those that another lane
// has too, it stores none (they may be written already where the state is
// updated in place).
//
// Measured, stores past the caches (and plain ones): 64 sequences of 32 heads of 128
// x 128, 270 MB, into another state 43 us over and over (46), 53 with cold ones
// (57; 5.0 TB/s); in place, a replayed loop of steps, 45.3 (44.7), 8 such layers 58.6
// each (58.8), 16 sequences 12.5 (11.7), 4 sequences or 14 heads of one the same.
template <class E, int W, bool ODD>
__global__ void __launch_bounds__(256) attention_step_kernel(AttnStepArgs a) {
  typedef typename E::raw raw;
  typedef float vec __attribute__((ext_vector_type(W)));
  typedef float any __attribute__((ext_vector_type(W), aligned(ODD ? 4 : 4 * W)));
  constexpr int kCols = 32 / W, kRows = 256 / kCols, U = 4;
  __shared__ float part[kRows][33];
  const int bh = (int)divide(blockIdx.x, a.tiles, a.by_tiles), col0 = ((int)blockIdx.x - bh * a.tiles) * 32;
  const int b = (int)divide(bh, a.H, a.by_heads), h = bh - b * a.H;
  const int rg = threadIdx.x / kCols;
  int cl = W * (threadIdx.x % kCols);
  const bool live = col0 + cl < a.Dv;
  const int again = ODD && live ? max(0, col0 + cl + W - a.Dv) : 0;  // columns of the lane before
  cl -= again;
  const int c = col0 + cl;
  const raw* q = static_cast<const raw*>(a.q.p) + (int64_t)b * a.q.batch + (int64_t)divide(h, a.q.group, a.q.inverse) * a.q.head;
  const raw* k = static_cast<const raw*>(a.k.p) + (int64_t)b * a.k.batch + (int64_t)divide(h, a.k.group, a.k.inverse) * a.k.head;
  const raw* v = static_cast<const raw*>(a.v.p) + (int64_t)b * a.v.batch + (int64_t)divide(h, a.v.group, a.v.inverse) * a.v.head;
  const size_t state = (size_t)bh * a.Dk * a.Dv + c;
  const float d = decay_power(a.log_decay[h], 1);
  float vv[W], acc[W];
#pragma unroll
  for (int e = 0; e < W; ++e) {
    vv[e] = live ? E::get(v[c + e]) : 0.f;
    acc[e] = 0.f;
  }
  for (int r0 = rg; r0 < a.Dk; r0 += U * kRows) {
    vec S[U];
    float kk[U], qq[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * kRows;
      const bool in = live && r < a.Dk;
      S[u] = in ? *reinterpret_cast<const any*>(a.s_in + state + (size_t)r * a.Dv) : vec(0.f);
      kk[u] = in ? E::get(k[r]) : 0.f;
      qq[u] = in ? E::get(q[r]) : 0.f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = r0 + u * kRows;
      if (live && r < a.Dk) {
#pragma unroll
        for (int e = 0; e < W; ++e) {
          S[u][e] = __builtin_fmaf(kk[u], vv[e], S[u][e] * d);
          acc[e] = __builtin_fmaf(qq[u], S[u][e], acc[e]);
        }
        float* const to = a.s_out + state + (size_t)r * a.Dv;
        if constexpr (!ODD) {
          __builtin_nontemporal_store(S[u], reinterpret_cast<vec*>(to));
        } else if (again == 0) {
          *reinterpret_cast<any*>(to) = S[u];
        } else {
#pragma unroll
          for (int e = 1; e < W; ++e)
            if (e >= again) to[e] = S[u][e];
        }
      }
    }
  }
#pragma unroll
  for (int e = 0; e < W; ++e)
    if (!ODD || e >= again) part[rg][cl + e] = acc[e];
  __syncthreads();
  // 32 columns x 8 threads, each summing every eighth row group in order
  const int col = threadIdx.x & 31, t8 = threadIdx.x >> 5;
  float sum = 0.f;
#pragma unroll
  for (int r = 0; r < kRows / 8; ++r) sum += part[t8 + 8 * r][col];
  __syncthreads();
  part[t8][col] = sum;
  __syncthreads();
  if (threadIdx.x < 32 && col0 + (int)threadIdx.x < a.Dv) {
    float o = 0.f;
#pragma unroll
    for (int r = 0; r < 8; ++r) o += part[r][threadIdx.x];
    static_cast<raw*>(const_cast<void*>(a.o.p))[(int64_t)b * a.o.batch + (int64_t)h * a.o.head + col0 + threadIdx.x] =
        E::put(o * a.scale);
  }
}

template <class F>
hipError_t for_type(prnnDataType_t type, F f) {
  switch (type) {
    case PRNN_DATA_FLOAT: return f(F32());
    case PRNN_DATA_HALF: return f(F16());
    default: return f(BF16());
  }
}

bool aligned16(const void* p) { return (uintptr_t)p % 16 == 0; }

}  // namespace

hipError_t launch_attention(const AttnArgs& a, prnnDataType_t type, hipStream_t stream) {
  if (a.keep > 0) {
    const int64_t blocks = (a.keep + 1023) / 1024;
    attention_keep_kernel<<<(unsigned)(blocks < 4096 ? blocks : 4096), 256, 0, stream>>>(a.keep_from, a.keep_to, a.keep);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  switch (type) {
    case PRNN_DATA_FLOAT: return launch_attention_f32(a, stream);
    case PRNN_DATA_HALF: return launch_attention_f16(a, stream);
    default: return launch_attention_bf16(a, stream);
  }
}

hipError_t launch_attention_reduce(const AttnReduceArgs& args, prnnDataType_t type, hipStream_t stream) {
  AttnReduceArgs a = args;
  const bool vec = a.grad[0].D % 4 == 0 && a.grad[1].D % 4 == 0 && aligned16(a.grad[0].src.p) && aligned16(a.grad[1].src.p);
  const int64_t blocks = ((int64_t)a.T * a.groups * std::max(a.grad[0].D, a.grad[1].D) / (vec ? 4 : 1) + 255) / 256,
                most = a.B < 2048 ? 2048 / a.B : 1;
  a.blocks = (int)(blocks < most ? blocks : most);
  const dim3 grid((unsigned)a.blocks * a.B, 2);
  return for_type(type, [&](auto e) {
    typedef decltype(e) E;
    if (vec)
      attention_reduce_kernel<E, true><<<grid, 256, 0, stream>>>(a);
    else
      attention_reduce_kernel<E, false><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
  });
}

hipError_t launch_attention_step(const AttnStepArgs& args, prnnDataType_t type, hipStream_t stream) {
  AttnStepArgs a = args;
  a.by_tiles = inverse_of(a.tiles);
  a.by_heads = inverse_of(a.H);
  for (AttnOperand* x : {&a.q, &a.k, &a.v}) x->inverse = inverse_of(x->group);
  const dim3 grid((unsigned)a.tiles * a.B * a.H);
  const bool whole = a.Dv % 4 == 0 && aligned16(a.s_in) && aligned16(a.s_out);
  return for_type(type, [&](auto e) {
    typedef decltype(e) E;
    if (whole)
      attention_step_kernel<E, 4, false><<<grid, 256, 0, stream>>>(a);
    else if (a.Dv >= 4)
      attention_step_kernel<E, 4, true><<<grid, 256, 0, stream>>>(a);
    else
      attention_step_kernel<E, 1, true><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
  });
}

}  // namespace prnn
