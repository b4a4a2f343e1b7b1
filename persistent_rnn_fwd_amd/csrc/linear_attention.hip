// Linear attention with a decay for each head.
//
//   S[t] = d S[t-1] + k[t] v[t]^T,  o[t] = scale S[t]^T q[t],  d = exp(log_decay)
//
// attention_token_kernel is the recurrence itself: one wave owns 16 columns of
// a head's state in registers and walks the tokens, so every column costs one
// pass over q and k.
#include "sequence.h"

namespace prnn {
namespace {

// First row and number of tokens of sequence b (see prnnAttention_t).
struct Span {
  int64_t first;
  int len;
};
template <class A>
__device__ __forceinline__ Span span_of(const A& a, int b) {
  Span s = {0, a.T};
  if (a.offsets != nullptr) {
    const int64_t lo = a.offsets[b], hi = a.offsets[b + 1];
    s.first = lo < 0 ? 0 : (lo > a.rows ? a.rows : lo);
    int64_t end = hi < s.first ? s.first : (hi > a.rows ? a.rows : hi);
    if (end - s.first > a.T) end = s.first + a.T;
    s.len = (int)(end - s.first);
  } else if (a.lengths != nullptr) {
    const int n = a.lengths[b];
    s.len = n < 0 ? 0 : (n > a.T ? a.T : n);
  }
  return s;
}

// Element offset of row `first` of sequence b, head h, of an operand.
template <class A>
__device__ __forceinline__ int64_t base_of(const AttnOperand& x, const A& a, const Span& s, int b, int h) {
  return (a.offsets != nullptr ? s.first * x.token : (int64_t)b * x.batch) + (int64_t)(h / x.group) * x.head;
}

// exp(log_decay n) to fp32's precision: the product's rounding error re-enters
// to first order.  n = 0 gives 1 and -infinity 0 for every other n.
__device__ __forceinline__ float decay_power(float log_decay, int n) {
  if (n == 0) return 1.f;
  const float x = log_decay * (float)n;
  if (x < -104.f) return 0.f;  // below the smallest fp32
  const float low = __builtin_fmaf(log_decay, (float)n, -x);
  return x > 89.f ? expf(x) : __builtin_fmaf(expf(x), low, expf(x));
}

constexpr int kTokenCols = 16;

// grid: (column tiles x B H, jobs), one wave each.  Lane l owns rows l / 4 +
// 16 j and columns 4 (l % 4) .. + 3 of the tile.
template <class E, int NR>
__global__ void __launch_bounds__(64) attention_token_kernel(AttnArgs a) {
  typedef typename E::raw raw;
  const AttnJob& job = a.job[blockIdx.y];
  const int col0 = (int)(blockIdx.x % a.tiles) * kTokenCols;
  if (col0 >= job.Dv) return;
  const int bh = blockIdx.x / a.tiles, b = bh / a.H, h = bh % a.H;
  const int lane = threadIdx.x, rg = lane >> 2, c = col0 + 4 * (lane & 3);
  const Span s = span_of(a, b);
  const raw* q = static_cast<const raw*>(job.q.p) + base_of(job.q, a, s, b, h);
  const raw* k = static_cast<const raw*>(job.k.p) + base_of(job.k, a, s, b, h);
  const raw* v = static_cast<const raw*>(job.v.p) + base_of(job.v, a, s, b, h);
  const int64_t o = base_of(job.o, a, s, b, h);
  const size_t state = ((size_t)b * a.H + h) * job.Dk * job.Dv;
  const float log_decay = a.log_decay[h];
  const float d = decay_power(log_decay, 1);

  float S[NR][4];
#pragma unroll
  for (int j = 0; j < NR; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int r = rg + 16 * j;
      S[j][e] = job.s_in != nullptr && r < job.Dk && c + e < job.Dv
                    ? job.s_in[state + (size_t)r * job.s_row + (size_t)(c + e) * job.s_col]
                    : 0.f;
    }
  const float before = job.reverse ? 1.f : d;  // decay of the state before a token takes it
  const float after = job.reverse ? d : 1.f;
  for (int i = 0; i < s.len; ++i) {
    const int64_t t = job.reverse ? s.len - 1 - i : i;
    float kv[NR], qv[NR], vv[4], acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < NR; ++j) {
      const int r = rg + 16 * j;
      kv[j] = r < job.Dk ? E::get(k[t * job.k.token + r]) * job.kscale : 0.f;
      qv[j] = r < job.Dk ? E::get(q[t * job.q.token + r]) : 0.f;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) vv[e] = c + e < job.Dv ? E::get(v[t * job.v.token + c + e]) : 0.f;
#pragma unroll
    for (int j = 0; j < NR; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (rg + 16 * j < job.Dk) {
          S[j][e] = __builtin_fmaf(kv[j], vv[e], S[j][e] * before);
          acc[e] = __builtin_fmaf(qv[j], S[j][e], acc[e]);
          S[j][e] *= after;
        }
      }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
#pragma unroll
      for (int m = 4; m < 64; m *= 2) acc[e] += __shfl_xor(acc[e], m);
      if (rg == 0 && c + e < job.Dv) {
        const int64_t at = o + t * job.o.token + c + e;
        if (job.o_f32)
          static_cast<float*>(const_cast<void*>(job.o.p))[at] = acc[e] * job.oscale;
        else
          static_cast<raw*>(const_cast<void*>(job.o.p))[at] = E::put(acc[e] * job.oscale);
      }
    }
  }
  if (a.lengths != nullptr && rg == 0) {
    for (int64_t t = s.len; t < a.T; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (c + e < job.Dv) {
          const int64_t at = o + t * job.o.token + c + e;
          if (job.o_f32)
            static_cast<float*>(const_cast<void*>(job.o.p))[at] = 0.f;
          else
            static_cast<raw*>(const_cast<void*>(job.o.p))[at] = E::put(0.f);
        }
  }
  if (job.s_out != nullptr) {
#pragma unroll
    for (int j = 0; j < NR; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = rg + 16 * j;
        if (r < job.Dk && c + e < job.Dv) job.s_out[state + (size_t)r * job.s_row + (size_t)(c + e) * job.s_col] = S[j][e];
      }
  }
}

// grid: `blocks` workgroups for each sequence, one thread per element of dst at a time.
template <class E>
__global__ void __launch_bounds__(256) attention_reduce_kernel(AttnReduceArgs a) {
  const int64_t n = (int64_t)a.T * a.groups * a.D;
  const int b = blockIdx.x / a.blocks;
  const Span s = span_of(a, b);
  typedef typename E::raw raw;
  raw* dst = static_cast<raw*>(const_cast<void*>(a.dst.p));
  const int H = a.groups * a.per_group;
  for (int64_t i = (blockIdx.x % a.blocks) * 256ll + threadIdx.x; i < n; i += a.blocks * 256ll) {
    const int d = (int)(i % a.D);
    const int g = (int)(i / a.D % a.groups);
    const int64_t t = i / a.D / a.groups;
    if (t >= s.len && a.lengths == nullptr) break;
    // src is dense: [T][B][H][D], or [rows][H][D] packed
    const int64_t row = a.offsets != nullptr ? s.first + t : t * a.B + b;
    float sum = 0.f;
    if (t < s.len)
      for (int j = 0; j < a.per_group; ++j) sum += a.src[(row * H + g * a.per_group + j) * a.D + d];
    const int64_t base = a.offsets != nullptr ? s.first * a.dst.token : (int64_t)b * a.dst.batch;
    dst[base + t * a.dst.token + (int64_t)g * a.dst.head + d] = E::put(sum);
  }
}

// One token: grid column tiles of 32 x B H.  With VEC (Dv % 4 == 0 and
// 16-byte states) lane l of the workgroup owns columns 4 (l % 8) .. + 3 of the
// tile and rows l / 8 + 32 j, else column l % 32 and rows l / 32 + 8 j.  The
// state is read once and written once, which is all this call costs.
template <class E, bool VEC>
__global__ void __launch_bounds__(256) attention_step_kernel(AttnStepArgs a) {
  typedef typename E::raw raw;
  typedef float vec __attribute__((ext_vector_type(VEC ? 4 : 1)));
  constexpr int W = VEC ? 4 : 1, kCols = 32 / W, kRows = 256 / kCols, U = 4;
  __shared__ float part[kRows][33];
  const int bh = blockIdx.x / a.tiles, col0 = (int)(blockIdx.x % a.tiles) * 32, b = bh / a.H, h = bh % a.H;
  const int rg = threadIdx.x / kCols, cl = W * (threadIdx.x % kCols), c = col0 + cl;
  const bool live = c < a.Dv;
  const raw* q = static_cast<const raw*>(a.q.p) + (int64_t)b * a.q.batch + (int64_t)(h / a.q.group) * a.q.head;
  const raw* k = static_cast<const raw*>(a.k.p) + (int64_t)b * a.k.batch + (int64_t)(h / a.k.group) * a.k.head;
  const raw* v = static_cast<const raw*>(a.v.p) + (int64_t)b * a.v.batch + (int64_t)(h / a.v.group) * a.v.head;
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
      S[u] = in ? *reinterpret_cast<const vec*>(a.s_in + state + (size_t)r * a.Dv) : vec(0.f);
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
        *reinterpret_cast<vec*>(a.s_out + state + (size_t)r * a.Dv) = S[u];
      }
    }
  }
#pragma unroll
  for (int e = 0; e < W; ++e) part[rg][cl + e] = acc[e];
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

}  // namespace

hipError_t launch_attention(const AttnArgs& args, prnnDataType_t type, hipStream_t stream) {
  AttnArgs a = args;
  int dk = 0, dv = 0;
  for (int i = 0; i < a.jobs; ++i) {
    dk = a.job[i].Dk > dk ? a.job[i].Dk : dk;
    dv = a.job[i].Dv > dv ? a.job[i].Dv : dv;
  }
  a.tiles = (dv + kTokenCols - 1) / kTokenCols;
  const dim3 grid((unsigned)a.tiles * a.B * a.H, a.jobs);
  return for_type(type, [&](auto e) {
    typedef decltype(e) E;
    if (dk <= 64)
      attention_token_kernel<E, 4><<<grid, 64, 0, stream>>>(a);
    else if (dk <= 128)
      attention_token_kernel<E, 8><<<grid, 64, 0, stream>>>(a);
    else
      attention_token_kernel<E, 16><<<grid, 64, 0, stream>>>(a);
    return hipGetLastError();
  });
}

hipError_t launch_attention_reduce(const AttnReduceArgs& args, prnnDataType_t type, hipStream_t stream) {
  AttnReduceArgs a = args;
  const int64_t blocks = ((int64_t)a.T * a.groups * a.D + 255) / 256, most = a.B < 2048 ? 2048 / a.B : 1;
  a.blocks = (int)(blocks < most ? blocks : most);
  const dim3 grid((unsigned)a.blocks * a.B);
  return for_type(type, [&](auto e) {
    attention_reduce_kernel<decltype(e)><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
  });
}

hipError_t launch_attention_step(const AttnStepArgs& args, prnnDataType_t type, hipStream_t stream) {
  AttnStepArgs a = args;
  a.tiles = (a.Dv + 31) / 32;
  const dim3 grid((unsigned)a.tiles * a.B * a.H);
  const bool vec = a.Dv % 4 == 0 && ((uintptr_t)a.s_in | (uintptr_t)a.s_out) % 16 == 0;
  return for_type(type, [&](auto e) {
    typedef decltype(e) E;
    if (vec)
      attention_step_kernel<E, true><<<grid, 256, 0, stream>>>(a);
    else
      attention_step_kernel<E, false><<<grid, 256, 0, stream>>>(a);
    return hipGetLastError();
  });
}

}  // namespace prnn
