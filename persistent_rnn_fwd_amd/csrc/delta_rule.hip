// The gated delta rule: one token, and the launches by element type (the chunks
// are in delta_chunk.h).
//
//   Sd = a S, u = beta (v - Sd^T k), S' = Sd + k u^T, o = scale S'^T q = scale (Sd^T q + (q.k) u)
#include "attention_chunk.h"
#include "delta_rule.h"

namespace prnn {
namespace {

using attn::base_of;
using attn::divide;

// One token: grid column tiles of 32 x B H.  Lane l of the workgroup owns W = 4
// columns, 4 (l % 8) .. + 3 of the tile, and rows l / 8 + 32 j, or one column, l %
// 32, and rows l / 32 + 8 j.  The rows stay in registers (NR a thread) between
// the sums over them, S^T k, S^T q and q.k in one go, and their update, so that
// the state is read once and written once, which is all this call costs (64 tokens of
// 32 bf16 heads of 128: 58 us, 4.7 TB/s; one token of 14 fp16 heads: 5.6 us).  ODD: rows
// of the state start at any element, and the last lane's columns are moved back
// to end with the row; of those that another lane has too, it stores none.
template <class E, int W, int NR, bool ODD>
__global__ void __launch_bounds__(256) delta_step_kernel(DeltaStepArgs a) {
  typedef typename E::raw raw;
  typedef float vec __attribute__((ext_vector_type(W)));
  typedef float any __attribute__((ext_vector_type(W), aligned(ODD ? 4 : 4 * W)));
  constexpr int kCols = 32 / W, kRows = 256 / kCols;
  __shared__ float part[3][4][33];  // sums of each wave
  const int bh = (int)divide(blockIdx.x, a.tiles, a.by_tiles), col0 = ((int)blockIdx.x - bh * a.tiles) * 32;
  const int b = (int)divide(bh, a.H, a.by_heads), h = bh - b * a.H;
  const int rg = threadIdx.x / kCols;
  int cl = W * (threadIdx.x % kCols);
  const bool live = col0 + cl < a.Dv;
  const int again = ODD && live ? max(0, col0 + cl + W - a.Dv) : 0;  // columns of the lane before
  cl -= again;
  const int c = col0 + cl;
  auto at = [&](const AttnOperand& x) { return (int64_t)b * x.batch + (int64_t)divide(h, x.group, x.inverse) * x.head; };
  const raw* q = static_cast<const raw*>(a.q.p) + at(a.q);
  const raw* k = static_cast<const raw*>(a.k.p) + at(a.k);
  const raw* v = static_cast<const raw*>(a.v.p) + at(a.v);
  const size_t state = (size_t)bh * a.Dk * a.Dv + c;
  vec S[NR];
  float kk[NR], qq[NR];
#pragma unroll
  for (int j = 0; j < NR; ++j) {
    const int r = rg + j * kRows;
    const bool in = live && r < a.Dk;
    S[j] = in ? *reinterpret_cast<const any*>(a.s_in + state + (size_t)r * a.Dv) : vec(0.f);
    kk[j] = r < a.Dk ? E::get(k[r]) : 0.f;
    qq[j] = r < a.Dk ? E::get(q[r]) : 0.f;
  }
  const float d = a.g.p != nullptr ? expf(static_cast<const float*>(a.g.p)[at(a.g)]) : 1.f;
  const float beta = static_cast<const float*>(a.beta.p)[at(a.beta)];
  float vv[W], sk[W], sq[W], qk = 0.f;
#pragma unroll
  for (int e = 0; e < W; ++e) {
    vv[e] = live ? E::get(v[c + e]) : 0.f;
    sk[e] = sq[e] = 0.f;
  }
#pragma unroll
  for (int j = 0; j < NR; ++j) {
    if (rg + j * kRows < a.Dk) {
#pragma unroll
      for (int e = 0; e < W; ++e) {
        S[j][e] *= d;
        sk[e] = __builtin_fmaf(kk[j], S[j][e], sk[e]);
        sq[e] = __builtin_fmaf(qq[j], S[j][e], sq[e]);
      }
      qk = __builtin_fmaf(qq[j], kk[j], qk);
    }
  }
  // sums over the lanes of a wave that have a column, then over the waves
#pragma unroll
  for (int m = kCols; m < 64; m *= 2) {
#pragma unroll
    for (int e = 0; e < W; ++e) {
      sk[e] += __shfl_xor(sk[e], m);
      sq[e] += __shfl_xor(sq[e], m);
    }
    qk += __shfl_xor(qk, m);
  }
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  if (lane < kCols) {
#pragma unroll
    for (int e = 0; e < W; ++e)
      if (!ODD || e >= again) {
        part[0][wave][cl + e] = sk[e];
        part[1][wave][cl + e] = sq[e];
      }
    if (lane == 0) part[2][wave][0] = qk;
  }
  __syncthreads();
  float u[W];
  qk = (part[2][0][0] + part[2][1][0]) + (part[2][2][0] + part[2][3][0]);
#pragma unroll
  for (int e = 0; e < W; ++e) {
    const float (&p)[4][33] = part[0];
    const int x = cl + e;
    u[e] = live && (!ODD || e >= again) ? beta * (vv[e] - ((p[0][x] + p[1][x]) + (p[2][x] + p[3][x]))) : 0.f;
  }
#pragma unroll
  for (int j = 0; j < NR; ++j) {
    const int r = rg + j * kRows;
    if (live && r < a.Dk) {
#pragma unroll
      for (int e = 0; e < W; ++e) S[j][e] = __builtin_fmaf(kk[j], u[e], S[j][e]);
      float* const to = a.s_out + state + (size_t)r * a.Dv;
      if constexpr (!ODD) {
        __builtin_nontemporal_store(S[j], reinterpret_cast<vec*>(to));
      } else if (again == 0) {
        *reinterpret_cast<any*>(to) = S[j];
      } else {
#pragma unroll
        for (int e = 1; e < W; ++e)
          if (e >= again) to[e] = S[j][e];
      }
    }
  }
  if (rg == 0 && live) {
    raw* const o = static_cast<raw*>(const_cast<void*>(a.o.p)) + at(a.o);
#pragma unroll
    for (int e = 0; e < W; ++e) {
      const int x = cl + e;
      if (ODD && e < again) continue;
      const float (&p)[4][33] = part[1];
      o[c + e] = E::put(a.scale * __builtin_fmaf(qk, u[e], (p[0][x] + p[1][x]) + (p[2][x] + p[3][x])));
    }
  }
}

template <class E>
void step_of(const DeltaStepArgs& a, bool whole, hipStream_t stream) {
  const dim3 grid((unsigned)a.tiles * a.B * a.H);
#define PRNN_STEP(W, NR, ODD) delta_step_kernel<E, W, NR, ODD><<<grid, 256, 0, stream>>>(a)
  if (a.Dv < 4) {
    PRNN_STEP(1, 32, true);
  } else if (a.Dk <= 64) {
    whole ? PRNN_STEP(4, 2, false) : PRNN_STEP(4, 2, true);
  } else if (a.Dk <= 128) {
    whole ? PRNN_STEP(4, 4, false) : PRNN_STEP(4, 4, true);
  } else {
    whole ? PRNN_STEP(4, 8, false) : PRNN_STEP(4, 8, true);
  }
#undef PRNN_STEP
}

}  // namespace

hipError_t launch_delta(const DeltaArgs& a, prnnDataType_t type, bool backward, hipStream_t stream) {
  switch (type) {
    case PRNN_DATA_FLOAT: return launch_delta_f32(a, backward, stream);
    case PRNN_DATA_HALF: return launch_delta_f16(a, backward, stream);
    default: return launch_delta_bf16(a, backward, stream);
  }
}

hipError_t launch_delta_step(const DeltaStepArgs& args, prnnDataType_t type, hipStream_t stream) {
  DeltaStepArgs a = args;
  a.by_tiles = inverse_of(a.tiles);
  a.by_heads = inverse_of(a.H);
  for (AttnOperand* x : {&a.q, &a.k, &a.v, &a.o, &a.g, &a.beta}) x->inverse = inverse_of(x->group);
  const bool whole = a.Dv % 4 == 0 && (uintptr_t)a.s_in % 16 == 0 && (uintptr_t)a.s_out % 16 == 0;
  switch (type) {
    case PRNN_DATA_FLOAT: step_of<F32>(a, whole, stream); break;
    case PRNN_DATA_HALF: step_of<F16>(a, whole, stream); break;
    default: step_of<BF16>(a, whole, stream); break;
  }
  return hipGetLastError();
}

}  // namespace prnn
