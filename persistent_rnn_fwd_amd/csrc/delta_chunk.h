// The gated delta rule in chunks of 32 tokens on the matrix cores.
//
//   S[t] = a S[t-1] + beta k (v - a S[t-1]^T k)^T,  o[t] = scale S[t]^T q,  a = exp(g[t])
//
// With i, j tokens of one chunk, S the state it starts from, G the sums of g
// inside the chunk, d_ij = exp(G_i - G_j), up_i = exp(G_i), down_j = d_Cj
// (C the chunk's last token):
//
//   A'_ij = d_ij (k_i.k_j) beta_j  (j < i),   T' = (I + A')^-1
//   x = T' (v - up o (K S)),   P'_ij = scale d_ij (q_i.k_j) beta_j  (j <= i)
//   o = scale up o (Q S) + P' x,   S <- up_C S + K^T (down beta o x)
//
// x_i is what token i's key finds missing of its value; beta x enters the state.
// Nothing is divided by beta, which may be 0.  Backward, with R the gradient
// of the state behind the chunk and dO that of o:
//
//   w = T'^T (P'^T dO + down beta o (K R))                        (= dv)
//   R <- up_C R + Q^T (scale up o dO) - K^T (up o w)
//   Y_ij = scale d_ij dO_i.x_j  (j <= i),   Z_ij = d_ij w_i.x_j  (j < i)
//   dq = scale up o (dO S^T) + (Y beta) K,   row = -up o (w S^T) - (Z beta) K
//   col = down o (x R^T) + Y^T Q - Z^T K,    dk = row + beta o col
//   dbeta_i = k_i.col_i,   dG_i = q_i.dq_i + k_i.row_i - beta_i dbeta_i
//   dg_t = up_C <R, S> + sum_j beta_j k_j.(down o x R^T)_j + sum_{i >= t} dG_i   (0 where exp(g_t) is)
//
// Launches.  T', P' and the factors depend on no state: a first launch, a wave
// for each chunk and head, leaves them in the workspace (delta_prepare_kernel).
// The walk along the sequence (delta_forward_kernel) has a workgroup of 4 waves
// for 64 columns of one head's state; each wave keeps its DKP x 16 of the state
// in registers.  The accumulators' layout (lane l: rows 4 (l / 16) + r, column l %
// 16) is that of an operand whose rows are dealt to suit, so K S, x, o^T and the
// state's update follow each other without a shuffle: two tiles of 16 tokens are
// the operand whose element e of lane group g is token 16 (e / 4) + 4 g + e % 4, and
// T' and P' are stored with their columns in that order.  Long sequences of few heads
// are split (plan_delta): a walk from zeros, and one from the identity without
// values, leave what each segment adds to the state and makes of it,
// delta_scan_kernel joins them, and the walk starts each segment from its own
// state.  The backward pass walks forward for x and the states that groups of chunks
// (group_chunks) start from, kept in the workspace, backwards for w and the gradients
// of the states they end with (delta_reverse_kernel; split the same way, with the
// moves transposed), and a last launch, a workgroup for each group and head, takes
// the gradients from these (delta_grad_kernel).
//
// What bounds it.  The walk: a chunk's chain of products (96 for each wave, bf16 and
// 128 rows, 1540 cycles), splitting of the state and of x (the most of 1700 cycles of vector
// instructions) and LDS between them, 5600 cycles alone on a unit, of which a second
// workgroup hides nearly half.  32768 tokens of 32 bf16 heads of 128: 1059 to 1135 us, on one card or
// another (traced one by one, at lower clocks: the first launch 166, 4.8 TB/s, ends and moves 530, the scan
// 27, the walk 490).  The gradients: what
// goes through memory, 8 x 2048 tokens of 16 bf16 heads of 128 782 to 824 us, of them the first launch
// 60, the walks 155 and 205, the gradients' own launch 390 (1 GB read, one workgroup on a
// unit).  Small calls: launches and first loads.
//
// Precision.  As linear attention's: operands in bf16 parts, exact (one for bf16,
// two for fp16, three for fp32), what is fp32 between the products in three, sums
// in fp32.  G is summed in fp64: decays of neighbouring tokens are then right
// however far the chunk has decayed.
//
// Infinities and NaN.  A masked 0 times a later token's infinity is NaN, so a
// wave whose outputs are not finite takes its columns again by the recurrence,
// token by token (delta_tokens).  (Gradients: a value that is not finite may make
// every gradient of its sequence and head NaN.)
#pragma once

#include <type_traits>

#include "attention_chunk.h"
#include "delta_rule.h"

namespace prnn {
namespace delta {

using namespace attn;

// Element offset of token 0 of sequence b, head h, of an operand (all the same in every lane).
__device__ __forceinline__ int64_t base_of(const AttnOperand& x, const DeltaArgs& a, const Span& s, int b, int h) {
  const int head = __builtin_amdgcn_readfirstlane((int)divide((uint32_t)h, (uint32_t)x.group, x.inverse));
  return (a.offsets != nullptr ? s.first * x.token : (int64_t)b * x.batch) + (int64_t)head * x.head;
}

constexpr int C = kDeltaChunk;

// Row and position of an element of a 32 x 32 matrix of bf16: rows of 64 bytes,
// their 16-byte units swizzled, columns dealt as the operands' (position()).
__host__ __device__ constexpr int delta_at(int row, int pos) {
  return row * 64 + (((pos >> 3) ^ ((row >> 2) & 3)) << 4) + 2 * (pos & 7);
}
__host__ __device__ constexpr int position(int column) { return 8 * ((column & 15) >> 2) + 4 * (column >> 4) + (column & 3); }
constexpr int kPart = 2048;  // bytes of a part of such a matrix

// 16 rows from 16 t on as operands (row 16 t + l, positions 8 g .. + 7).
template <int P>
__device__ __forceinline__ void read_matrix(b16x8 (&x)[P], const char* m, int t, int lane) {
  const int g = lane >> 4, l = lane & 15;
#pragma unroll
  for (int p = 0; p < P; ++p) x[p] = read_row(m, p * kPart + (16 * t + l) * 64 + ((g ^ (l >> 2)) << 4));
}
// ... and of the transpose: row 16 t + l is column 16 t + l, its elements the rows dealt as an operand's.
template <int P>
__device__ __forceinline__ void read_transposed(b16x8 (&x)[P], const char* m, int t, int lane) {
  const int g = lane >> 4, l = lane & 15;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    u32x2 half[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      half[h] = read_columns(m, p * kPart + (16 * h + 4 * g + (l >> 2)) * 64 + (((l & 3) ^ g) << 4) + 8 * t);
    const uint32_t words[4] = {half[0][0], half[0][1], half[1][0], half[1][1]};
    x[p] = operand(words);
  }
}

// 8 values of a row, zeros where the row or a column does not exist, on their
// way to an operand.  row: its byte offset, or kOutside.
template <class E, bool VEC>
struct RowPart {
  typedef typename E::raw raw;
  static constexpr int IN = Parts<E>::kIn;
  uint32_t w[IN == 3 ? 8 : 4];
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t row, int col, int cols) {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < (IN == 3 ? 2 : 1); ++i) {
        const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(r, col + 4 * i < cols ? row + (uint32_t)((col + 4 * i) * (int)sizeof(raw)) : kOutside, 0, kPlain);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[4 * i + e] = v[e];
      }
    } else {
      uint32_t e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t at = col + i < cols ? row + (uint32_t)((col + i) * (int)sizeof(raw)) : kOutside;
        e[i] = sizeof(raw) == 4 ? __builtin_amdgcn_raw_buffer_load_b32(r, at, 0, kPlain)
                                : (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(r, at, 0, kPlain);
      }
#pragma unroll
      for (int i = 0; i < (IN == 3 ? 8 : 4); ++i) w[i] = IN == 3 ? e[i % 8] : e[2 * i % 8] | e[(2 * i + 1) % 8] << 16;
    }
  }
  __device__ __forceinline__ void take(b16x8 (&f)[IN]) const {
    if constexpr (IN == 1) {
      f[0] = operand(w);
    } else {
      float x[8];
      if constexpr (IN == 2) {
        typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
        const u32x4 v = {w[0], w[1], w[2], w[3]};
        const f16x8 h = __builtin_bit_cast(f16x8, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (float)h[i];
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
      }
      uint32_t words[IN][4];
      split<IN, 8>(x, words);
#pragma unroll
      for (int p = 0; p < IN; ++p) f[p] = operand(words[p]);
    }
  }
};

template <int P>
__device__ __forceinline__ void split_operand(b16x8 (&f)[P], const float (&x)[8]) {
  uint32_t words[P][4];
  split<P, 8>(x, words);
#pragma unroll
  for (int p = 0; p < P; ++p) f[p] = operand(words[p]);
}

// exp of a difference of sums: 2 to the power of its fp32 part, what that leaves made good
// to first order.
__device__ __forceinline__ float exp_sum(double d) {
  const double y = d * 1.4426950408889634;
  const float x = (float)y, e = __builtin_amdgcn_exp2f(x);
  return x > 127.f ? e : __builtin_fmaf(e, (float)(y - (double)x) * 0.69314718f, e);
}

// A token's log decay as it is summed: minus infinity (and what else exp makes
// 0) as a finite number, so that differences of sums stay what they are.
__device__ __forceinline__ double summand(float g) { return g < -1e6f ? -1e6 : (double)g; }

// LDS written by a wave is read by its other lanes.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// A number that is the same in every lane, in a scalar register: the addresses and
// buffers made of it are too (else every access goes round a loop over its lanes' buffers).
__device__ __forceinline__ int scalar(int x) { return __builtin_amdgcn_readfirstlane(x); }

// First chunk of a sequence in the workspace, and a chunk's sequence and number in it.
__device__ __forceinline__ int64_t first_chunk(const DeltaArgs& a, const Span& s, int b) {
  return a.offsets != nullptr ? s.first / C + b : (int64_t)b * a.chunks;
}
__device__ __forceinline__ bool chunk_of(const DeltaArgs& a, uint32_t slot, int& b, int& c) {
  if (a.offsets != nullptr) {
    const Pieces p = {a.offsets, a.rows, a.B, C, 0xffffffffu / C + 1};
    const bool found = find_unit(p, slot, b, c);
    b = scalar(b);
    c = scalar(c);
    return found;
  }
  b = scalar((int)divide(slot, a.chunks, a.by_chunks));
  c = (int)slot - b * a.chunks;
  return true;
}

// Chunks that the gradients are taken of at once, and whose first state (and the
// gradient of the last one) is kept: as many as LDS holds.
template <class E, int DKP>
__host__ __device__ constexpr int group_chunks() {
  return DKP == 128 && E::id != PRNN_DATA_FLOAT ? 2 : 1;
}
// First group of a sequence in the workspace, and a group's sequence and number in it.
__device__ __forceinline__ int64_t first_group(const DeltaArgs& a, const Span& s, int b) {
  return a.offsets != nullptr ? s.first / (a.group * C) + b : (int64_t)b * a.groups;
}
__device__ __forceinline__ bool group_of(const DeltaArgs& a, uint32_t slot, int& b, int& c) {
  if (a.offsets != nullptr) {
    const Pieces p = {a.offsets, a.rows, a.B, a.group * C, a.by_group_tokens};
    const bool found = find_unit(p, slot, b, c);
    b = scalar(b);
    c = scalar(c);
    return found;
  }
  b = scalar((int)divide(slot, a.groups, a.by_groups));
  c = (int)slot - b * a.groups;
  return true;
}

// Workgroups are dealt to the 8 XCDs in turn; those of neighbouring numbers, which
// read the same rows, go to one of them, whose L2 then has them.
__device__ __forceinline__ uint32_t near(uint32_t id, uint32_t count) {
  const uint32_t whole = count / 8 * 8;
  return id < whole ? id % 8 * (whole / 8) + id / 8 : id;
}

// acc += x y for single accumulators.
template <int NX, int NY>
__device__ __forceinline__ void product(f32x4& acc, const b16x8 (&x)[NX], const b16x8 (&y)[NY]) {
#pragma unroll
  for (int s = kFull - 1; s >= 0; --s)  // small terms first
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const int j = s - i;
      if (j < 0 || j >= NY) continue;
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[i], y[j], acc, 0, 0, 0);
    }
}

// -- what depends on no state ------------------------------------------------------------------

// A wave for each chunk and head, alone in its workgroup where that spreads them over
// more units.  T' is inverted in fp32: its two diagonal blocks of 16 by
// substitution, a column a lane, then T'_21 = -T'_22 A'_21 T'_11 on the matrix
// cores.
template <class E, int DKP, bool VEC>
__global__ void __launch_bounds__(256) delta_prepare_kernel(DeltaArgs a) {
  typedef typename E::raw raw;
  constexpr int IN = Parts<E>::kIn, kRow = 36;
  __shared__ float mem[4][2][C][kRow];
  __shared__ double sums[4][C];
  __shared__ float betas[4][C];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, g = lane >> 4, l = lane & 15;
  const uint32_t id = blockIdx.x * (blockDim.x / 64) + wave;
  const uint32_t slot = scalar((int)divide(id, a.H, a.by_heads));
  const int h = (int)(id - slot * a.H);
  int b, c;
  if (slot >= (uint32_t)a.slots || !chunk_of(a, slot, b, c)) return;
  const Span s = span_of(a, b);
  const int n = min(C, s.len - c * C);
  if (n <= 0) return;
  float (&A)[C][kRow] = mem[wave][0], (&T)[C][kRow] = mem[wave][1];
  char* const block = a.blocks + ((int64_t)slot * a.H + h) * kDeltaBlock;
  const int64_t t0 = (int64_t)c * C;

  // The rows of k and q, as much as registers hold of them at once before anything
  // waits: where there are few chunks, a trip to memory is most of what this launch takes.
  constexpr int kAhead = VEC ? (DKP / 32 < 4 ? DKP / 32 : 4) : 1;
  const uint32_t ks = (uint32_t)a.k.token * (uint32_t)sizeof(raw), qs = (uint32_t)a.q.token * (uint32_t)sizeof(raw);
  const __amdgpu_buffer_rsrc_t rk = make_rsrc(
      static_cast<const raw*>(a.k.p) + base_of(a.k, a, s, b, h) + t0 * a.k.token, (uint32_t)scalar((n - 1) * (int)ks + a.Dk * (int)sizeof(raw)));
  const __amdgpu_buffer_rsrc_t rq = make_rsrc(
      static_cast<const raw*>(a.q.p) + base_of(a.q, a, s, b, h) + t0 * a.q.token, (uint32_t)scalar((n - 1) * (int)qs + a.Dk * (int)sizeof(raw)));
  RowPart<E, VEC> pk[kAhead][2], pq[kAhead][2];
  auto fetch = [&](int d) {
#pragma unroll
    for (int y = 0; y < kAhead; ++y)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int row = 16 * x + l;
        pk[y][x].load(rk, row < n ? row * ks : kOutside, d + 32 * y + 8 * g, a.Dk);
        pq[y][x].load(rq, row < n ? row * qs : kOutside, d + 32 * y + 8 * g, a.Dk);
      }
  };
  float log_decay = 0.f, beta = 0.f;
  const int t = lane & 31;
  if (t < n) {
    if (a.g.p != nullptr) log_decay = static_cast<const float*>(a.g.p)[base_of(a.g, a, s, b, h) + (t0 + t) * a.g.token];
    beta = static_cast<const float*>(a.beta.p)[base_of(a.beta, a, s, b, h) + (t0 + t) * a.beta.token];
  }
  fetch(0);

  // the decays' sums, and the factors
  double G = summand(log_decay);
#pragma unroll
  for (int d = 1; d < C; d *= 2) {
    const double y = __shfl_up(G, d, C);
    if (t >= d) G += y;
  }
  if (lane < C) {
    sums[wave][t] = G;
    betas[wave][t] = beta;
  }
  wave_sync();
  if (lane < C) {
    const float up = exp_sum(G), down = exp_sum(sums[wave][C - 1] - G);
    float* const f = reinterpret_cast<float*>(block + kDeltaVec) + t;
    f[kUp * C] = up;
    f[kScaledUp * C] = a.scale * up;
    f[kInto * C] = down * beta;
    f[kDown * C] = down;
    f[kBeta * C] = beta;
    reinterpret_cast<double*>(block + kDeltaSums)[t] = G;
  }

  // k k^T and q k^T as tiles (j, i): lane (g, l) has tokens j = 16 tj + 4 g + r of i = 16 ti + l
  f32x4 kk[3], qk[3];  // (ti, tj) = (0, 0), (1, 0), (1, 1)
#pragma unroll
  for (int x = 0; x < 3; ++x) kk[x] = qk[x] = f32x4(0.f);
  for (int d = 0; d < a.Dk; d += 32 * kAhead) {
    if (d > 0) fetch(d);
#pragma unroll
    for (int y = 0; y < kAhead; ++y) {
      b16x8 K[2][IN], Q[2][IN];
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        pk[y][x].take(K[x]);
        pq[y][x].take(Q[x]);
      }
#pragma unroll
      for (int x = 0; x < 3; ++x) {
        const int ti = (x + 1) / 2, tj = x / 2;
        product(kk[x], K[tj], K[ti]);
        product(qk[x], K[tj], Q[ti]);
      }
    }
  }
#pragma unroll
  for (int x = 0; x < 3; ++x) {
    const int ti = (x + 1) / 2, tj = x / 2, i = 16 * ti + l, j = 16 * tj + 4 * g;
    f32x4 y;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float f = j + r <= i ? exp_sum(sums[wave][i] - sums[wave][j + r]) * betas[wave][j + r] : 0.f;
      y[r] = j + r < i ? kk[x][r] * f : 0.f;
      qk[x][r] = j + r <= i ? qk[x][r] * (a.scale * f) : 0.f;
    }
    *reinterpret_cast<f32x4*>(&A[i][j]) = y;
  }
  wave_sync();
  // the diagonal blocks' inverses, column l of block g % 2
  {
    const int o = 16 * (g & 1);
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = i == l ? 1.f : 0.f;
    // four columns of the block at a time, each as soon as it is done into all rows below
#pragma unroll
    for (int j0 = 0; j0 < 16; j0 += 4) {
#pragma unroll
      for (int i = j0 + 1; i < 16; ++i) {
        const f32x4 row = *reinterpret_cast<const f32x4*>(&A[o + i][o + j0]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j0 + j < i) x[i] = __builtin_fmaf(-row[j], x[j0 + j], x[i]);
      }
    }
    if (g < 2) {
#pragma unroll
      for (int i = 0; i < 16; ++i) T[o + i][o + l] = x[i];
    } else if (g == 2) {
#pragma unroll
      for (int i = 0; i < 16; ++i) T[i][16 + l] = 0.f;
    }
  }
  wave_sync();
  {
    f32x4 x = f32x4(0.f);
#pragma unroll
    for (int m = 0; m < 4; ++m) x = __builtin_amdgcn_mfma_f32_16x16x4f32(A[16 + l][4 * m + g], T[4 * m + g][l], x, 0, 0, 0);
#pragma unroll
    for (int r = 0; r < 4; ++r) A[4 * g + r][16 + l] = x[r];
    wave_sync();
    f32x4 y = f32x4(0.f);
#pragma unroll
    for (int m = 0; m < 4; ++m) y = __builtin_amdgcn_mfma_f32_16x16x4f32(T[16 + l][16 + 4 * m + g], A[4 * m + g][16 + l], y, 0, 0, 0);
#pragma unroll
    for (int r = 0; r < 4; ++r) T[16 + 4 * g + r][l] = -y[r];
  }
  wave_sync();
  // out in parts: a row and 16 positions a lane
  auto put = [&](const float (&m)[C][kRow], int to) {
    const int row = lane >> 1;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int unit = 2 * (lane & 1) + u;
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = m[row][16 * (e / 4) + 4 * unit + e % 4];
      uint32_t words[kFull][4];
      split<kFull, 8>(x, words);
#pragma unroll
      for (int p = 0; p < kFull; ++p)
        *reinterpret_cast<u32x4*>(block + to + p * kPart + delta_at(row, 8 * unit)) = u32x4{words[p][0], words[p][1], words[p][2], words[p][3]};
    }
  };
  put(T, kDeltaT);
#pragma unroll
  for (int x = 0; x < 3; ++x) {
    const int ti = (x + 1) / 2, tj = x / 2;
    *reinterpret_cast<f32x4*>(&A[16 * ti + l][16 * tj + 4 * g]) = qk[x];
  }
  *reinterpret_cast<f32x4*>(&A[l][16 + 4 * g]) = f32x4(0.f);
  wave_sync();
  put(A, kDeltaP);
}

// -- the walk along a sequence --------------------------------------------------------------------

// QUERIES: with q and P'.
template <class E, int DKP, bool QUERIES>
struct Shape {
  static constexpr int IN = Parts<E>::kIn, KT = DKP / 16, kTile = 2 * C * IN;  // bytes of a tile's column
  static constexpr int kK = 0, kQ = kTile * DKP, kV = kQ + (QUERIES ? kTile * DKP : 0), kM = kV + kTile * 64;
  static constexpr int kVecs = kM + (QUERIES ? 2 : 1) * 3 * kPart, kLds = kVecs + 5 * 4 * C;
};

// What a workgroup works on: 64 columns of one head's state, or of what a segment
// makes of the identity (move), and one segment of a sequence.
struct Where {
  int b, h, col0, cols;
  bool move;
  Span s;
  int seg, segments;  // its number, and the sequence's
  int lo, hi;         // its chunks
  int chunks;         // of the sequence
  int64_t chunk, group, part;  // the sequence's first chunk, group and segment in the workspace
};

// tiles: column tiles of a head; the launch has as many workgroups for every
// head and segment.  HEADS_FIRST: all segments of a head before the next head's.  In the walks for the
// ends some segments have less to do or nothing, and an XCD, which has a run of
// neighbouring numbers, would be left with only such (packed sequences of 1 .. 700 tokens 69.1 -> 66.1 us,
// 32768 tokens of 32 heads of 128 1087 -> 1073).  Elsewhere it gains nothing: there an XCD has the heads of a
// few segments.
template <bool HEADS_FIRST>
__device__ __forceinline__ bool where(const DeltaArgs& a, int tiles, uint32_t by_tiles, Where& w) {
  const uint32_t id = near(blockIdx.x, gridDim.x), state = scalar((int)divide(id, tiles, by_tiles));
  const int tile = (int)(id - state * tiles);
  uint32_t piece;
  if (HEADS_FIRST) {
    w.h = scalar((int)divide(state, a.pieces, a.by_pieces));
    piece = state - (uint32_t)w.h * a.pieces;
  } else {
    piece = scalar((int)divide(state, a.H, a.by_heads));
    w.h = (int)(state - piece * a.H);
  }
  if (a.units > 0) {
    const Pieces p = {a.offsets, a.rows, a.B, a.seg_chunks * C, a.by_seg_tokens};
    if (!find_unit(p, piece, w.b, w.seg)) return false;
    w.b = scalar(w.b);
    w.seg = scalar(w.seg);
  } else {
    w.b = scalar((int)divide(piece, a.segments, a.by_segments));
    w.seg = (int)piece - w.b * a.segments;
  }
  w.move = tile >= a.tiles;
  w.col0 = 64 * (w.move ? tile - a.tiles : tile);
  w.cols = min(64, (w.move ? a.Dk : a.Dv) - w.col0);
  w.s = span_of(a, w.b);
  w.chunks = (w.s.len + C - 1) / C;
  w.segments = w.chunks > 0 ? scalar((int)divide(w.chunks - 1, a.seg_chunks, a.by_seg_chunks)) + 1 : 1;
  w.lo = w.seg * a.seg_chunks;
  w.hi = min(w.chunks, w.lo + a.seg_chunks);
  w.chunk = first_chunk(a, w.s, w.b);
  w.group = first_group(a, w.s, w.b);
  w.part = a.offsets != nullptr ? w.s.first / (a.seg_chunks * C) : (int64_t)w.b * a.segments;
  return true;
}

// A state in memory, [Dk][stride], as this lane's elements: row 32 (t / 2) + 8 g +
// 4 (t % 2) + r of its column.
struct StateAt {
  __amdgpu_buffer_rsrc_t rsrc;
  int rows, first, step;
  __device__ __forceinline__ StateAt(const float* p, int Dk, int stride, int col, bool exists, int lane)
      : rsrc(make_rsrc(p, (uint32_t)(Dk * stride) * 4u)),
        rows(exists ? Dk - 8 * (lane >> 4) : 0),
        first(4 * (8 * (lane >> 4) * stride + col)),
        step(4 * stride) {}
  __device__ __forceinline__ uint32_t at(int t, int r) const {
    const int row = 32 * (t / 2) + 4 * (t % 2) + r;
    return row < rows ? (uint32_t)(first + row * step) : kOutside;
  }
};

template <int KT>
__device__ __forceinline__ void load_state(f32x4 (&S)[KT], const float* p, int Dk, int stride, int col, bool exists, int lane) {
  if (p == nullptr) {
#pragma unroll
    for (int t = 0; t < KT; ++t) S[t] = f32x4(0.f);
    return;
  }
  const StateAt x(p, Dk, stride, col, exists, lane);
#pragma unroll
  for (int t = 0; t < KT; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) S[t][r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(x.rsrc, x.at(t, r), 0, kPlain));
}
template <int KT>
__device__ __forceinline__ void store_state(const f32x4 (&S)[KT], float* p, int Dk, int stride, int col, bool exists, int lane) {
  const StateAt x(p, Dk, stride, col, exists, lane);
#pragma unroll
  for (int t = 0; t < KT; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[t][r]), x.rsrc, x.at(t, r), 0, kPlain);
}

// 4 x 4 values of 4 neighbouring lanes, transposed: lane i's value j becomes lane j's i.
__device__ __forceinline__ f32x4 transposed(const f32x4& x, int lane) {
  auto from = [](float v, auto way) { return __uint_as_float(__builtin_amdgcn_update_dpp(0u, __float_as_uint(v), decltype(way)::value, 0xF, 0xF, false)); };
  const std::integral_constant<int, 0xB1> beside;   // lane ^ 1
  const std::integral_constant<int, 0x4E> across;   // lane ^ 2
  const bool odd = lane & 1, high = lane & 2;
  // (every lane exchanges, then chooses)
  const float b0 = from(x[0], beside), b1 = from(x[1], beside), b2 = from(x[2], beside), b3 = from(x[3], beside);
  const float a0 = odd ? b1 : x[0], a1 = odd ? x[1] : b0, a2 = odd ? b3 : x[2], a3 = odd ? x[3] : b2;
  const float c0 = from(a0, across), c1 = from(a1, across), c2 = from(a2, across), c3 = from(a3, across);
  return f32x4{high ? c2 : a0, high ? c3 : a1, high ? a2 : c0, high ? a3 : c1};
}

// A state into the workspace, rows `pitch` (a multiple of 4) apart from `p` on, 16
// bytes a lane: columns col0 + 16 wave .. + 15 of it.  Stored 4 bytes a lane it
// takes four times the accesses, as many as the rest of a chunk's work takes time.
template <int KT>
__device__ __forceinline__ void keep_state(const f32x4 (&S)[KT], float* p, int Dk, int pitch, int col0, int lane) {
  const __amdgpu_buffer_rsrc_t rsrc = make_rsrc(p, (uint32_t)(Dk * pitch) * 4u);
  const int col = col0 + (lane & 12), row = 8 * (lane >> 4) + (lane & 3);
  const int rows = col < pitch ? Dk - row : 0, first = (row * pitch + col) * 4;
#pragma unroll
  for (int t = 0; t < KT; ++t) {
    const int to = 32 * (t / 2) + 4 * (t % 2);
    const f32x4 y = transposed(S[t], lane);
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, y), rsrc, to < rows ? (uint32_t)(first + to * pitch * 4) : kOutside, 0, kPlain);
  }
}

// The chunk's matrices and factors on their way from the workspace to LDS.
// (PAIRS: P' too; T' alone leaves half of the last round's threads to the factors.)
template <bool PAIRS>
struct Block {
  static constexpr int kUnits = (PAIRS ? 2 : 1) * 3 * kPart / 16, kWhole = kUnits / 256, kRest = kUnits % 256, kFactors = 5 * C / 4;
  u32x4 m[kWhole], f;
  __device__ __forceinline__ void load(const char* p) {
#pragma unroll
    for (int i = 0; i < kWhole; ++i) m[i] = reinterpret_cast<const u32x4*>(p)[i * 256 + threadIdx.x];
    if ((int)threadIdx.x < kRest)
      f = reinterpret_cast<const u32x4*>(p)[kWhole * 256 + threadIdx.x];
    else if ((int)threadIdx.x < kRest + kFactors)
      f = reinterpret_cast<const u32x4*>(p + kDeltaVec)[threadIdx.x - kRest];
  }
  // (the factors lie behind the matrices: see Shape)
  __device__ __forceinline__ void store(char* matrices) const {
#pragma unroll
    for (int i = 0; i < kWhole; ++i) reinterpret_cast<u32x4*>(matrices)[i * 256 + threadIdx.x] = m[i];
    if ((int)threadIdx.x < kRest + kFactors) reinterpret_cast<u32x4*>(matrices)[kWhole * 256 + threadIdx.x] = f;
  }
};

// The factors of an operand's 8 tokens.
__device__ __forceinline__ void factors(float (&f)[8], const char* vecs, int which, int lane) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const f32x4 x = *reinterpret_cast<const f32x4*>(vecs + 4 * (which * C + 16 * h + 4 * (lane >> 4)));
#pragma unroll
    for (int r = 0; r < 4; ++r) f[4 * h + r] = x[r];
  }
}

// The wave's 16 columns of a tile of W = 64, tokens as an operand's.
template <class E>
__device__ __forceinline__ void read_values(b16x8 (&V)[Parts<E>::kIn], const char* v, int wave, int lane) {
  const int g = lane >> 4, l = lane & 15;
  const int base = (row_at<64>(4 * g + (l >> 2)) ^ ((2 * wave + ((l & 3) >> 1)) << 4)) + 8 * (l & 1);
#pragma unroll
  for (int p = 0; p < Parts<E>::kIn; ++p) {
    u32x2 half[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) half[h] = read_columns(v, base + p * (C * 64 * 2) + 16 * h * (2 * 64));
    const uint32_t words[4] = {half[0][0], half[0][1], half[1][0], half[1][1]};
    V[p] = operand(words);
  }
}
template <int P>
__device__ __forceinline__ void values_of(float (&x)[8], const b16x8 (&V)[P]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    x[e] = (float)V[P - 1][e];
#pragma unroll
    for (int p = P - 2; p >= 0; --p) x[e] += (float)V[p][e];
  }
}

// Rows 16 t .. (as the state deals them) of a tile's transpose, tokens as an operand's.
template <class E, int DKP>
__device__ __forceinline__ void read_keys(b16x8 (&K)[Parts<E>::kIn], const char* k, int lane, int t) {
  const int g = lane >> 4, l = lane & 15;
  const int base = row_at<DKP>(4 * g + (l >> 2)) ^ ((l & 3) << 4);
#pragma unroll
  for (int p = 0; p < Parts<E>::kIn; ++p) {
    u32x2 half[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      half[h] = read_columns(k, (base ^ (64 * (t / 2))) + p * (C * DKP * 2) + 16 * h * (2 * DKP) + 8 * (t % 2));
    const uint32_t words[4] = {half[0][0], half[0][1], half[1][0], half[1][1]};
    K[p] = operand(words);
  }
}

template <int P>
__device__ __forceinline__ void state_operand(b16x8 (&A)[P], const f32x4& lo, const f32x4& hi) {
  const float x[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  split_operand<P>(A, x);
}

// NaN from the first value on that is not finite.
template <int N>
__device__ __forceinline__ void watch(float& z, const f32x4 (&x)[N]) {
#pragma unroll
  for (int t = 0; t < N; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) z = __builtin_fmaf(x[t][r], 0.f, z);
}

// Four neighbouring values of a row.
template <class E>
__device__ __forceinline__ void put4(void* p, int64_t at, const f32x4& x, int live, bool wide, bool vec) {
  typedef typename E::raw raw;
  if (live <= 0) return;
  if (wide || sizeof(raw) == 4) {
    float* const to = static_cast<float*>(p) + at;
    if (vec) {
      *reinterpret_cast<f32x4*>(to) = x;
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (r < live) to[r] = x[r];
    }
    return;
  }
  raw* const to = static_cast<raw*>(p) + at;
  typedef raw raw4 __attribute__((ext_vector_type(4)));
  if (vec) {
    raw4 y;
#pragma unroll
    for (int r = 0; r < 4; ++r) y[r] = E::put(x[r]);
    *reinterpret_cast<raw4*>(to) = y;
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (r < live) to[r] = E::put(x[r]);
  }
}

// The recurrence over a segment for this wave's columns, straight from memory:
// the rows of o, and S.  Slow; see the file comment.
template <class E, int DKP>
__device__ __forceinline__ void delta_tokens(const DeltaArgs& a, const Where& w, int wave, int lane, f32x4 (&S)[DKP / 16]) {
  typedef typename E::raw raw;
  const int first = 8 * (lane >> 4), col = 16 * wave + (lane & 15);
  const raw* q = static_cast<const raw*>(a.q.p) + base_of(a.q, a, w.s, w.b, w.h) + first;
  const raw* k = static_cast<const raw*>(a.k.p) + base_of(a.k, a, w.s, w.b, w.h) + first;
  const raw* v = static_cast<const raw*>(a.v.p) + base_of(a.v, a, w.s, w.b, w.h) + w.col0;
  raw* o = static_cast<raw*>(const_cast<void*>(a.o.p)) + base_of(a.o, a, w.s, w.b, w.h) + w.col0;
  const float* g = a.g.p != nullptr ? static_cast<const float*>(a.g.p) + base_of(a.g, a, w.s, w.b, w.h) : nullptr;
  const float* beta = static_cast<const float*>(a.beta.p) + base_of(a.beta, a, w.s, w.b, w.h);
  int rows = a.Dk - first;  // rows of the state from the lane's first one on
  keep(rows);
#pragma nounroll
  for (int64_t t = (int64_t)w.lo * C; t < min((int64_t)w.s.len, (int64_t)w.hi * C); ++t) {
    const float d = g != nullptr ? expf(g[t * a.g.token]) : 1.f;
    float found = 0.f, out = 0.f;
#pragma unroll
    for (int x = 0; x < DKP / 16; ++x)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 32 * (x / 2) + 4 * (x % 2) + r;
        if (row < rows) {
          S[x][r] *= d;
          found = __builtin_fmaf(E::get(k[t * a.k.token + row]), S[x][r], found);
        }
      }
    found += __shfl_xor(found, 16);
    found += __shfl_xor(found, 32);
    const float u = beta[t * a.beta.token] * ((col < w.cols ? E::get(v[t * a.v.token + col]) : 0.f) - found);
#pragma unroll
    for (int x = 0; x < DKP / 16; ++x)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 32 * (x / 2) + 4 * (x % 2) + r;
        if (row < rows) {
          S[x][r] = __builtin_fmaf(E::get(k[t * a.k.token + row]), u, S[x][r]);
          out = __builtin_fmaf(E::get(q[t * a.q.token + row]), S[x][r], out);
        }
      }
    out += __shfl_xor(out, 16);
    out += __shfl_xor(out, 32);
    if (lane < 16 && col < w.cols) o[t * a.o.token + col] = E::put(out * a.scale);
  }
}

// acc[t] += x[t] y and, with BOTH, other[t] += y z[t], the accumulators in turn.
template <int IN, bool BOTH>
__device__ __forceinline__ void state_products(f32x4 (&acc)[2], f32x4 (&other)[2], const b16x8 (&x)[2][IN],
                                               const b16x8 (&z)[2][IN], const b16x8 (&y)[kFull]) {
#pragma unroll
  for (int s = kFull - 1; s >= 0; --s)  // small terms first
#pragma unroll
    for (int i = 0; i < IN; ++i) {
      const int j = s - i;
      if (j < 0) continue;
#pragma unroll
      for (int t = 0; t < 2; ++t) acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[t][i], y[j], acc[t], 0, 0, 0);
      if (BOTH)
#pragma unroll
        for (int t = 0; t < 2; ++t) other[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(y[j], z[t][i], other[t], 0, 0, 0);
    }
}

// The priority of a wave by the chunks it has done.  Of two workgroups on a unit
// the older one's waves issue first: it ends after 345 us, the other after 450 (128 chunks of 128 x 64
// bf16 each).  A step lower every two chunks, the one that is behind mostly comes first.  Taken by
// the walks of split sequences, whose workgroups are all there from the start: 32768 tokens of 32 bf16
// heads of 128 1123 us without, 1097 with; 4 x 8192 of 16 592 and 568.  (In the walks of 8 x 1024 tokens of
// 64 heads, which follow one another on a unit, 335 and 343; in those of the gradients, 18 fp32 heads of
// 64, 74.7 and 76.1.)
__device__ __forceinline__ void urge(int done) {
  switch (done >> 1 & 3) {
    case 0: __builtin_amdgcn_s_setprio(3); break;
    case 1: __builtin_amdgcn_s_setprio(2); break;
    case 2: __builtin_amdgcn_s_setprio(1); break;
    default: __builtin_amdgcn_s_setprio(0);
  }
}

// What the walk does: the outputs and the final state; x and the chunks' first
// states for the gradients; or the segments' ends and moves.
enum Walk { kOutputs, kKeep, kEnds };

// Forward: grid tiles (kEnds: and move tiles) x H x segments.
template <class E, int DKP, bool VEC, Walk WALK>
__global__ void __launch_bounds__(256, DKP == 256 ? 1 : WALK == kOutputs && VEC && E::id != PRNN_DATA_FLOAT ? 3 : 2) delta_forward_kernel(DeltaArgs a) {
  constexpr bool OUT = WALK == kOutputs;
  typedef Shape<E, DKP, OUT> Sh;
  typedef typename E::raw raw;
  constexpr int IN = Sh::IN, KT = Sh::KT, GROUP = group_chunks<E, DKP>();
  extern __shared__ __attribute__((aligned(16))) char lds[];
  char *const kt = lds + Sh::kK, *const qt = lds + Sh::kQ, *const vt = lds + Sh::kV, *const mt = lds + Sh::kM,
              *const vecs = lds + Sh::kVecs;
  Where w;
  if (!where<WALK == kEnds>(a, WALK == kEnds ? a.tiles + a.move_tiles : a.tiles, WALK == kEnds ? a.by_all_tiles : a.by_tiles, w)) return;
  // (the ends of the last segment are not needed, nor what the first one makes of any state but its own)
  if (WALK == kEnds && (w.seg + 1 >= w.segments || (w.move && w.seg == 0))) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4, l = lane & 15;
  const int col = 16 * wave + l;
  if (OUT && a.lengths != nullptr) {  // rows of padding are zeros
    raw* const o = static_cast<raw*>(const_cast<void*>(a.o.p)) + base_of(a.o, a, w.s, w.b, w.h) + w.col0;
    const int64_t end = min((int64_t)a.T, (int64_t)(w.seg + 1) * a.seg_chunks * C);
    for (int64_t t = max((int64_t)w.s.len, (int64_t)w.lo * C); t < end; ++t)
      if ((int)threadIdx.x < w.cols) o[t * a.o.token + threadIdx.x] = E::put(0.f);
  }
  if (w.seg >= w.segments) return;
  const uint32_t qs = (uint32_t)a.q.token * (uint32_t)sizeof(raw), ks = (uint32_t)a.k.token * (uint32_t)sizeof(raw),
                 vs = (uint32_t)a.v.token * (uint32_t)sizeof(raw);
  const raw* const q = static_cast<const raw*>(a.q.p) + base_of(a.q, a, w.s, w.b, w.h);
  const raw* const k = static_cast<const raw*>(a.k.p) + base_of(a.k, a, w.s, w.b, w.h);
  const raw* const v = static_cast<const raw*>(a.v.p) + base_of(a.v, a, w.s, w.b, w.h) + (w.move ? 0 : w.col0);
  const int vcols = w.move ? 0 : w.cols;  // (moves: values of zeros)
  Rows<E, C, DKP, 256, VEC> rq(qs, a.Dk, false), rk(ks, a.Dk, false);
  Rows<E, C, 64, 256, VEC> rv(vs, vcols, false);
  Block<OUT> block;
  static_assert(Sh::kVecs == Sh::kM + 16 * Block<OUT>::kUnits, "factors behind the matrices");
  // (in two parts: all at once they fill the queue of the unit's loads, and the waves wait to issue them)
  auto fetch = [&](int c) {
    const int n = c < w.hi ? min(C, w.s.len - c * C) : 0;
    const int64_t t0 = n == 0 ? 0 : (int64_t)c * C;
    rk.load(k, t0, n, ks, a.Dk, false);
    if (OUT) rq.load(q, t0, n, qs, a.Dk, false);
  };
  auto fetch_rest = [&](int c) {
    const int n = c < w.hi ? min(C, w.s.len - c * C) : 0;
    const int64_t t0 = n == 0 ? 0 : (int64_t)c * C;
    rv.load(v, t0, n, vs, vcols, false);
    if (n > 0) block.load(a.blocks + ((w.chunk + c) * a.H + w.h) * kDeltaBlock);
  };
  fetch(w.lo);
  fetch_rest(w.lo);
  const size_t head = (size_t)w.b * a.H + w.h;
  const int64_t matrix = (int64_t)a.Dk * a.pitch;
  const bool split = w.segments > 1;
  // The state the segment starts from.  (A split sequence's own first state is
  // kept in the workspace by the launch for the ends: another workgroup may write the
  // final state in its place.)
  auto start = [&](f32x4 (&S)[KT]) {
    if (WALK == kEnds && w.move) {
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[t][r] = 32 * (t / 2) + 8 * g + 4 * (t % 2) + r == w.col0 + col ? 1.f : 0.f;
    } else if (WALK == kEnds && w.seg > 0) {
      load_state<KT>(S, nullptr, a.Dk, a.Dv, 0, false, lane);
    } else if (WALK != kEnds && split && w.seg > 0) {
      load_state<KT>(S, a.ends + ((w.part + w.seg - 1) * a.H + w.h) * matrix, a.Dk, a.pitch, w.col0 + col, col < w.cols, lane);
    } else if (WALK != kEnds && split && a.s_in != nullptr) {
      load_state<KT>(S, a.firsts + (w.part * a.H + w.h) * matrix, a.Dk, a.pitch, w.col0 + col, col < w.cols, lane);
    } else {
      load_state<KT>(S, a.s_in != nullptr ? a.s_in + head * a.Dk * a.Dv : nullptr, a.Dk, a.Dv, w.col0 + col, col < w.cols, lane);
    }
  };
  f32x4 S[KT];
  start(S);
  const bool kept = w.col0 + col < a.pitch;
  if (WALK == kEnds && w.seg == 0 && a.s_in != nullptr)
    keep_state<KT>(S, a.firsts + (w.part * a.H + w.h) * matrix, a.Dk, a.pitch, w.col0 + 16 * wave, lane);
  bool broken = false;

  for (int c = w.lo; c < w.hi; ++c) {
    const int n = min(C, w.s.len - c * C);
    if (WALK != kKeep && split) urge(c - w.lo);
    rk.store(kt);
    if (OUT) rq.store(qt);
    rv.store(vt);
    block.store(mt);
    __syncthreads();
    fetch(c + 1);
    if constexpr (WALK == kKeep) {
      // (the stores behind all loads: what waits for a load waits for the stores before it)
      fetch_rest(c + 1);
      if (c % GROUP == 0) store_state<KT>(S, a.S + ((w.group + c / GROUP) * a.H + w.h) * matrix, a.Dk, a.pitch, w.col0 + col, kept, lane);
    }
    const float whole = *reinterpret_cast<const float*>(vecs + 4 * (kUp * C + C - 1));

    // K S and (Q S)^T
    const int rows = row_at<DKP>(l) ^ (g << 4);  // row l of a tile of 16, unit g
    f32x4 x[2], O[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) x[t] = O[t] = f32x4(0.f);
#pragma unroll
    for (int s = 0; s < DKP / 32; ++s) {
      b16x8 A[kFull], K[2][IN], Q[2][IN];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int p = 0; p < IN; ++p) {
          K[t][p] = read_row(kt, (rows ^ (64 * s)) + p * (C * DKP * 2) + t * (32 * DKP));
          if (OUT) Q[t][p] = read_row(qt, (rows ^ (64 * s)) + p * (C * DKP * 2) + t * (32 * DKP));
        }
      state_operand<kFull>(A, S[2 * s], S[2 * s + 1]);
      state_products<IN, OUT>(x, O, K, Q, A);
    }
    if (WALK != kKeep) fetch_rest(c + 1);
    // x = T' (v - up K S)
    float y[8], f[8];
    {
      b16x8 V[IN], Y[kFull], T[2][kFull];
      read_values<E>(V, vt, wave, lane);
      values_of(y, V);
      factors(f, vecs, kUp, lane);
#pragma unroll
      for (int t = 0; t < 2; ++t) read_matrix<kFull>(T[t], mt, t, lane);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = __builtin_fmaf(-f[e], x[e / 4][e % 4], y[e]);
      split_operand<kFull>(Y, y);
      x[0] = x[1] = f32x4(0.f);
      products<kFull, kFull, 2>(x, T, Y);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = x[e / 4][e % 4];
    if constexpr (WALK == kKeep) {
      float* const to = a.x + (((w.group + c / GROUP) * a.H + w.h) * GROUP + c % GROUP) * C * a.pitch + w.col0 + col;
      if (kept)
#pragma unroll
        for (int e = 0; e < 8; ++e) to[(16 * (e / 4) + 4 * g + e % 4) * a.pitch] = y[e];
    }
    // S = up_C S + K^T (down beta x)
    b16x8 D[kFull];
    {
      float z[8];
      factors(f, vecs, kInto, lane);
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] = y[e] * f[e];
      split_operand<kFull>(D, z);
    }
    if constexpr (OUT) {
      // o^T = scale up (Q S)^T + x^T P'^T
      b16x8 Y[kFull], P[2][kFull];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        read_matrix<kFull>(P[t], mt + kDeltaP, t, lane);
        O[t] *= *reinterpret_cast<const float*>(vecs + 4 * (kScaledUp * C + 16 * t + l));
      }
      split_operand<kFull>(Y, y);
      products<kFull, kFull, 2>(O, Y, P);
    }
#pragma unroll
    for (int t = 0; t < KT; t += 2) {
      b16x8 K[2][IN];
      f32x4 z[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        read_keys<E, DKP>(K[u], kt, lane, t + u);
        z[u] = S[t + u] * whole;
      }
      products<IN, kFull, 2>(z, K, D);
      S[t] = z[0];
      S[t + 1] = z[1];
    }
    if constexpr (OUT) {
      float z = 0.f;
      watch(z, O);
      broken = broken || wave_any(z != 0.f);
      raw* const o = static_cast<raw*>(const_cast<void*>(a.o.p));
      const int64_t to = base_of(a.o, a, w.s, w.b, w.h) + (int64_t)c * C * a.o.token + w.col0 + 16 * wave + 4 * g;
#pragma unroll
      for (int t = 0; t < 2; ++t)
        if (16 * t + l < n) put4<E>(o, to + (16 * t + l) * a.o.token, O[t], w.cols - 16 * wave - 4 * g, false, (a.vec & 2) != 0);
    }
    __syncthreads();
  }
  if constexpr (OUT) {
    float z = 0.f;
    watch(z, S);
    if (broken || wave_any(z != 0.f)) {
      start(S);
      delta_tokens<E, DKP>(a, w, wave, lane, S);
    }
    if (a.s_out != nullptr && w.seg + 1 == w.segments)
      store_state<KT>(S, a.s_out + head * a.Dk * a.Dv, a.Dk, a.Dv, w.col0 + col, col < w.cols, lane);
  } else if constexpr (WALK == kEnds) {
    const int64_t part = (w.part + w.seg) * a.H + w.h;
    if (w.move)
      keep_state<KT>(S, a.moves + part * a.Dk * a.move_pitch, a.Dk, a.move_pitch, w.col0 + 16 * wave, lane);
    else
      keep_state<KT>(S, a.ends + part * matrix, a.Dk, a.pitch, w.col0 + 16 * wave, lane);
  }
}

// The states that segments start from, along each split sequence: ends[i] +=
// moves[i] ends[i - 1], or backwards ends[i - 1] += moves[i]^T ends[i] (ends[i - 1] holds the
// gradient of the state that segment i starts from).  Grid tiles of 16 columns x H
// x B.  A step is a chain of loads, product and store, so its rows are spread over the
// waves, the state goes round through LDS, and the next step's matrix is on its
// way meanwhile.
template <int DKP, bool REVERSE>
__global__ void __launch_bounds__(256) delta_scan_kernel(DeltaArgs a) {
  constexpr int TILES = DKP / 64, STEPS = DKP / 32, kRow = DKP + 4;  // tiles of 16 rows a wave
  constexpr bool kAhead = DKP <= 128;  // (registers)
  __shared__ __attribute__((aligned(16))) float lds[16][kRow];
  const uint32_t tiles = (uint32_t)(a.pitch + 15) / 16u, state = blockIdx.x / tiles;
  const uint32_t b = scalar((int)divide(state, a.H, a.by_heads));
  const int h = (int)(state - b * a.H), col0 = 16 * (int)(blockIdx.x - state * tiles);
  const Span s = span_of(a, (int)b);
  const int segments = (s.len - 1) / (a.seg_chunks * C) + 1;
  if (segments <= 2) return;
  const int64_t part = a.offsets != nullptr ? s.first / (a.seg_chunks * C) : (int64_t)b * a.segments;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4, l = lane & 15;
  const int64_t matrix = (int64_t)a.Dk * a.pitch;
  // tile i of the wave: rows 16 (wave TILES + i) + l, columns 4 g .. + 3
  auto at = [&](int i) {
    const int row = 16 * (wave * TILES + i) + l, col = col0 + 4 * g;
    return row < a.Dk && col < a.pitch ? (uint32_t)(row * a.pitch + col) * 4u : kOutside;
  };
  auto end_of = [&](int seg) {
    return make_rsrc(a.ends + ((part + (REVERSE ? seg - 1 : seg)) * a.H + h) * matrix, (uint32_t)matrix * 4u);
  };
  u32x4 E[TILES];
  float M[TILES][STEPS][8];
  auto fetch_tile = [&](int seg, int i) {
    const __amdgpu_buffer_rsrc_t m = make_rsrc(a.moves + ((part + seg) * a.H + h) * a.Dk * a.move_pitch, (uint32_t)(a.Dk * a.move_pitch) * 4u);
    E[i] = __builtin_amdgcn_raw_buffer_load_b128(end_of(seg), at(i), 0, kPlain);
    const int row = 16 * (wave * TILES + i) + l;
#pragma unroll
    for (int y = 0; y < STEPS; ++y) {
      const int from = 32 * y + 8 * g;
      if constexpr (REVERSE) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          M[i][y][e] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(m, row < a.Dk && from + e < a.Dk ? (uint32_t)((from + e) * a.move_pitch + row) * 4u : kOutside, 0, kPlain));
      } else {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(m, row < a.Dk && from + 4 * u < a.move_pitch ? (uint32_t)(row * a.move_pitch + from + 4 * u) * 4u : kOutside, 0, kPlain);
#pragma unroll
          for (int e = 0; e < 4; ++e) M[i][y][4 * u + e] = __uint_as_float(v[e]);
        }
      }
    }
  };
  auto seg_of = [&](int i) { return REVERSE ? segments - 1 - i : i; };
  {
    const __amdgpu_buffer_rsrc_t first = end_of(REVERSE ? segments - 1 : 0);
    u32x4 S[TILES];
#pragma unroll
    for (int i = 0; i < TILES; ++i) S[i] = __builtin_amdgcn_raw_buffer_load_b128(first, at(i), 0, kPlain);
    if (kAhead)
#pragma unroll
      for (int i = 0; i < TILES; ++i) fetch_tile(seg_of(1), i);
#pragma unroll
    for (int i = 0; i < TILES; ++i)
#pragma unroll
      for (int r = 0; r < 4; ++r) lds[4 * g + r][16 * (wave * TILES + i) + l] = __uint_as_float(S[i][r]);
  }
  for (int i = 1; i + 1 < segments; ++i) {
    __syncthreads();
    b16x8 S[STEPS][kFull];
#pragma unroll
    for (int y = 0; y < STEPS; ++y) {
      float x[8];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const f32x4 v = *reinterpret_cast<const f32x4*>(&lds[l][32 * y + 8 * g + 4 * u]);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[4 * u + e] = v[e];
      }
      split_operand<kFull>(S[y], x);
    }
    f32x4 next[TILES];
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
      if (!kAhead) fetch_tile(seg_of(i), t);
      next[t] = __builtin_bit_cast(f32x4, E[t]);
#pragma unroll
      for (int y = 0; y < STEPS; ++y) {
        b16x8 B[kFull];
        split_operand<kFull>(B, M[t][y]);
        product(next[t], S[y], B);  // (columns x rows)
      }
    }
    if (kAhead && i + 2 < segments)
#pragma unroll
      for (int t = 0; t < TILES; ++t) fetch_tile(seg_of(i + 1), t);
    const __amdgpu_buffer_rsrc_t end = end_of(seg_of(i));
    __syncthreads();
#pragma unroll
    for (int t = 0; t < TILES; ++t) {
#pragma unroll
      for (int r = 0; r < 4; ++r) lds[4 * g + r][16 * (wave * TILES + t) + l] = next[t][r];
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, next[t]), end, at(t), 0, kPlain);
    }
  }
}

// Backwards: leaves w and the gradients of the states behind the chunks, and
// that of the initial state; or (ENDS) the gradients of the states that segments
// start from, by themselves.  Grid tiles x H x segments.
template <class E, int DKP, bool VEC, bool ENDS>
__global__ void __launch_bounds__(256, DKP == 256 ? 1 : 2) delta_reverse_kernel(DeltaArgs a) {
  typedef Shape<E, DKP, true> Sh;
  typedef typename E::raw raw;
  constexpr int IN = Sh::IN, KT = Sh::KT, GROUP = group_chunks<E, DKP>();
  extern __shared__ __attribute__((aligned(16))) char lds[];
  char *const kt = lds + Sh::kK, *const qt = lds + Sh::kQ, *const vt = lds + Sh::kV, *const mt = lds + Sh::kM,
              *const vecs = lds + Sh::kVecs;
  Where w;
  if (!where<ENDS>(a, a.tiles, a.by_tiles, w) || w.seg >= w.segments || (ENDS && w.seg == 0)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4, l = lane & 15;
  const int col = 16 * wave + l;
  const uint32_t qs = (uint32_t)a.q.token * (uint32_t)sizeof(raw), ks = (uint32_t)a.k.token * (uint32_t)sizeof(raw),
                 os = (uint32_t)a.o.token * (uint32_t)sizeof(raw);
  const raw* const q = static_cast<const raw*>(a.q.p) + base_of(a.q, a, w.s, w.b, w.h);
  const raw* const k = static_cast<const raw*>(a.k.p) + base_of(a.k, a, w.s, w.b, w.h);
  const raw* const o = static_cast<const raw*>(a.o.p) + base_of(a.o, a, w.s, w.b, w.h) + w.col0;
  Rows<E, C, DKP, 256, VEC> rq(qs, a.Dk, false), rk(ks, a.Dk, false);
  Rows<E, C, 64, 256, VEC> ro(os, w.cols, false);
  Block<true> block;
  static_assert(Sh::kVecs == Sh::kM + 16 * Block<true>::kUnits, "factors behind the matrices");
  auto fetch = [&](int c) {
    const int n = c < w.lo ? 0 : min(C, w.s.len - c * C);
    const int64_t t0 = n <= 0 ? 0 : (int64_t)c * C;
    rk.load(k, t0, n, ks, a.Dk, false);
    rq.load(q, t0, n, qs, a.Dk, false);
  };
  auto fetch_rest = [&](int c) {
    const int n = c < w.lo ? 0 : min(C, w.s.len - c * C);
    const int64_t t0 = n <= 0 ? 0 : (int64_t)c * C;
    ro.load(o, t0, n, os, w.cols, false);
    if (n > 0) block.load(a.blocks + ((w.chunk + c) * a.H + w.h) * kDeltaBlock);
  };
  fetch(w.hi - 1);
  fetch_rest(w.hi - 1);
  const size_t head = (size_t)w.b * a.H + w.h;
  const int64_t matrix = (int64_t)a.Dk * a.pitch;
  const bool kept = w.col0 + col < a.pitch, last = w.seg + 1 == w.segments;
  f32x4 R[KT];
  if (ENDS && !last)
    load_state<KT>(R, nullptr, a.Dk, a.Dv, 0, false, lane);
  else if (!ENDS && !last)
    load_state<KT>(R, a.ends + ((w.part + w.seg) * a.H + w.h) * matrix, a.Dk, a.pitch, w.col0 + col, col < w.cols, lane);
  else if (!ENDS && w.segments > 1 && a.ds_in != nullptr)
    load_state<KT>(R, a.firsts + (w.part * a.H + w.h) * matrix, a.Dk, a.pitch, w.col0 + col, col < w.cols, lane);
  else
    load_state<KT>(R, a.ds_in != nullptr ? a.ds_in + head * a.Dk * a.Dv : nullptr, a.Dk, a.Dv, w.col0 + col, col < w.cols, lane);
  if (ENDS && last && a.ds_in != nullptr)
    keep_state<KT>(R, a.firsts + (w.part * a.H + w.h) * matrix, a.Dk, a.pitch, w.col0 + 16 * wave, lane);

  for (int c = w.hi - 1; c >= w.lo; --c) {
    rk.store(kt);
    rq.store(qt);
    ro.store(vt);
    block.store(mt);
    __syncthreads();
    fetch(c - 1);
    if (!ENDS) {
      fetch_rest(c - 1);
      if (c % GROUP == GROUP - 1 || c + 1 == w.chunks)
        store_state<KT>(R, a.R + ((w.group + c / GROUP) * a.H + w.h) * matrix, a.Dk, a.pitch, w.col0 + col, kept, lane);
    }
    const float whole = *reinterpret_cast<const float*>(vecs + 4 * (kUp * C + C - 1));

    // K R
    const int rows = row_at<DKP>(l) ^ (g << 4);
    f32x4 x[2], u[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) x[t] = u[t] = f32x4(0.f);
#pragma unroll
    for (int s = 0; s < DKP / 32; ++s) {
      b16x8 A[kFull], K[2][IN];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int p = 0; p < IN; ++p) K[t][p] = read_row(kt, (rows ^ (64 * s)) + p * (C * DKP * 2) + t * (32 * DKP));
      state_operand<kFull>(A, R[2 * s], R[2 * s + 1]);
      state_products<IN, false>(x, u, K, K, A);
    }
    if (ENDS) fetch_rest(c - 1);
    // w = T'^T (P'^T dO + down beta K R)
    float y[8], f[8];
    b16x8 D[IN];
    read_values<E>(D, vt, wave, lane);
    {
      b16x8 P[2][kFull], T[2][kFull], Y[kFull];
#pragma unroll
      for (int t = 0; t < 2; ++t) read_transposed<kFull>(P[t], mt + kDeltaP, t, lane);
      products<kFull, IN, 2>(u, P, D);
      factors(f, vecs, kInto, lane);
#pragma unroll
      for (int t = 0; t < 2; ++t) read_transposed<kFull>(T[t], mt, t, lane);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = __builtin_fmaf(f[e], x[e / 4][e % 4], u[e / 4][e % 4]);
      split_operand<kFull>(Y, y);
      x[0] = x[1] = f32x4(0.f);
      products<kFull, kFull, 2>(x, T, Y);
    }
    if (!ENDS) {
      float* const to = a.w + (((w.group + c / GROUP) * a.H + w.h) * GROUP + c % GROUP) * C * a.pitch + w.col0 + col;
      if (kept)
#pragma unroll
        for (int e = 0; e < 8; ++e) to[(16 * (e / 4) + 4 * g + e % 4) * a.pitch] = x[e / 4][e % 4];
    }
    // R = up_C R + Q^T (scale up dO) - K^T (up w)
    b16x8 M[2][kFull];
    values_of(y, D);
    factors(f, vecs, kScaledUp, lane);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] *= f[e];
    split_operand<kFull>(M[0], y);
    factors(f, vecs, kUp, lane);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = -f[e] * x[e / 4][e % 4];
    split_operand<kFull>(M[1], y);
#pragma unroll
    for (int t = 0; t < KT; t += 2) {
      b16x8 K[2][IN], Q[2][IN];
      f32x4 z[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        read_keys<E, DKP>(Q[i], qt, lane, t + i);
        read_keys<E, DKP>(K[i], kt, lane, t + i);
        z[i] = R[t + i] * whole;
      }
      products<IN, kFull, 2>(z, Q, M[0]);
      products<IN, kFull, 2>(z, K, M[1]);
      R[t] = z[0];
      R[t + 1] = z[1];
    }
    __syncthreads();
  }
  if (ENDS)
    keep_state<KT>(R, a.ends + ((w.part + w.seg - 1) * a.H + w.h) * matrix, a.Dk, a.pitch, w.col0 + 16 * wave, lane);
  else if (a.ds_out != nullptr && w.seg == 0)
    store_state<KT>(R, a.ds_out + head * a.Dk * a.Dv, a.Dk, a.Dv, w.col0 + col, col < w.cols, lane);
}

// -- the gradients of a group of chunks ------------------------------------------------------------

// Tokens of a group: its formulas are a chunk's, of 64 tokens where LDS holds them:
// states and their gradients are then kept, and split, for every second chunk only.
// Nothing is moved across: reads of operands ahead would take the registers of the sums.
__device__ __forceinline__ void hold() { __builtin_amdgcn_sched_barrier(0); }

template <class E, int DKP>
struct GradShape {
  static constexpr int IN = Parts<E>::kIn, TC = group_chunks<E, DKP>() * C, TT = TC / 16;
  static constexpr int WAVES = delta_grad_waves(DKP), KT = DKP / 16 / WAVES;  // tiles of 16 rows of the state a wave
  static constexpr int kPart = 2 * TC * 64;         // a part of 64 columns of TC rows
  // k, then q; dO, x and w of 64 columns, then two matrices of scores, then the sums of the waves
  static constexpr int kK = 0, kA = 2 * TC * IN * DKP, kO = kA, kX = kO + IN * kPart, kW = kX + 3 * kPart,
                       kVecs = kW + 3 * kPart, kSums = kVecs + 4 * 4 * TC, kLds = kSums + 8 * TC;
  static constexpr int kScore = 3 * 128 * TC;  // bytes of a matrix of scores: rows of 128 bytes
  static_assert(2 * kScore <= kVecs - kA && WAVES * 16 * TC + 64 <= kVecs - kA, "overlays");
};
enum GradVec { kGUp, kGScaledUp, kGDown, kGBeta };

// Grid groups x H.  The columns of the state are taken 64 at a time; a wave has KT
// tiles of 16 of its rows.
template <class E, int DKP, bool VEC>
__global__ void __launch_bounds__(64 * delta_grad_waves(DKP), 2) delta_grad_kernel(DeltaArgs a) {
  typedef GradShape<E, DKP> Sh;
  typedef typename E::raw raw;
  constexpr int IN = Sh::IN, KT = Sh::KT, TC = Sh::TC, TT = Sh::TT, WAVES = Sh::WAVES, THREADS = 64 * WAVES;
  // tiles (i, j) of the scores: those with j <= i, then those above the diagonal that the products read
  constexpr bool kAhead = TC > C;  // one workgroup on a unit: its loads early
  constexpr int kTiles = TT * (TT + 1) / 2, kJobs = kTiles + TT / 2, kOwn = (kJobs + WAVES - 1) / WAVES;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  char *const kt = lds + Sh::kK, *const ot = lds + Sh::kO, *const xt = lds + Sh::kX, *const wt = lds + Sh::kW,
              *const scores = lds + Sh::kA;
  float* const vecs = reinterpret_cast<float*>(lds + Sh::kVecs);
  double* const sums = reinterpret_cast<double*>(lds + Sh::kSums);
  float* const dots = reinterpret_cast<float*>(lds + Sh::kA);  // [waves][4][TC], then <R, S> of each wave
  const uint32_t id = near(blockIdx.x, gridDim.x), slot = scalar((int)divide(id, a.H, a.by_heads));
  const int h = (int)(id - slot * a.H);
  int b, c;
  if (!group_of(a, slot, b, c)) return;
  const Span s = span_of(a, b);
  const int64_t t0 = (int64_t)c * TC;
  const int n = (int)max((int64_t)0, min((int64_t)TC, s.len - t0));
  const int all = a.lengths != nullptr ? (int)min((int64_t)TC, a.T - t0) : n;  // rows to write: padding as zeros
  if (all <= 0) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4, l = lane & 15;
  const int64_t at = (int64_t)slot * a.H + h;
  const int pitch = a.pitch;
  void* const dv = const_cast<void*>(a.dv.p);
  const int64_t dv0 = base_of(a.dv, a, s, b, h) + t0 * a.dv.token;
  if (n == 0) {
    for (int i = threadIdx.x; i < all * a.Dv; i += THREADS) static_cast<raw*>(dv)[dv0 + (i / a.Dv) * a.dv.token + i % a.Dv] = E::put(0.f);
  }

  const uint32_t qs = (uint32_t)a.q.token * (uint32_t)sizeof(raw), ks = (uint32_t)a.k.token * (uint32_t)sizeof(raw),
                 os = (uint32_t)a.o.token * (uint32_t)sizeof(raw);
  typedef Rows<E, TC, 64, THREADS, VEC> Values;
  typedef Rows<F32, TC, 64, THREADS, true> Wide;
  typedef Rows<E, TC, DKP, THREADS, VEC> Keys;
  Values ro(os, 64, false);
  Wide rx((uint32_t)pitch * 4u, 64, false), rw((uint32_t)pitch * 4u, 64, false);
  Keys rq(qs, a.Dk, false);
  const raw* const o = static_cast<const raw*>(a.o.p) + base_of(a.o, a, s, b, h);
  const float *const xs = a.x + at * TC * pitch, *const ws = a.w + at * TC * pitch;
  auto fetch = [&](int col) {
    const int m = col < a.Dv ? n : 0;
    const int64_t first = m == 0 ? 0 : t0;
    ro.whole = Values(os, a.Dv - col, false).whole;  // (the last columns are fewer)
    rx.whole = Wide((uint32_t)pitch * 4u, pitch - col, false).whole;
    rw.whole = rx.whole;
    ro.load(o + col, first, m, os, min(64, a.Dv - col), false);
    rx.load(xs + col, 0, m, (uint32_t)pitch * 4u, min(64, pitch - col), false);
    rw.load(ws + col, 0, m, (uint32_t)pitch * 4u, min(64, pitch - col), false);
  };
  f32x4 dq[KT][TT], row[KT][TT], cl[KT][TT], so[kOwn], sw[kOwn];
  float inner = 0.f;  // <R, S>
#pragma unroll
  for (int i = 0; i < KT; ++i)
#pragma unroll
    for (int t = 0; t < TT; ++t) dq[i][t] = row[i][t] = cl[i][t] = f32x4(0.f);
#pragma unroll
  for (int m = 0; m < kOwn; ++m) so[m] = sw[m] = f32x4(0.f);
  int ti[kOwn], tj[kOwn];
#pragma unroll
  for (int m = 0; m < kOwn; ++m) {
    const int job = wave + WAVES * m;
    ti[m] = job >= kTiles ? 2 * (job - kTiles) : job >= 6 ? 3 : job >= 3 ? 2 : job >= 1 ? 1 : 0;
    tj[m] = job >= kTiles ? ti[m] + 1 : job - ti[m] * (ti[m] + 1) / 2;
  }
  float sum[4][TT];  // of tokens 16 t + l: k.(down x R^T), q.dq, k.row, k.col
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int t = 0; t < TT; ++t) sum[i][t] = 0.f;
  if (n > 0) {
    fetch(0);
    {
      Keys rk(ks, a.Dk, false);
      rk.load(static_cast<const raw*>(a.k.p) + base_of(a.k, a, s, b, h), t0, n, ks, a.Dk, false);
      // the sums and factors of the group, from its chunks'
      if (threadIdx.x < TC) {
        const int t = threadIdx.x;
        const char* const block = a.blocks + ((first_chunk(a, s, b) + c * (TC / C)) * a.H + h) * kDeltaBlock;
        double G = reinterpret_cast<const double*>(block + kDeltaSums)[t < C ? t : C - 1], end = reinterpret_cast<const double*>(block + kDeltaSums)[C - 1];
        float beta = t < C ? reinterpret_cast<const float*>(block + kDeltaVec)[kBeta * C + t] : 0.f;
        if (TC > C && n > C) {
          const char* const second = block + (int64_t)a.H * kDeltaBlock;
          const double* const more = reinterpret_cast<const double*>(second + kDeltaSums);
          if (t >= C) {
            G += more[t - C];
            beta = reinterpret_cast<const float*>(second + kDeltaVec)[kBeta * C + t - C];
          }
          end += more[C - 1];
        }
        const float up = exp_sum(G);
        sums[t] = G;
        vecs[kGUp * TC + t] = up;
        vecs[kGScaledUp * TC + t] = a.scale * up;
        vecs[kGDown * TC + t] = exp_sum(end - G);
        vecs[kGBeta * TC + t] = beta;
      }
      rk.store(kt);
    }
    const __amdgpu_buffer_rsrc_t rS = make_rsrc(a.S + at * a.Dk * pitch, (uint32_t)(a.Dk * pitch) * 4u),
                                 rR = make_rsrc(a.R + at * a.Dk * pitch, (uint32_t)(a.Dk * pitch) * 4u);
    u32x4 fs[KT][2], fr[KT][2];
    auto fetch_states = [&](int col) {  // 32 columns
#pragma unroll
      for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int dk = 16 * (wave * KT + i) + l, d = col + 8 * g + 4 * u;
          const uint32_t from = d < pitch && dk < a.Dk ? (uint32_t)(dk * pitch + d) * 4u : kOutside;
          fs[i][u] = __builtin_amdgcn_raw_buffer_load_b128(rS, from, 0, kPlain);
          fr[i][u] = __builtin_amdgcn_raw_buffer_load_b128(rR, from, 0, kPlain);
        }
    };
    fetch_states(0);
    if (kAhead) rq.load(static_cast<const raw*>(a.q.p) + base_of(a.q, a, s, b, h), t0, n, qs, a.Dk, false);
    for (int col = 0; col < a.Dv; col += 64) {
      ro.store(ot);
      rx.store(xt);
      rw.store(wt);
      // dv, from the registers that w came in
#pragma unroll
      for (int i = 0; i < Wide::N; ++i) {
        const int v = (int)threadIdx.x + THREADS * i, r = v / 16, d = col + 4 * (v % 16);
        const u32x4 y = rw.v[i];
        const f32x4 z = {__uint_as_float(y[0]), __uint_as_float(y[1]), __uint_as_float(y[2]), __uint_as_float(y[3])};
        if (r < all) put4<E>(dv, dv0 + r * a.dv.token + d, r < n ? z : f32x4(0.f), a.Dv - d, false, (a.vec & 4) != 0);
      }
      __syncthreads();
      if (kAhead) fetch(col + 64);
#pragma unroll
      for (int st = 0; st < 2; ++st) {
        const int unit = row_at<64>(l) ^ (g << 4) ^ (64 * st);
#pragma unroll
        for (int i = 0; i < KT; ++i) {
          b16x8 A[kFull];
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            x[e] = __uint_as_float(fs[i][e / 4][e % 4]);
            inner = __builtin_fmaf(x[e], __uint_as_float(fr[i][e / 4][e % 4]), inner);
          }
          split_operand<kFull>(A, x);
          hold();
#pragma unroll
          for (int t = 0; t < TT; ++t) {
            b16x8 O[IN], W[kFull];
#pragma unroll
            for (int p = 0; p < IN; ++p) O[p] = read_row(ot, unit + p * Sh::kPart + t * (16 * 128));
#pragma unroll
            for (int p = 0; p < kFull; ++p) W[p] = read_row(wt, unit + p * Sh::kPart + t * (16 * 128));
#pragma unroll
            for (int z = kFull - 1; z >= 0; --z)
#pragma unroll
              for (int y = 0; y <= z; ++y) {
                row[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A[z - y], W[y], row[i][t], 0, 0, 0);
                if (y < IN) dq[i][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A[z - y], O[y < IN ? y : 0], dq[i][t], 0, 0, 0);
              }
            hold();
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(fr[i][e / 4][e % 4]);
          split_operand<kFull>(A, x);
          if (i == KT - 1) fetch_states(col + 32 * st + 32);
          hold();
#pragma unroll
          for (int t = 0; t < TT; t += 2) {
            b16x8 X[2][kFull];
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int p = 0; p < kFull; ++p) X[u][p] = read_row(xt, unit + p * Sh::kPart + (t + u) * (16 * 128));
#pragma unroll
            for (int z = kFull - 1; z >= 0; --z)
#pragma unroll
              for (int y = 0; y <= z; ++y)
#pragma unroll
                for (int u = 0; u < 2; ++u) cl[i][t + u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(A[z - y], X[u][y], cl[i][t + u], 0, 0, 0);
            hold();
          }
        }
#pragma unroll
        for (int m = 0; m < kOwn; ++m)
          if (wave + WAVES * m < kTiles) {
            b16x8 O[IN], X[kFull], W[kFull];
#pragma unroll
            for (int p = 0; p < IN; ++p) O[p] = read_row(ot, unit + p * Sh::kPart + ti[m] * (16 * 128));
#pragma unroll
            for (int p = 0; p < kFull; ++p) {
              X[p] = read_row(xt, unit + p * Sh::kPart + tj[m] * (16 * 128));
              W[p] = read_row(wt, unit + p * Sh::kPart + ti[m] * (16 * 128));
            }
            product(so[m], O, X);
            product(sw[m], W, X);
            hold();
          }
      }
      __syncthreads();
      if (!kAhead) fetch(col + 64);
    }
    if (!kAhead) rq.load(static_cast<const raw*>(a.q.p) + base_of(a.q, a, s, b, h), t0, n, qs, a.Dk, false);

    // The scores as matrices in parts: rows of tokens i, each with its factor of j (`by_rows`), or
    // rows of tokens j.  Which: Y, or -Z.
    float decays[kOwn][4];
#pragma unroll
    for (int m = 0; m < kOwn; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 16 * ti[m] + 4 * g + r, j = 16 * tj[m] + l;
        decays[m][r] = wave + WAVES * m < kTiles && j <= i ? exp_sum(sums[i] - sums[j]) : 0.f;
      }
    auto put_scores = [&](char* to, const f32x4 (&x)[kOwn], bool minus, bool by_rows) {
#pragma unroll
      for (int m = 0; m < kOwn; ++m) {
        if (wave + WAVES * m >= kJobs) break;
        const int j = 16 * tj[m] + l, i0 = 16 * ti[m] + 4 * g;
        float y[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int i = i0 + r;
          const float d = decays[m][r] * ((minus ? -1.f : a.scale) * (by_rows ? vecs[kGBeta * TC + j] : 1.f));
          y[r] = j < i || (!minus && j == i) ? x[m][r] * d : 0.f;
        }
        uint32_t words[kFull][2];
        split<kFull, 4>(y, words);
#pragma unroll
        for (int p = 0; p < kFull; ++p) {
          if (by_rows) {
#pragma unroll
            for (int r = 0; r < 4; ++r)
              *reinterpret_cast<uint16_t*>(to + p * (128 * TC) + (row_at<64>(i0 + r) ^ ((j >> 3) << 4)) + 2 * (j & 7)) = (uint16_t)(words[p][r / 2] >> (16 * (r % 2)));
          } else {
            *reinterpret_cast<u32x2*>(to + p * (128 * TC) + (row_at<64>(j) ^ ((i0 >> 3) << 4)) + 2 * (i0 & 7)) = u32x2{words[p][0], words[p][1]};
          }
        }
        hold();
      }
    };
    // acc[i][t] += keys^T scores for the wave's rows of the state; LOWER: scores by rows i (tokens j <= i), else by rows j.
    auto take = [&](f32x4 (&acc)[KT][TT], const char* m, bool lower) {
#pragma unroll
      for (int y = 0; y < TC / 32; ++y) {
        b16x8 K[KT][IN];
#pragma unroll
        for (int i = 0; i < KT; ++i) {
          const int base = row_at<DKP>(8 * g + (l >> 2)) ^ ((2 * (wave * KT + i) + ((l & 3) >> 1)) << 4);
#pragma unroll
          for (int p = 0; p < IN; ++p) {
            u32x2 half[2];
#pragma unroll
            for (int u = 0; u < 2; ++u)
              half[u] = read_columns(kt, (base ^ (16 * u)) + 8 * (l & 1) + p * (TC * DKP * 2) + (32 * y + 4 * u) * (2 * DKP));
            const uint32_t words[4] = {half[0][0], half[0][1], half[1][0], half[1][1]};
            K[i][p] = operand(words);
          }
        }
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          if (lower ? y > t / 2 : y < t / 2) continue;
          b16x8 M[kFull];
#pragma unroll
          for (int p = 0; p < kFull; ++p) M[p] = read_row(m, p * (128 * TC) + (row_at<64>(l) ^ (g << 4) ^ (64 * y)) + t * (16 * 128));
#pragma unroll
          for (int i = 0; i < KT; ++i) product(acc[i][t], K[i], M);
          hold();
        }
      }
    };
    // the values of keys at the accumulators' places: tokens 16 t + l, 4 rows of the state
    f32x4 keys[KT][TT];
    auto read_values_of_keys = [&]() {
      typedef __bf16 b16x4 __attribute__((ext_vector_type(4)));
#pragma unroll
      for (int i = 0; i < KT; ++i) {
        const int d0 = 16 * (wave * KT + i) + 4 * g;
#pragma unroll
        for (int t = 0; t < TT; ++t) {
          keys[i][t] = f32x4(0.f);
#pragma unroll
          for (int p = IN - 1; p >= 0; --p) {
            const b16x4 x = *reinterpret_cast<const b16x4*>(kt + (row_at<DKP>(l) ^ ((d0 >> 3) << 4)) + 2 * (d0 & 7) + p * (TC * DKP * 2) + t * (32 * DKP));
#pragma unroll
            for (int r = 0; r < 4; ++r) keys[i][t][r] += (float)x[r];
          }
        }
      }
    };
    auto dot = [&](float (&to)[TT], const f32x4 (&acc)[KT][TT]) {
#pragma unroll
      for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int t = 0; t < TT; ++t)
#pragma unroll
          for (int r = 0; r < 4; ++r) to[t] = __builtin_fmaf(keys[i][t][r], acc[i][t][r], to[t]);
      hold();
    };
    read_values_of_keys();
    hold();
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const float* const f = vecs + 16 * t + l;
#pragma unroll
      for (int i = 0; i < KT; ++i) {
        dq[i][t] *= f[kGScaledUp * TC];
        row[i][t] *= -f[kGUp * TC];
        cl[i][t] *= f[kGDown * TC];
      }
      hold();
    }
    dot(sum[0], cl);
    put_scores(scores, so, false, true);
    put_scores(scores + Sh::kScore, sw, true, true);
    __syncthreads();
    take(dq, scores, true);
    take(row, scores + Sh::kScore, true);
    dot(sum[2], row);
    __syncthreads();
    put_scores(scores, so, false, false);
    put_scores(scores + Sh::kScore, sw, true, false);
    __syncthreads();
    take(cl, scores + Sh::kScore, false);
    __syncthreads();
    rq.store(kt);
    __syncthreads();
    take(cl, scores, false);
    dot(sum[3], cl);
    read_values_of_keys();
    dot(sum[1], dq);
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int i = 0; i < KT; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) row[i][t][r] = __builtin_fmaf(vecs[kGBeta * TC + 16 * t + l], cl[i][t][r], row[i][t][r]);
    __syncthreads();  // the scores' place is the sums'
  }
#pragma unroll
  for (int i = 0; i < KT; ++i) {
    const int d0 = 16 * (wave * KT + i) + 4 * g;
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      const int token = 16 * t + l;
      if (token < all) {
        const bool in = token < n;
        const int64_t atq = base_of(a.dq, a, s, b, h) + (t0 + token) * a.dq.token + d0, atk = base_of(a.dk, a, s, b, h) + (t0 + token) * a.dk.token + d0;
        put4<E>(const_cast<void*>(a.dq.p), atq, in ? dq[i][t] : f32x4(0.f), a.Dk - d0, a.qk_f32 != 0, (a.vec & 8) != 0);
        put4<E>(const_cast<void*>(a.dk.p), atk, in ? row[i][t] : f32x4(0.f), a.Dk - d0, a.qk_f32 != 0, (a.vec & 8) != 0);
      }
    }
  }
  // the scalars' gradients
  if (n > 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        sum[i][t] += __shfl_xor(sum[i][t], 16);
        sum[i][t] += __shfl_xor(sum[i][t], 32);
        if (lane < 16) dots[(wave * 4 + i) * TC + 16 * t + l] = sum[i][t];
      }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) inner += __shfl_xor(inner, d);
    if (lane == 0) dots[WAVES * 4 * TC + wave] = inner;
  }
  __syncthreads();
  if (threadIdx.x < TC) {
    const int t = threadIdx.x;
    float dbeta = 0.f;
    double dg = 0.;
    if (n > 0) {
      float y[4], rs = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[i] = 0.f;
#pragma unroll
        for (int m = 0; m < WAVES; ++m) y[i] += dots[(m * 4 + i) * TC + t];
      }
#pragma unroll
      for (int m = 0; m < WAVES; ++m) rs += dots[WAVES * 4 * TC + m];
      const float beta = vecs[kGBeta * TC + t];
      dbeta = y[3];
      dg = t < n ? ((double)y[1] + (double)y[2]) - (double)(beta * dbeta) : 0.;
      double behind = t < n ? (double)(beta * y[0]) : 0.;
#pragma unroll
      for (int d = 1; d < TC; d *= 2) {
        behind += __shfl_xor(behind, d, TC);
        const double z = __shfl_down(dg, d, TC);
        if (t + d < TC) dg += z;
      }
      dg += behind + (double)vecs[kGUp * TC + TC - 1] * (double)rs;
      if (t == 0 && c == 0 && a.s_in == nullptr) dg = 0.;  // nothing there to decay before the first token
      // What a decay of 0 leaves does not depend on its logarithm.  (From sums that cancel, the
      // difference would be their rounding.  exp is 0 in fp32 below -103.98; NaN stays.)
      if (sums[t] - (t > 0 ? sums[t - 1] : 0.) < -104.) dg *= 0.;
    }
    if (t < all) {
      static_cast<float*>(const_cast<void*>(a.dbeta.p))[base_of(a.dbeta, a, s, b, h) + (t0 + t) * a.dbeta.token] = t < n ? dbeta : 0.f;
      if (a.dg.p != nullptr)
        static_cast<float*>(const_cast<void*>(a.dg.p))[base_of(a.dg, a, s, b, h) + (t0 + t) * a.dg.token] = t < n ? (float)dg : 0.f;
    }
  }
}

// -- launches of one element type ---------------------------------------------------------------------

template <class K>
hipError_t launch_kernel(K kernel, unsigned grid, int lds, const DeltaArgs& a, hipStream_t stream, int threads = 256) {
  const void* fn = reinterpret_cast<const void*>(kernel);
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  DeltaArgs args = a;
  void* list[] = {&args};
  return hipLaunchKernel(fn, dim3(grid), dim3(threads), list, (size_t)lds, stream);
}

template <class E, int DKP, bool VEC>
hipError_t launch_shape(const DeltaArgs& a, bool backward, hipStream_t stream) {
  const unsigned blocks = (unsigned)(a.slots * a.H), heads = (unsigned)((int64_t)a.B * a.H),
                 pieces = (unsigned)(a.units > 0 ? (int64_t)a.units * a.H : (int64_t)heads * a.segments);
  const unsigned columns = (unsigned)(a.pitch + 15) / 16;  // (tiles of the scan)
  constexpr int kLds = Shape<E, DKP, true>::kLds, kLdsNarrow = Shape<E, DKP, false>::kLds;
  const bool split = a.seg_slots > 0;
  hipError_t e = hipSuccess;
  // (448 chunks and heads of 128, fp32: 12.5 us in fours, 10 alone)
  if (blocks > 0) {
    const bool alone = blocks <= 1024;
    e = launch_kernel(delta_prepare_kernel<E, DKP, VEC>, alone ? blocks : (blocks + 3) / 4, 0, a, stream, alone ? 64 : 256);
  }
  if (e == hipSuccess && split) {
    e = launch_kernel(delta_forward_kernel<E, DKP, VEC, kEnds>, pieces * (a.tiles + a.move_tiles), kLdsNarrow, a, stream);
    if (e == hipSuccess && a.segments > 2) e = launch_kernel(delta_scan_kernel<DKP, false>, heads * columns, 0, a, stream);
  }
  if (e != hipSuccess) return e;
  if (!backward) return launch_kernel(delta_forward_kernel<E, DKP, VEC, kOutputs>, pieces * a.tiles, kLds, a, stream);
  if (blocks > 0) e = launch_kernel(delta_forward_kernel<E, DKP, VEC, kKeep>, pieces * a.tiles, kLdsNarrow, a, stream);
  if (e == hipSuccess && split) {
    e = launch_kernel(delta_reverse_kernel<E, DKP, VEC, true>, pieces * a.tiles, kLds, a, stream);
    if (e == hipSuccess && a.segments > 2) e = launch_kernel(delta_scan_kernel<DKP, true>, heads * columns, 0, a, stream);
  }
  if (e == hipSuccess) e = launch_kernel(delta_reverse_kernel<E, DKP, VEC, false>, pieces * a.tiles, kLds, a, stream);
  if (e == hipSuccess && blocks > 0) e = launch_kernel(delta_grad_kernel<E, DKP, VEC>, (unsigned)(a.group_slots * a.H), GradShape<E, DKP>::kLds, a, stream, 64 * GradShape<E, DKP>::WAVES);
  return e;
}

template <class E, bool VEC>
hipError_t launch_vec(const DeltaArgs& a, bool backward, hipStream_t stream) {
  if (a.dkp == 64) return launch_shape<E, 64, VEC>(a, backward, stream);
  if (a.dkp == 128) return launch_shape<E, 128, VEC>(a, backward, stream);
  return launch_shape<E, 256, VEC>(a, backward, stream);
}

template <class E>
hipError_t launch_type(const DeltaArgs& a, bool backward, hipStream_t stream) {
  return (a.vec & 1) != 0 ? launch_vec<E, true>(a, backward, stream) : launch_vec<E, false>(a, backward, stream);
}

}  // namespace delta
}  // namespace prnn
