// Linear attention in chunks of tokens on the matrix cores.
//
// With d = exp(log_decay), i, j tokens of one chunk of C and S the state the
// chunk starts from (p = 1; for a reversed job S comes decayed already, p = 0):
//
//   P_ij = kscale d^(i-j) q_i.k_j                (j <= i, else 0)
//   o_i  = oscale (sum_j P_ij v_j + d^(i+p) q_i S)
//   S   <- d^n S + kscale sum_j d^(n-p-j) k_j^T v_j   (n tokens in the chunk)
//
// Every exponent is >= 0, so nothing overflows that the recurrence does not.
//
// Work split.  One workgroup of 4 or 8 waves owns 16 columns a wave of one
// head's state and walks its segment of the sequence; each wave keeps its DKP x
// 16 of the state in registers as fp32 accumulators, for all its chunks.  q, k and v
// of a chunk are read once into LDS (the next chunk's loads are in flight
// meanwhile, held in registers), and the scores P, which all waves need, are
// computed once and exchanged through LDS.  The state never leaves the
// registers: an MFMA accumulator (lane l: rows 4 (l / 16) + r, column l % 16)
// has exactly the layout of an operand once the 32 rows of two accumulator
// tiles are dealt as row 8 (l / 16) + 4 tile + r, so S^T enters o^T = S^T q^T
// as its A operand without a shuffle, and the transposed operands k^T and v^T
// come from LDS with transposing reads (ds_read_b64_tr_b16) whose addresses
// deal the same rows.
//
// Precision.  Operands are split into bf16 parts, high part first, each the
// truncation of what is left (the last one rounded): bf16 is one part, fp16
// two, fp32 three, all exact.  Scores and state enter the output's products
// in 2 parts (2^-16) for 16-bit types and 3 (2^-24) for fp32; the decayed v
// enters the state, which is fp32 for every type, in 3 parts.  Products of
// parts below the last kept bit are left out.  bf16 parts have fp32's range,
// so large fp16 scores and states do not overflow.  Sums are fp32.
//
// Infinities and NaN.  A masked score is 0, and 0 times a later token's
// infinity would be NaN.  A wave whose output accumulators hold a value that
// is not finite therefore recomputes its columns of that chunk by the
// recurrence itself, token by token (attention_tokens), which is also what
// makes an overflow an infinity.  This costs finite inputs one multiply-add
// an output.
#pragma once

#include "device_common.h"
#include "sequence.h"

namespace prnn {
namespace attn {

typedef __bf16 b16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Parts of an input (kIn), of the scores and the state in the output's
// products (kOut), and of the decayed v in the state's (kState).
template <class E>
struct Parts;
template <>
struct Parts<BF16> {
  static constexpr int kIn = 1, kOut = 2, kState = 3;
};
template <>
struct Parts<F16> {
  static constexpr int kIn = 2, kOut = 2, kState = 3;
};
template <>
struct Parts<F32> {
  static constexpr int kIn = 3, kOut = 3, kState = 3;
};

// Tokens of a chunk.
template <class E, int DKP>
constexpr int chunk_tokens() {
  return 32;
}

// First row and number of tokens of sequence b (see prnnAttention_t).
struct Span {
  int64_t first;
  int len;
};
template <class A>
__device__ __forceinline__ Span span_of(const A& a, int b) {  // b the same in every lane
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
  s.first = __builtin_amdgcn_readfirstlane((int)s.first);  // rows fit 31 bits
  s.len = __builtin_amdgcn_readfirstlane(s.len);
  return s;
}

// Element offset of token 0 of sequence b, head h, of an operand.
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

// -- splitting into bf16 parts -----------------------------------------------------

__device__ __forceinline__ float cut(float x) { return __uint_as_float(__float_as_uint(x) & 0xffff0000u); }

// The high halves of two words, a in the low one.
__device__ __forceinline__ uint32_t pack_high(float a, float b) {
  return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}
__device__ __forceinline__ uint32_t pack_round(float a, float b) {
  typedef __bf16 b16x2 __attribute__((ext_vector_type(2)));
  const b16x2 v = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, v);
}

// out[part][i / 2] of N values.  An infinity becomes NaN.
template <int P, int N>
__device__ __forceinline__ void split(const float (&x)[N], uint32_t (&out)[P][N / 2]) {
  float r[N];
#pragma unroll
  for (int i = 0; i < N; ++i) r[i] = x[i];
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      if (p == P - 1) {
        out[p][i / 2] = pack_round(r[i], r[i + 1]);
      } else {
        out[p][i / 2] = pack_high(r[i], r[i + 1]);
        r[i] -= cut(r[i]);
        r[i + 1] -= cut(r[i + 1]);
      }
    }
}

__device__ __forceinline__ b16x8 operand(const uint32_t (&w)[4]) {
  const u32x4 v = {w[0], w[1], w[2], w[3]};
  return __builtin_bit_cast(b16x8, v);
}

// acc += x y over the parts' products that matter: i + j <= L.
template <int NX, int NY, int L>
__device__ __forceinline__ void products(f32x4& acc, const b16x8 (&x)[NX], const b16x8 (&y)[NY]) {
#pragma unroll
  for (int s = L; s >= 0; --s)  // small terms first
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const int j = s - i;
      if (j >= 0 && j < NY) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[i], y[j], acc, 0, 0, 0);
    }
}

// -- LDS tiles ------------------------------------------------------------------------

// A tile of rows of W bf16 in units of 16 bytes.  Unit u of a row lies at u ^
// swizzle(row): the 16 rows that a wave reads at one column, and the 4 rows x
// 4 units of a transposing read, then fall on 16 different units of the 64
// banks.  As bytes that is row_at(row) ^ 16 u, so one register per access
// pattern reaches every unit; row_at repeats every 16 rows, 32 W bytes on.
template <int W>
__device__ __forceinline__ int row_at(int row) {
  const int swizzle = W >= 128 ? ((row & 3) << 2) | ((row >> 2) & 3) : (((row >> 1) & 1) << 2) | ((row >> 2) & 3);
  return row * (2 * W) + (swizzle << 4);
}

// Keeps what depends on x from being computed ahead of a loop and held in
// registers through it.
__device__ __forceinline__ void keep(int& x) { asm volatile("" : "+v"(x)); }

__device__ __forceinline__ b16x8 read_row(const char* lds, int at) {
  return __builtin_bit_cast(b16x8, *reinterpret_cast<const u32x4*>(lds + at));
}
// Lane l of each 16 gives the address of 4 columns of row (l % 16) / 4 and
// gets the 4 rows of column l % 16.
__device__ __forceinline__ u32x2 read_columns(const char* lds, int at) {
  typedef __attribute__((address_space(3))) s16x4* ptr;
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((ptr)(lds + at)));
}

// -- global to LDS -----------------------------------------------------------------------

// Offset past every chunk's buffer: such a load returns zeros.
constexpr uint32_t kOutside = 0xFFFFFFE0u;

// The rows of one operand of a chunk: C rows of W columns, `cols` of which
// exist.  Thread t takes 16-byte vectors t, t + THREADS, ... of the tile.
template <class E, int C, int W, int THREADS, bool VEC>
struct Rows {
  typedef typename E::raw raw;
  static constexpr int kVec = 16 / (int)sizeof(raw), kPerRow = W / kVec;
  static constexpr int N = C * kPerRow >= THREADS ? C * kPerRow / THREADS : 1;  // (fewer vectors than threads: some idle)
  static constexpr int kStep = THREADS / kPerRow;  // rows from one vector of a thread to its next
  u32x4 v[N];

  // Rows [t0, t0 + n) of the sequence in memory order; reversed: token t0 + n
  // - 1 first.  p: token 0; stride in bytes.
  __device__ __forceinline__ void load(const void* p, int64_t t0, int n, uint32_t stride, int cols, bool reverse) {
    const __amdgpu_buffer_rsrc_t r = make_rsrc(static_cast<const char*>(p) + t0 * (int64_t)stride,
                                               (uint32_t)(n - 1) * stride + (uint32_t)cols * (uint32_t)sizeof(raw));
    int c = (int)threadIdx.x % kPerRow * kVec, row = (int)threadIdx.x / kPerRow;
    keep(c);
    keep(row);
#pragma unroll
    for (int i = 0; i < N; ++i, row += kStep) {
      // rows past n and columns past the operand's read zeros
      const uint32_t at = (uint32_t)(reverse ? n - 1 - row : row) * stride + (uint32_t)c * (uint32_t)sizeof(raw);
      if constexpr (VEC) {
        v[i] = __builtin_amdgcn_raw_buffer_load_b128(r, row < n && c < cols ? at : kOutside, 0, kPlain);
      } else {
        uint32_t e[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          const uint32_t o = row < n && c + j < cols ? at + j * (uint32_t)sizeof(raw) : kOutside;
          e[j] = sizeof(raw) == 4 ? __builtin_amdgcn_raw_buffer_load_b32(r, o, 0, kPlain)
                                  : (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(r, o, 0, kPlain);
        }
        if constexpr (sizeof(raw) == 4)
          v[i] = u32x4{e[0], e[1], e[2], e[3]};
        else
          v[i] = u32x4{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4 % kVec] | e[5 % kVec] << 16, e[6 % kVec] | e[7 % kVec] << 16};
      }
    }
  }

  // Into the tile's parts, C W bf16 each.
  __device__ __forceinline__ void store(char* lds) const {
    constexpr int P = Parts<E>::kIn;
    int c = (int)threadIdx.x % kPerRow, row = (int)threadIdx.x / kPerRow;
    keep(c);
    keep(row);
    if (C * kPerRow < THREADS && row >= C) return;
#pragma unroll
    for (int i = 0; i < N; ++i, row += kStep) {
      if constexpr (P == 1) {
        *reinterpret_cast<u32x4*>(lds + (row_at<W>(row) ^ (c << 4))) = v[i];
      } else if constexpr (P == 2) {
        typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
        const f16x8 h = __builtin_bit_cast(f16x8, v[i]);
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = (float)h[e];
        uint32_t w[2][4];
        split<2, 8>(x, w);
#pragma unroll
        for (int p = 0; p < 2; ++p)
          *reinterpret_cast<u32x4*>(lds + p * (C * W * 2) + (row_at<W>(row) ^ (c << 4))) =
              u32x4{w[p][0], w[p][1], w[p][2], w[p][3]};
      } else {
        float x[4];
        uint32_t w[3][2];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = __uint_as_float(v[i][e]);
        split<3, 4>(x, w);
#pragma unroll
        for (int p = 0; p < 3; ++p)
          *reinterpret_cast<u32x2*>(lds + p * (C * W * 2) + (row_at<W>(row) ^ (c / 2 << 4)) + 8 * (c & 1)) =
              u32x2{w[p][0], w[p][1]};
      }
    }
  }
};

// -- the workgroup's problem -----------------------------------------------------------------

template <class E, int DKP, int WAVES>
struct Shape {
  static constexpr int C = chunk_tokens<E, DKP>();
  static constexpr int DVT = 16 * WAVES;       // columns of a workgroup
  static constexpr int KT = DKP / 16;       // 16-row tiles of the state
  static constexpr int kTile = 2 * C * Parts<E>::kIn;  // bytes of a tile's column
  static constexpr int kQ = 0, kK = kTile * DKP, kV = 2 * kTile * DKP, kP = kV + kTile * DVT;
  static constexpr int kPRow = C + 8;       // bf16 of a row of scores: rows 16 bytes apart on the banks
  static constexpr int kPPart = 2 * C * kPRow;
  static constexpr int kW = kP + Parts<E>::kOut * kPPart;  // kscale d^(C - x), x = 0 .. C
  static constexpr int kLds = kW + 4 * (C + 4);
  // without scores: k and v only
  static constexpr int kLdsState = kTile * (DKP + DVT) + 4 * (C + 4);
};

// The state of one head in memory, as this lane's elements of it: element r of
// tile t lies at(t, r) bytes on, past the buffer where it does not exist.
struct StateAt {
  __amdgpu_buffer_rsrc_t rsrc;
  int rows, first, step;  // rows from the lane's first one on; its offset; bytes from row to row
  __device__ __forceinline__ StateAt(const float* p, const AttnJob& job, size_t head, int col, bool exists, int lane)
      : rsrc(make_rsrc(p + head * job.Dk * job.Dv, (uint32_t)(job.Dk * job.Dv) * 4u)),
        rows(exists ? job.Dk - 8 * (lane >> 4) : 0),
        first(4 * (8 * (lane >> 4) * job.s_row + col * job.s_col)),
        step(4 * job.s_row) {}
  __device__ __forceinline__ uint32_t at(int t, int r) const {
    const int row = 32 * (t / 2) + 4 * (t % 2) + r;
    return row < rows ? (uint32_t)(first + row * step) : kOutside;
  }
};

// What a workgroup works on.
struct Where {
  int b, h, col0, cols;  // the first of its columns of the state, and how many exist
  int seg;
  Span s;
  const char *q, *k, *v;  // token 0 (v: of its columns)
  int64_t o;              // element of token 0, first column
  float log_decay;
  float* states;          // the segment's states in register order, or nullptr
};

template <class E, int DKP, int WAVES>
__device__ __forceinline__ bool where(const AttnArgs& a, const AttnJob& job, int segments, Where& w) {
  typedef typename E::raw raw;
  constexpr int DVT = 16 * WAVES;
  int id = blockIdx.x;
  w.col0 = id % a.tiles * DVT;
  const int tile = id % a.tiles;
  id /= a.tiles;
  const int bh = id % (a.B * a.H);
  w.seg = id / (a.B * a.H);
  w.b = bh / a.H;
  w.h = bh % a.H;
  w.cols = job.Dv - w.col0;
  if (w.cols <= 0) return false;
  w.s = span_of(a, w.b);
  w.q = static_cast<const char*>(job.q.p) + base_of(job.q, a, w.s, w.b, w.h) * (int64_t)sizeof(raw);
  w.k = static_cast<const char*>(job.k.p) + base_of(job.k, a, w.s, w.b, w.h) * (int64_t)sizeof(raw);
  w.v = static_cast<const char*>(job.v.p) + (base_of(job.v, a, w.s, w.b, w.h) + w.col0) * (int64_t)sizeof(raw);
  w.o = base_of(job.o, a, w.s, w.b, w.h) + w.col0;
  w.log_decay = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(a.log_decay[w.h])));
  w.states = job.segments == nullptr
                 ? nullptr
                 : job.segments + (((int64_t)w.seg * a.B * a.H + bh) * a.tiles + tile) * (DKP * DVT);
  if (w.cols > DVT) w.cols = DVT;
  return true;
}

// Row and column (in the workgroup's columns) of the state that element r of
// accumulator tile (t, n) of a lane holds.
__device__ __forceinline__ int state_row(int t, int r, int lane) {
  return 32 * (t / 2) + 8 * (lane >> 4) + 4 * (t % 2) + r;
}
__device__ __forceinline__ int state_col(int wave, int lane) { return 16 * wave + (lane & 15); }

template <class E>
__device__ __forceinline__ void put_out(const AttnJob& job, int64_t at, float x) {
  if (job.o_f32)
    static_cast<float*>(const_cast<void*>(job.o.p))[at] = x;
  else
    static_cast<typename E::raw*>(const_cast<void*>(job.o.p))[at] = E::put(x);
}

// The recurrence over tokens [lo, hi) of the job's order for this wave's
// columns, straight from memory: S is updated and, with OUT, the rows of o
// written.  Slow; see the file comment.
template <class E, int DKP, bool OUT>
__device__ __forceinline__ void attention_tokens(const AttnJob& job, const Where& w, int lo, int hi, int col, int lane,
                                                 f32x4 (&S)[DKP / 16]) {
  typedef typename E::raw raw;
  const float d = decay_power(w.log_decay, 1);
  const float before = job.reverse ? 1.f : d, after = job.reverse ? d : 1.f;
  const int first = 8 * (lane >> 4);
#pragma nounroll
  for (int i = lo; i < hi; ++i) {
    const int64_t t = job.reverse ? w.s.len - 1 - i : i;
    const raw* q = reinterpret_cast<const raw*>(w.q) + t * job.q.token + first;
    const raw* k = reinterpret_cast<const raw*>(w.k) + t * job.k.token + first;
    const raw* v = reinterpret_cast<const raw*>(w.v) + t * job.v.token;
    const float vv = col < w.cols ? E::get(v[col]) : 0.f;
    float acc = 0.f;
    int rows = job.Dk - first;  // rows of the state from the lane's first one on
    keep(rows);
#pragma unroll
    for (int x = 0; x < DKP / 16; ++x)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 32 * (x / 2) + 4 * (x % 2) + r;
        if (row < rows) {
          S[x][r] = __builtin_fmaf(E::get(k[row]) * job.kscale, vv, S[x][r] * before);
          if (OUT) acc = __builtin_fmaf(E::get(q[row]), S[x][r], acc);
          S[x][r] *= after;
        }
      }
    if constexpr (OUT) {
      acc += __shfl_xor(acc, 16);
      acc += __shfl_xor(acc, 32);
      if (lane < 16 && col < w.cols) put_out<E>(job, w.o + t * job.o.token + col, acc * job.oscale);
    }
  }
}

// S += sum_j (kscale d^(n - p - j) v_j) k_j^T, S having been decayed; V: the
// chunk's columns of v as operands.  skip = C - n + p, weights from the table
// kscale d^(C - x).
template <class E, int DKP, int C>
__device__ __forceinline__ void update_state(f32x4 (&S)[DKP / 16], const b16x8 (&V)[C / 32][Parts<E>::kIn],
                                             const char* k, const float* weights, int skip) {
  constexpr int IN = Parts<E>::kIn, ST = Parts<E>::kState;
  const int lane = threadIdx.x & 63, g = lane >> 4, l = lane & 15;
  // row 8 g + l / 4, and 4 rows on: 8 W bytes and the swizzle's lowest bit
  int base = row_at<DKP>(8 * g + (l >> 2)) ^ ((l & 3) << 4);
  keep(base);
#pragma unroll
  for (int j = 0; j < C / 32; ++j) {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int at = skip + 32 * j + 8 * g + e;
      x[e] = 0.f;
#pragma unroll
      for (int p = IN - 1; p >= 0; --p) x[e] += (float)V[j][p][e];
      x[e] *= weights[at < C ? at : C];
    }
    uint32_t parts[ST][4];
    split<ST, 8>(x, parts);
    b16x8 D[ST];
#pragma unroll
    for (int p = 0; p < ST; ++p) D[p] = operand(parts[p]);
#pragma unroll
    for (int t = 0; t < DKP / 16; ++t) {
      b16x8 K[IN];
#pragma unroll
      for (int p = 0; p < IN; ++p) {
        u32x2 half[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          half[h] = read_columns(k, (base ^ (64 * (t / 2) + 16 * h)) + p * (C * DKP * 2) + (32 * j + 4 * h) * (2 * DKP) + 8 * (t % 2));
        const uint32_t words[4] = {half[0][0], half[0][1], half[1][0], half[1][1]};
        K[p] = operand(words);
      }
      products<IN, ST, 2>(S[t], K, D);
    }
  }
}

// The wave's columns of the chunk's v, as operands.
template <class E, int W, int C>
__device__ __forceinline__ void read_values(b16x8 (&V)[C / 32][Parts<E>::kIn], const char* v, int wave) {
  const int lane = threadIdx.x & 63, g = lane >> 4, l = lane & 15;
  int base = (row_at<W>(8 * g + (l >> 2)) ^ ((2 * wave + ((l & 3) >> 1)) << 4)) + 8 * (l & 1);
  keep(base);
#pragma unroll
  for (int j = 0; j < C / 32; ++j)
#pragma unroll
    for (int p = 0; p < Parts<E>::kIn; ++p) {
      u32x2 half[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        half[h] = read_columns(v, (base ^ (16 * h)) + p * (C * W * 2) + (32 * j + 4 * h) * (2 * W));
      const uint32_t words[4] = {half[0][0], half[0][1], half[1][0], half[1][1]};
      V[j][p] = operand(words);
    }
}

// NaN from the first value on that is not finite, 0 until then.
template <int N>
__device__ __forceinline__ void watch(float& z, const f32x4 (&x)[N]) {
#pragma unroll
  for (int t = 0; t < N; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) z = __builtin_fmaf(x[t][r], 0.f, z);
}

// The state a segment starts from.
template <int DKP>
__device__ __forceinline__ void first_state(f32x4 (&S)[DKP / 16], const AttnJob& job, const Where& w, size_t head,
                                            int col, int wave, int lane) {
  constexpr int KT = DKP / 16;
  if (w.states != nullptr) {
#pragma unroll
    for (int t = 0; t < KT; ++t) S[t] = reinterpret_cast<const f32x4*>(w.states)[(wave * KT + t) * 64 + lane];
  } else if (job.s_in != nullptr) {
    const StateAt x(job.s_in, job, head, w.col0 + col, col < w.cols, lane);
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        S[t][r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(x.rsrc, x.at(t, r), 0, kPlain));
  } else {
#pragma unroll
    for (int t = 0; t < KT; ++t) S[t] = f32x4(0.f);
  }
}
template <int DKP>
__device__ __forceinline__ void last_state(const f32x4 (&S)[DKP / 16], const AttnJob& job, const Where& w, size_t head,
                                           int col, int lane) {
  const StateAt x(job.s_out, job, head, w.col0 + col, col < w.cols, lane);
#pragma unroll
  for (int t = 0; t < DKP / 16; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[t][r]), x.rsrc, x.at(t, r), 0, kPlain);
}

// The state that tokens of each segment but the last leave by themselves:
// grid tiles x B H x (segments - 1), jobs.
template <class E, int DKP, int WAVES, bool VEC>
__global__ void __launch_bounds__(64 * WAVES, DKP == 256 ? 2 : WAVES / 2) attention_state_kernel(AttnArgs a) {
  typedef Shape<E, DKP, WAVES> Sh;
  constexpr int C = Sh::C;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  char *const kt = lds, *const vt = lds + Sh::kTile * DKP;
  float* const weights = reinterpret_cast<float*>(lds + Sh::kTile * (DKP + Sh::DVT));
  const AttnJob& job = a.job[blockIdx.y];
  Where w;
  if (!where<E, DKP, WAVES>(a, job, a.segments, w)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lo = w.seg * a.seg_tokens, hi = min(w.s.len, lo + a.seg_tokens);
  if ((int)threadIdx.x <= C) weights[threadIdx.x] = job.kscale * decay_power(w.log_decay, C - (int)threadIdx.x);
  const float decay = decay_power(w.log_decay, C);
  const int p = job.reverse ? 0 : 1;
  const uint32_t ks = (uint32_t)job.k.token * (uint32_t)sizeof(typename E::raw),
                 vs = (uint32_t)job.v.token * (uint32_t)sizeof(typename E::raw);

  f32x4 S[Sh::KT];
#pragma unroll
  for (int t = 0; t < Sh::KT; ++t) S[t] = f32x4(0.f);
  Rows<E, C, DKP, 64 * WAVES, VEC> rk;
  Rows<E, C, Sh::DVT, 64 * WAVES, VEC> rv;
  auto fetch = [&](int i) {
    const int n = min(C, hi - i);
    const int64_t t0 = job.reverse ? w.s.len - i - n : i;
    rk.load(w.k, t0, n, ks, job.Dk, job.reverse);
    rv.load(w.v, t0, n, vs, w.cols, job.reverse);
  };
  if (lo < hi) fetch(lo);
  for (int i = lo; i < hi; i += C) {
    const int n = min(C, hi - i);
    rk.store(kt);
    rv.store(vt);
    __syncthreads();
    if (i + C < hi) fetch(i + C);
    b16x8 V[C / 32][Parts<E>::kIn];
    read_values<E, Sh::DVT, C>(V, vt, wave);
    const float dn = n == C ? decay : decay_power(w.log_decay, n);
#pragma unroll
    for (int t = 0; t < Sh::KT; ++t) S[t] *= dn;
    update_state<E, DKP, C>(S, V, kt, weights, C - n + p);
    __syncthreads();
  }
  float z = 0.f;
  watch(z, S);
  if (wave_any(z != 0.f)) {
#pragma unroll
    for (int t = 0; t < Sh::KT; ++t) S[t] = f32x4(0.f);
    attention_tokens<E, DKP, false>(job, w, lo, hi, 16 * wave + (lane & 15), lane, S);
  }
#pragma unroll
  for (int t = 0; t < Sh::KT; ++t) reinterpret_cast<f32x4*>(w.states)[(wave * Sh::KT + t) * 64 + lane] = S[t];
}

// Turns the segments' own states into the states they start from: one thread
// per element.  grid: tiles x B H x (DKP DVT / 256) workgroups, jobs.
template <int DKP, int WAVES>
__global__ void __launch_bounds__(256) attention_scan_kernel(AttnArgs a) {
  constexpr int DVT = 16 * WAVES, KT = DKP / 16, kBlocks = DKP * DVT / 256;
  const AttnJob& job = a.job[blockIdx.y];
  const int part = blockIdx.x % kBlocks, id = blockIdx.x / kBlocks, tile = id % a.tiles, bh = id / a.tiles;
  const int b = bh / a.H, h = bh % a.H;
  if (tile * DVT >= job.Dv) return;
  const Span s = span_of(a, b);
  const int x = part * 256 + (int)threadIdx.x;  // element in register order
  const int r = x & 3, lane = (x >> 2) & 63, t = (x >> 8) % KT, wave = (x >> 8) / KT;
  const int row = state_row(t, r, lane), col = tile * DVT + state_col(wave, lane);
  float S = job.s_in != nullptr && row < job.Dk && col < job.Dv
                ? job.s_in[(size_t)bh * job.Dk * job.Dv + (size_t)row * job.s_row + (size_t)col * job.s_col]
                : 0.f;
  float* p = job.segments + ((int64_t)bh * a.tiles + tile) * (DKP * DVT) + x;
  const int64_t step = (int64_t)a.B * a.H * a.tiles * (DKP * DVT);
  for (int seg = 0; seg < a.segments; ++seg, p += step) {
    const float own = seg + 1 < a.segments ? *p : 0.f;
    *p = S;
    const int tokens = max(0, min(s.len - seg * a.seg_tokens, a.seg_tokens));
    S = tokens > 0 ? __builtin_fmaf(S, decay_power(a.log_decay[h], tokens), own) : S;
  }
}

// The attention: grid tiles x B H x segments, jobs.
template <class E, int DKP, int WAVES, bool VEC>
__global__ void __launch_bounds__(64 * WAVES, DKP == 256 ? 2 : WAVES / 2) attention_chunk_kernel(AttnArgs a) {
  typedef Shape<E, DKP, WAVES> Sh;
  typedef typename E::raw raw;
  constexpr int C = Sh::C, IT = C / 16, IN = Parts<E>::kIn, OUT = Parts<E>::kOut;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  char *const qt = lds + Sh::kQ, *const kt = lds + Sh::kK, *const vt = lds + Sh::kV, *const pt = lds + Sh::kP;
  float* const weights = reinterpret_cast<float*>(lds + Sh::kW);
  const AttnJob& job = a.job[blockIdx.y];
  Where w;
  if (!where<E, DKP, WAVES>(a, job, a.segments, w)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4, l = lane & 15;
  const int lo = w.seg * a.seg_tokens, hi = min(w.s.len, lo + a.seg_tokens);
  const int p = job.reverse ? 0 : 1;
  const bool reverse = job.reverse != 0;

  // rows of padding are zeros
  if (a.lengths != nullptr) {
    const int64_t end = min((int64_t)a.T, (int64_t)lo + a.seg_tokens);
    for (int64_t t = max(w.s.len, lo); t < end; ++t)
      if ((int)threadIdx.x < w.cols) put_out<E>(job, w.o + t * job.o.token + threadIdx.x, 0.f);
  }
  const bool last = w.seg == (w.s.len > 0 ? (w.s.len - 1) / a.seg_tokens : 0);
  if (lo >= hi && !(last && job.s_out != nullptr)) return;

  if ((int)threadIdx.x <= C) weights[threadIdx.x] = job.kscale * decay_power(w.log_decay, C - (int)threadIdx.x);
  // Score tiles above the diagonal that the products read: zero throughout.
  for (int x = threadIdx.x; x < OUT * Sh::kPPart / 4; x += 64 * WAVES) reinterpret_cast<uint32_t*>(pt)[x] = 0u;
  const float d16 = decay_power(w.log_decay, 16), decay = decay_power(w.log_decay, C);
  float from_state = decay_power(w.log_decay, l + p) * job.oscale;  // of i = l

  f32x4 S[Sh::KT];
  const size_t head = (size_t)w.b * a.H + w.h;
  const int col = 16 * wave + l;  // of the workgroup's columns: this lane's
  first_state<DKP>(S, job, w, head, col, wave, lane);
  float z = 0.f;

  const uint32_t qs = (uint32_t)job.q.token * (uint32_t)sizeof(raw), ks = (uint32_t)job.k.token * (uint32_t)sizeof(raw),
                 vs = (uint32_t)job.v.token * (uint32_t)sizeof(raw);
  Rows<E, C, DKP, 64 * WAVES, VEC> rq, rk;
  Rows<E, C, Sh::DVT, 64 * WAVES, VEC> rv;
  auto fetch = [&](int i) {
    const int n = min(C, hi - i);
    const int64_t t0 = reverse ? w.s.len - i - n : i;
    rq.load(w.q, t0, n, qs, job.Dk, reverse);
    rk.load(w.k, t0, n, ks, job.Dk, reverse);
    rv.load(w.v, t0, n, vs, w.cols, reverse);
  };
  if (lo < hi) fetch(lo);
  for (int i0 = lo; i0 < hi; i0 += C) {
    const int n = min(C, hi - i0);
    rq.store(qt);
    rk.store(kt);
    rv.store(vt);
    __syncthreads();
    if (i0 + C < hi) fetch(i0 + C);

    int rows = row_at<DKP>(l) ^ (g << 4);  // row l of a tile of 16, unit g
    keep(rows);

    // Scores, as P^T = k q^T, so that a lane has 4 tokens j of one i: the
    // tiles on and below the diagonal, dealt to the waves.
#pragma nounroll
    for (int x = wave; x < IT * (IT + 1) / 2; x += WAVES) {
      const int ti = x < 1 ? 0 : x < 3 ? 1 : x < 6 ? 2 : 3, tj = x - ti * (ti + 1) / 2;
      f32x4 acc = f32x4(0.f);
      const int qa = ti * (32 * DKP), ka = tj * (32 * DKP);
#pragma unroll
      for (int s = 0; s < DKP / 32; ++s) {
        b16x8 Q[IN], K[IN];
#pragma unroll
        for (int c = 0; c < IN; ++c) {
          Q[c] = read_row(qt, qa + (rows ^ (64 * s)) + c * (C * DKP * 2));
          K[c] = read_row(kt, ka + (rows ^ (64 * s)) + c * (C * DKP * 2));
        }
        products<IN, IN, IN - 1>(acc, K, Q);
      }
      float f[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int e = 16 * (ti - tj) + l - 4 * g - r;  // i - j
        f[r] = e >= 0 ? acc[r] * weights[C - max(e, 0)] : 0.f;  // a masked score is 0 whatever the product is
      }
      uint32_t words[OUT][2];
      split<OUT, 4>(f, words);
#pragma unroll
      for (int c = 0; c < OUT; ++c)
        *reinterpret_cast<u32x2*>(pt + c * Sh::kPPart + 2 * ((16 * ti + l) * Sh::kPRow + 16 * tj + 4 * g)) =
            u32x2{words[c][0], words[c][1]};
    }

    // o^T = S^T q^T, then times d^(i + p)
    f32x4 O[IT];
#pragma unroll
    for (int t = 0; t < IT; ++t) O[t] = f32x4(0.f);
#pragma unroll
    for (int s = 0; s < DKP / 32; ++s) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = S[2 * s + e / 4][e % 4];
      uint32_t words[OUT][4];
      split<OUT, 8>(x, words);
      b16x8 A[OUT];
#pragma unroll
      for (int c = 0; c < OUT; ++c) A[c] = operand(words[c]);
#pragma unroll
      for (int t = 0; t < IT; ++t) {
        b16x8 Q[IN];
#pragma unroll
        for (int c = 0; c < IN; ++c) Q[c] = read_row(qt, (rows ^ (64 * s)) + c * (C * DKP * 2) + t * (32 * DKP));
        products<OUT, IN, OUT - 1>(O[t], A, Q);
      }
    }
    float f = from_state;
#pragma unroll
    for (int t = 0; t < IT; ++t, f *= d16) O[t] *= f;
    __syncthreads();  // the scores are in LDS

    // o^T += oscale v^T P^T
    b16x8 V[C / 32][IN];
    read_values<E, Sh::DVT, C>(V, vt, wave);
#pragma unroll
    for (int t = 0; t < IT; ++t) {
      f32x4 I = f32x4(0.f);
#pragma unroll
      for (int j = 0; j <= t / 2; ++j) {
        b16x8 P[OUT];
#pragma unroll
        for (int c = 0; c < OUT; ++c)
          P[c] = read_row(pt, c * Sh::kPPart + 2 * ((16 * t + l) * Sh::kPRow + 32 * j + 8 * g));
        products<IN, OUT, OUT - 1>(I, V[j], P);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) O[t][r] = __builtin_fmaf(I[r], job.oscale, O[t][r]);
    }

    watch(z, O);
    {
      // A lane has 4 neighbouring columns of token 16 t + l.
      const bool wide = job.o_f32 || E::id == PRNN_DATA_FLOAT;
      const int size = wide ? 4 : 2, stride = (int)job.o.token * size;
      const int64_t t0 = reverse ? w.s.len - i0 - n : i0;
      const __amdgpu_buffer_rsrc_t out =
          make_rsrc(static_cast<const char*>(job.o.p) + (w.o + t0 * job.o.token) * size,
                    (uint32_t)(n - 1) * (uint32_t)stride + (uint32_t)(w.cols * size));
      int c0 = 16 * wave + 4 * g, row = l;
      keep(c0);
      keep(row);
#pragma unroll
      for (int t = 0; t < IT; ++t, row += 16) {
        const uint32_t at = (uint32_t)(reverse ? n - 1 - row : row) * (uint32_t)stride + (uint32_t)(c0 * size);
        if (!job.o_vec) {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const uint32_t to = row < n && c0 + r < w.cols ? at + r * size : kOutside;
            if (wide)
              __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(O[t][r]), out, to, 0, kPlain);
            else if constexpr (sizeof(raw) == 2)
              __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, E::put(O[t][r])), out, to, 0, kPlain);
          }
        } else {
          const uint32_t to = row < n && c0 < w.cols ? at : kOutside;
          if (wide) {
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, O[t]), out, to, 0, kPlain);
          } else {
            typedef raw vec __attribute__((ext_vector_type(4)));
            const vec x = {E::put(O[t][0]), E::put(O[t][1]), E::put(O[t][2]), E::put(O[t][3])};
            if constexpr (sizeof(raw) == 2) __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, x), out, to, 0, kPlain);
          }
        }
      }
      const float dn = n == C ? decay : decay_power(w.log_decay, n);
#pragma unroll
      for (int t = 0; t < Sh::KT; ++t) S[t] *= dn;
      update_state<E, DKP, C>(S, V, kt, weights, C - n + p);
    }
    __syncthreads();  // before the next chunk's tiles
  }
  watch(z, S);
  const bool ends = last && job.s_out != nullptr;
  if (!wave_any(z != 0.f)) {
    if (ends) last_state<DKP>(S, job, w, head, col, lane);
    return;
  }
  first_state<DKP>(S, job, w, head, col, wave, lane);
  attention_tokens<E, DKP, true>(job, w, lo, hi, col, lane, S);
  if (ends) last_state<DKP>(S, job, w, head, col, lane);
}

// -- launches of one element type --------------------------------------------------------------

// A kernel with more than 64 KiB of dynamic LDS.
template <class K>
hipError_t launch_wide(K kernel, dim3 grid, int threads, int lds, const AttnArgs& a, hipStream_t stream) {
  const void* fn = reinterpret_cast<const void*>(kernel);
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(fn, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
  }
  AttnArgs args = a;
  void* list[] = {&args};
  return hipLaunchKernel(fn, grid, dim3(threads), list, (size_t)lds, stream);
}

template <class E, int DKP, int WAVES, bool VEC>
hipError_t launch_shape(const AttnArgs& a, hipStream_t stream) {
  typedef Shape<E, DKP, WAVES> Sh;
  const unsigned states = (unsigned)a.tiles * a.B * a.H;
  if (a.segments > 1) {
    hipError_t e = launch_wide(attention_state_kernel<E, DKP, WAVES, VEC>, dim3(states * (a.segments - 1), a.jobs),
                               64 * WAVES, Sh::kLdsState, a, stream);
    if (e != hipSuccess) return e;
    e = launch_wide(attention_scan_kernel<DKP, WAVES>, dim3(states * (DKP * Sh::DVT / 256), a.jobs), 256, 0, a, stream);
    if (e != hipSuccess) return e;
  }
  return launch_wide(attention_chunk_kernel<E, DKP, WAVES, VEC>, dim3(states * a.segments, a.jobs), 64 * WAVES, Sh::kLds,
                     a, stream);
}

template <class E, bool VEC>
hipError_t launch_vec(const AttnArgs& a, hipStream_t stream) {
  if (a.dkp == 64) return a.waves == 4 ? launch_shape<E, 64, 4, VEC>(a, stream) : launch_shape<E, 64, 8, VEC>(a, stream);
  if (a.dkp == 128) return a.waves == 4 ? launch_shape<E, 128, 4, VEC>(a, stream) : launch_shape<E, 128, 8, VEC>(a, stream);
  return a.waves == 4 ? launch_shape<E, 256, 4, VEC>(a, stream) : launch_shape<E, 256, 8, VEC>(a, stream);
}

template <class E>
hipError_t launch_type(const AttnArgs& a, hipStream_t stream) {
  return a.vec ? launch_vec<E, true>(a, stream) : launch_vec<E, false>(a, stream);
}

}  // namespace attn
}  // namespace prnn
