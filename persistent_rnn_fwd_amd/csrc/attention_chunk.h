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
// Work split.  One workgroup of 4 waves owns 16 NT columns a wave (NT 1 or 2)
// of one head's state and walks its segment of the sequence; each wave keeps its
// DKP x 16 NT of the state in registers as fp32 accumulators, for all its chunks.
// q, k and v of a chunk are read once into LDS (the next chunk's loads are in
// flight meanwhile, held in registers), and the scores P, which all waves need,
// are computed once and exchanged through LDS.  The state never leaves the
// registers: an MFMA accumulator (lane l: rows 4 (l / 16) + r, column l % 16)
// has exactly the layout of an operand once the 32 rows of two accumulator
// tiles are dealt as row 8 (l / 16) + 4 tile + r, so S^T enters o^T = S^T q^T
// as its A operand without a shuffle, and the transposed operands k^T and v^T
// come from LDS with transposing reads (ds_read_b64_tr_b16) whose addresses
// deal the same rows.  32 rows at a time enter the output's products and then
// take the chunk's tokens, so that two independent groups of products are in
// hand.  NT = 2 halves the reads of q and k a product needs, and is taken where
// its workgroups fill the chip; a chunk is 64 tokens where registers and LDS
// allow, which halves the splitting and scaling of the state a token.
//
// Split sequences.  Where the heads do not fill the chip, segments of a sequence
// run side by side: a first kernel leaves each segment's own end state (k and v
// read once more), from 9 segments on a second one adds them up along the
// sequence (fewer are added by whoever needs them), and the main kernel starts
// each segment from its sum.
//
// What bounds it.  Large calls in 16 bits: what they move, which is more than they
// have to.  k and v are read once more for the segments' states, the three jobs of
// a backward pass read nine operands where four exist, and o's rows are written
// in pieces of 64 bytes that cost 30 to 38 % more than o.  Measured, operands not
// in the caches: 32768 bf16 tokens of 32 heads of 128, 1.79 GB moved (1.07 needed),
// 437 us (4.1 TB/s); backward of 8 x 2048 tokens of 16 bf16 heads of 128, 844 MB
// moved (470 needed), 247 us (3.4 TB/s): there the products are in issue for 38 %
// of the time as well, and half the units have two workgroups, half one.  fp32: the
// issue of its six products a product and of the splitting, 5.3 us a chunk of 32
// tokens alone on a unit.
// Small calls: launches and first loads, 3 us a kernel before its first product.
//
// Precision.  Operands are split into bf16 parts, high part first, each the
// truncation of what is left (the last one rounded): bf16 is one part, fp16
// two, fp32 three, all exact.  What is fp32 between the products (the decayed
// scores, the state, the decayed v that enters it) is three parts for every
// type, so it keeps fp32's 24 bits.  Products of parts whose orders add up to 3
// or more are left out: at most 2^-21 of the product, 2^-25 on average, where
// both operands have them (a bf16 operand has one part, so none are missing, and
// fp16 scores have all four).  Two parts between the products of 16-bit types
// would take 204 us instead of 247 for the backward of 8 x 2048 tokens of 16 bf16
// heads of 128, and 409 instead of 437 for 32768 tokens of 32, but where terms
// cancel the result is off by up to 2^-17 of them, and 2^-14 for fp16 scores.
// bf16 parts have fp32's range, so large fp16 scores and states do not overflow.
// Sums are fp32.
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

// Parts of an input, and of an fp32 value.
template <class E>
struct Parts;
template <>
struct Parts<BF16> {
  static constexpr int kIn = 1;
};
template <>
struct Parts<F16> {
  static constexpr int kIn = 2;
};
template <>
struct Parts<F32> {
  static constexpr int kIn = 3;
};
constexpr int kFull = 3;

// Tokens of a chunk.  64 halves what a token pays for splitting and scaling
// the state; the parts of the other types, and 256 rows, leave LDS and
// registers for 32.
template <class E, int DKP>
constexpr int chunk_tokens() {
  return E::id == PRNN_DATA_BFLOAT && DKP <= 128 ? 64 : 32;
}

// n / d, with inverse_of(d): the estimate is right or one less.
__device__ __forceinline__ uint32_t divide(uint32_t n, uint32_t d, uint32_t inverse) {
  const uint32_t q = __umulhi(n, inverse);
  return n - q * d >= d ? q + 1 : q;
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
  return (a.offsets != nullptr ? s.first * x.token : (int64_t)b * x.batch) + (int64_t)divide((uint32_t)h, (uint32_t)x.group, x.inverse) * x.head;
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

// A value that is the same in every lane, in a scalar register.
__device__ __forceinline__ float uniform(float x) {
  return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(x)));
}

// A state carried over many tokens at once, S d^n + own, with whole = d^n and one =
// d.  The recurrence keeps an infinity, and a zero, for any number of tokens, where
// d^n may have become 0 or infinity and the product NaN: those take one token's d.
__device__ __forceinline__ float carried(float S, float own, float whole, float one) {
  return __builtin_fmaf(S, S == 0.f || __builtin_isinf(S) ? one : whole, own);
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

// acc[m] += x y[m] over the parts' products that matter, i + j < 3, the
// accumulators in turn.
template <int NX, int NY, int M>
__device__ __forceinline__ void products(f32x4 (&acc)[M], const b16x8 (&x)[NX], const b16x8 (&y)[M][NY]) {
#pragma unroll
  for (int s = kFull - 1; s >= 0; --s)  // small terms first
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const int j = s - i;
      if (j < 0 || j >= NY) continue;
#pragma unroll
      for (int m = 0; m < M; ++m) acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[i], y[m][j], acc[m], 0, 0, 0);
    }
}
// ... and acc[m] += x[m] y.
template <int NX, int NY, int M>
__device__ __forceinline__ void products(f32x4 (&acc)[M], const b16x8 (&x)[M][NX], const b16x8 (&y)[NY]) {
#pragma unroll
  for (int s = kFull - 1; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const int j = s - i;
      if (j < 0 || j >= NY) continue;
#pragma unroll
      for (int m = 0; m < M; ++m) acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x[m][i], y[j], acc[m], 0, 0, 0);
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

// An offset past every chunk's buffer, also after a chunk's rows (below 2^30
// bytes) are added to it or taken from it: loads there return zeros and stores
// do nothing.
constexpr uint32_t kOutside = 0x80000000u;

// The rows of one operand of a chunk: C rows of W columns, `cols` of which
// exist.  Thread t takes 16-byte vectors t, t + THREADS, ... of the tile.
template <class E, int C, int W, int THREADS, bool VEC>
struct Rows {
  typedef typename E::raw raw;
  static constexpr int kVec = 16 / (int)sizeof(raw), kPerRow = W / kVec;
  static constexpr int N = C * kPerRow >= THREADS ? C * kPerRow / THREADS : 1;  // (fewer vectors than threads: some idle)
  static constexpr int kStep = THREADS / kPerRow;  // rows from one vector of a thread to its next
  u32x4 v[N];
  int to;           // bytes of this thread's first vector in the tile
  uint32_t whole;   // ... and in memory, for a chunk of C tokens
  uint32_t step;    // from there to the next one's

  __device__ __forceinline__ Rows(uint32_t stride, int cols, bool reverse) {
    const int c = (int)threadIdx.x % kPerRow, row = (int)threadIdx.x / kPerRow;
    to = place(row, c);
    whole = c * kVec < cols && row < C ? (uint32_t)(reverse ? C - 1 - row : row) * stride + 16u * (uint32_t)c : kOutside;
    step = reverse ? 0u - kStep * stride : kStep * stride;
  }
  // 16-byte vectors (fp32: its 8 bytes of each part).
  static __device__ __forceinline__ int place(int row, int c) {
    return Parts<E>::kIn == 3 ? (row_at<W>(row) ^ (c / 2 << 4)) + 8 * (c & 1) : row_at<W>(row) ^ (c << 4);
  }

  // Rows [t0, t0 + n) of the sequence in memory order; reversed: token t0 + n
  // - 1 first; n <= 0: zeros.  p: token 0; stride in bytes.
  __device__ __forceinline__ void load(const void* p, int64_t t0, int n, uint32_t stride, int cols, bool reverse) {
    const __amdgpu_buffer_rsrc_t r = make_rsrc(
        static_cast<const char*>(p) + t0 * (int64_t)stride,
        // (in a scalar register, or the loads go round a loop over their lanes' buffers)
        (uint32_t)__builtin_amdgcn_readfirstlane(n > 0 ? (uint32_t)(n - 1) * stride + (uint32_t)cols * (uint32_t)sizeof(raw) : 0u));
    if (VEC && n == C) {
      int at = (int)whole;
      keep(at);
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = __builtin_amdgcn_raw_buffer_load_b128(r, (uint32_t)at + i * step, 0, kPlain);
      return;
    }
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
    if (C * kPerRow < THREADS && (int)threadIdx.x >= C * kPerRow) return;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      // 8 rows on, the swizzle's second bit is the other one; 16 rows on it is the same
      const int at = kStep % 8 == 0 ? (to ^ (kStep * i % 16 == 8 ? 32 : 0)) + i * kStep * (2 * W)
                                    : place((int)threadIdx.x / kPerRow + i * kStep, (int)threadIdx.x % kPerRow);
      char* const p0 = lds + at;
      if constexpr (P == 1) {
        *reinterpret_cast<u32x4*>(p0) = v[i];
      } else if constexpr (P == 2) {
        typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
        const f16x8 h = __builtin_bit_cast(f16x8, v[i]);
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = (float)h[e];
        uint32_t w[2][4];
        split<2, 8>(x, w);
#pragma unroll
        for (int p = 0; p < 2; ++p) *reinterpret_cast<u32x4*>(p0 + p * (C * W * 2)) = u32x4{w[p][0], w[p][1], w[p][2], w[p][3]};
      } else {
        float x[4];
        uint32_t w[3][2];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = __uint_as_float(v[i][e]);
        split<3, 4>(x, w);
#pragma unroll
        for (int p = 0; p < 3; ++p) *reinterpret_cast<u32x2*>(p0 + p * (C * W * 2)) = u32x2{w[p][0], w[p][1]};
      }
    }
  }
};

// -- the workgroup's problem -----------------------------------------------------------------

template <class E, int DKP, int NT, int WAVES>
struct Shape {
  static constexpr int C = chunk_tokens<E, DKP>();
  static constexpr int DVT = 16 * NT * WAVES;       // columns of a workgroup
  static constexpr int KT = DKP / 16;       // 16-row tiles of the state
  static constexpr int kTile = 2 * C * Parts<E>::kIn;  // bytes of a tile's column
  static constexpr int kQ = 0, kK = kTile * DKP, kV = 2 * kTile * DKP, kP = kV + kTile * DVT;
  static constexpr int kPRow = C + 8;       // bf16 of a row of scores: rows 16 bytes apart on the banks
  static constexpr int kPPart = 2 * C * kPRow;
  static constexpr int kW = kP + kFull * kPPart;  // C weights of the state (state_weight)
  static constexpr int kD = kW + 4 * C;  // oscale kscale d^(C - x), x = 0 .. C; zeros to C + 15
  static constexpr int kLds = kD + 4 * (C + 16);
  // without scores: k and v only
  static constexpr int kLdsState = kTile * (DKP + DVT) + 4 * C;
};

// The weight of token j of n (at most C, reversed: p = 0) in the state after them.
__device__ __forceinline__ float state_weight(const AttnJob& job, float log_decay, int n, int p, int j) {
  return job.kscale * decay_power(log_decay, max(n - p - j, 0));  // (past n: rows of zeros)
}

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

// Keeps a value that is the same in every lane in a scalar register (the
// compiler would rather load it again inside the loop and wait for it).
__device__ __forceinline__ int pinned(int x) {
  x = __builtin_amdgcn_readfirstlane(x);
  asm volatile("" : "+s"(x));
  return x;
}

// Where o goes.
struct Out {
  char* p;
  int token;
  bool vec, wide;
};

// What a workgroup works on.
struct Where {
  int b, h, col0, cols;  // the first of its columns of the state, and how many exist
  int seg;
  Span s;
  const char *q, *k, *v;  // token 0 (v: of its columns)
  int64_t o;              // element of token 0, first column
  float log_decay;        // (set after the first loads are under way)
  float* states;          // slot 0 of a split sequence's states, in register order, or nullptr
  int64_t slot;           // elements from slot to slot
  int initial;            // the slot of the initial state, or -1
};

// The sequence and segment of a unit (see `pieces`): the last sequence whose first
// unit is not past it, by 64 offsets at a time.  False where there is none.  Offsets
// that decrease give any of them.
template <class A>
__device__ __forceinline__ bool find_unit(const A& a, uint32_t unit, int& b, int& seg) {
  const int lane = threadIdx.x & 63;
  int lo = 0, n = a.B;
  for (;;) {
    const int step = (n + 63) >> 6, probe = lo + lane * step;
    uint32_t own = ~0u;
    if (lane * step < n) {
      const int64_t first = a.offsets[probe];
      own = divide((uint32_t)(first < 0 ? 0 : first > a.rows ? a.rows : first), a.seg_tokens, a.by_seg) + probe;
    }
    const uint64_t before = __ballot(own <= unit);
    if (before == 0) return false;
    const int last = 63 - __builtin_clzll(before);
    lo += last * step;
    n = min(step, n - last * step);
    if (step == 1) {
      b = lo;
      seg = (int)(unit - (uint32_t)__builtin_amdgcn_readlane(own, last));
      return true;
    }
  }
}

template <class E, int DKP, int NT, int WAVES>
__device__ __forceinline__ bool where(const AttnArgs& a, const AttnJob& job, int segments, Where& w) {
  typedef typename E::raw raw;
  constexpr int DVT = 16 * NT * WAVES;
  // Every argument that the first loads need, and every cache line of the
  // others, at once: read where they are used, they take one trip to memory
  // after another.
  const AttnOperand q = job.q, k = job.k, v = job.v;
  asm volatile("" ::"s"(q.p), "s"(q.token), "s"(q.batch), "s"(q.head), "s"(q.group), "s"(q.inverse), "s"(k.p),
               "s"(k.token), "s"(k.batch), "s"(k.head), "s"(k.group), "s"(k.inverse), "s"(v.p), "s"(v.token),
               "s"(v.batch), "s"(v.head), "s"(v.group), "s"(v.inverse), "s"(a.lengths), "s"(a.offsets), "s"(a.rows),
               "s"(a.B), "s"(a.T), "s"(a.H), "s"(a.tiles), "s"(a.seg_tokens), "s"(a.by_tiles), "s"(a.by_seg), "s"(job.Dv),
               "s"(job.o.p), "s"(job.s_out), "s"(job.reverse));
  const uint32_t id = blockIdx.x, state = divide(id, a.tiles, a.by_tiles), tile = id - state * a.tiles;
  w.col0 = (int)tile * DVT;
  w.cols = job.Dv - w.col0;
  if (w.cols <= 0) return false;
  if (a.units > 0) {
    const uint32_t unit = divide(state, a.H, a.by_heads);
    w.h = (int)(state - unit * a.H);
    if (!find_unit(a, unit, w.b, w.seg)) return false;
    w.s = span_of(a, w.b);
    if (w.seg > 0 && (int64_t)w.seg * a.seg_tokens >= w.s.len) return false;
  } else {
    const uint32_t states = (uint32_t)a.B * a.H, seg = divide(state, states, a.by_states), bh = state - seg * states;
    w.seg = (int)seg;
    w.b = (int)divide(bh, a.H, a.by_heads);
    w.h = (int)bh - w.b * a.H;
    w.s = span_of(a, w.b);
  }
  w.q = static_cast<const char*>(q.p) + base_of(q, a, w.s, w.b, w.h) * (int64_t)sizeof(raw);
  w.k = static_cast<const char*>(k.p) + base_of(k, a, w.s, w.b, w.h) * (int64_t)sizeof(raw);
  w.v = static_cast<const char*>(v.p) + (base_of(v, a, w.s, w.b, w.h) + w.col0) * (int64_t)sizeof(raw);
  w.o = base_of(job.o, a, w.s, w.b, w.h) + w.col0;
  w.states = nullptr;
  w.slot = 0;
  w.initial = -1;
  if (job.segments != nullptr && w.s.len > a.seg_tokens) {
    const int64_t slot = first_slot(a, job, w.b, divide((uint32_t)w.s.first, a.seg_tokens, a.by_seg));
    w.states = job.segments + ((slot * a.H + w.h) * a.tiles + tile) * (DKP * DVT);
    w.slot = (int64_t)a.H * a.tiles * (DKP * DVT);
    if (job.s_in != nullptr) w.initial = (int)divide((uint32_t)w.s.len - 1, a.seg_tokens, a.by_seg);
  }
  if (w.cols > DVT) w.cols = DVT;
  return true;
}

// Row and column (in the workgroup's columns) of the state that element r of
// accumulator tile (t, n) of a lane holds.
__device__ __forceinline__ int state_row(int t, int r, int lane) {
  return 32 * (t / 2) + 8 * (lane >> 4) + 4 * (t % 2) + r;
}
template <int NT>
__device__ __forceinline__ int state_col(int m, int wave, int lane) {
  const int l = lane & 15;
  return NT == 2 ? 32 * wave + 8 * (l >> 2) + 4 * m + (l & 3) : 16 * wave + l;
}

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
template <class E, int DKP, int NT, bool OUT>
__device__ __forceinline__ void attention_tokens(const AttnJob& job, const Where& w, int lo, int hi, int wave, int lane,
                                                 f32x4 (&S)[DKP / 16][NT]) {
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
    float vv[NT], acc[NT];
#pragma unroll
    for (int m = 0; m < NT; ++m) {
      const int col = state_col<NT>(m, wave, lane);
      vv[m] = col < w.cols ? E::get(v[col]) : 0.f;
      acc[m] = 0.f;
    }
    int rows = job.Dk - first;  // rows of the state from the lane's first one on
    keep(rows);
#pragma unroll
    for (int x = 0; x < DKP / 16; ++x)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 32 * (x / 2) + 4 * (x % 2) + r;
        if (row < rows) {
          const float kk = E::get(k[row]) * job.kscale, qq = OUT ? E::get(q[row]) : 0.f;
#pragma unroll
          for (int m = 0; m < NT; ++m) {
            S[x][m][r] = __builtin_fmaf(kk, vv[m], S[x][m][r] * before);
            if (OUT) acc[m] = __builtin_fmaf(qq, S[x][m][r], acc[m]);
            S[x][m][r] *= after;
          }
        }
      }
    if constexpr (OUT) {
#pragma unroll
      for (int m = 0; m < NT; ++m) {
        const int col = state_col<NT>(m, wave, lane);
        acc[m] += __shfl_xor(acc[m], 16);
        acc[m] += __shfl_xor(acc[m], 32);
        if (lane < 16 && col < w.cols) put_out<E>(job, w.o + t * job.o.token + col, acc[m] * job.oscale);
      }
    }
  }
}

// Rows 32 j .. + 31 of the wave's columns of the chunk's v, as operands.
template <class E, int NT, int W, int C>
__device__ __forceinline__ void read_values(b16x8 (&V)[NT][Parts<E>::kIn], const char* v, int wave, int lane, int j) {
  const int g = lane >> 4, l = lane & 15;
  const int base = NT == 2 ? row_at<W>(8 * g + (l >> 2)) ^ ((4 * wave + (l & 3)) << 4)
                           : (row_at<W>(8 * g + (l >> 2)) ^ ((2 * wave + ((l & 3) >> 1)) << 4)) + 8 * (l & 1);
#pragma unroll
  for (int m = 0; m < NT; ++m)
#pragma unroll
    for (int p = 0; p < Parts<E>::kIn; ++p) {
      u32x2 half[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        half[h] = read_columns(v, (base ^ (16 * h)) + p * (C * W * 2) + (32 * j + 4 * h) * (2 * W) + 8 * m);
      const uint32_t words[4] = {half[0][0], half[0][1], half[1][0], half[1][1]};
      V[m][p] = operand(words);
    }
}

// Rows 32 j .. + 31 of the wave's columns of weights[j] v_j, as operands.
template <class E, int NT, int W, int C>
__device__ __forceinline__ void decayed_values(b16x8 (&D)[NT][kFull], const char* v, const float* weights, int wave,
                                               int lane, int j) {
  constexpr int IN = Parts<E>::kIn;
  b16x8 V[NT][IN];
  read_values<E, NT, W, C>(V, v, wave, lane, j);
  float w[8];
#pragma unroll
  for (int e = 0; e < 8; e += 4) {
    const f32x4 x = *reinterpret_cast<const f32x4*>(weights + 32 * j + 8 * (lane >> 4) + e);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[e + i] = x[i];
  }
#pragma unroll
  for (int m = 0; m < NT; ++m) {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[e] = (float)V[m][IN - 1][e];
#pragma unroll
      for (int p = IN - 2; p >= 0; --p) x[e] += (float)V[m][p][e];
      x[e] *= w[e];
    }
    uint32_t parts[kFull][4];
    split<kFull, 8>(x, parts);
#pragma unroll
    for (int p = 0; p < kFull; ++p) D[m][p] = operand(parts[p]);
  }
}

// Rows 16 t .. + 15 (as the state deals them) of the chunk's k^T, as operands.
// base: row 8 g + l / 4 of the tile of k, unit l % 4.
template <class E, int DKP, int C>
__device__ __forceinline__ void read_keys(b16x8 (&K)[C / 32][Parts<E>::kIn], const char* k, int base, int t) {
#pragma unroll
  for (int j = 0; j < C / 32; ++j)
#pragma unroll
    for (int p = 0; p < Parts<E>::kIn; ++p) {
      // 4 rows on: 8 W bytes and the swizzle's lowest bit
      u32x2 half[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        half[h] = read_columns(k, (base ^ (64 * (t / 2) + 16 * h)) + p * (C * DKP * 2) + (32 * j + 4 * h) * (2 * DKP) + 8 * (t % 2));
      const uint32_t words[4] = {half[0][0], half[0][1], half[1][0], half[1][1]};
      K[j][p] = operand(words);
    }
}

// S += k^T (D of all the chunk's tokens), for 16 rows of the state.
template <class E, int NT, int C>
__device__ __forceinline__ void update_tile(f32x4 (&S)[NT], const b16x8 (&D)[C / 32][NT][kFull],
                                            const b16x8 (&K)[C / 32][Parts<E>::kIn]) {
#pragma unroll
  for (int j = 0; j < C / 32; ++j) products<Parts<E>::kIn, kFull, NT>(S, K[j], D[j]);
}

// NaN from the first value on that is not finite, 0 until then.
template <int N, int M>
__device__ __forceinline__ void watch(float& z, const f32x4 (&x)[N][M]) {
  float y[4] = {z, 0.f, 0.f, 0.f};
#pragma unroll
  for (int t = 0; t < N; ++t)
#pragma unroll
    for (int m = 0; m < M; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) y[r] = __builtin_fmaf(x[t][m][r], 0.f, y[r]);
  z = (y[0] + y[1]) + (y[2] + y[3]);
}

// The head's initial state.
template <int DKP, int NT>
__device__ __forceinline__ void initial_state(f32x4 (&S)[DKP / 16][NT], const AttnJob& job, const Where& w, size_t head,
                                              int wave, int lane) {
#pragma unroll
  for (int m = 0; m < NT; ++m) {
    if (job.s_in == nullptr) {
#pragma unroll
      for (int t = 0; t < DKP / 16; ++t) S[t][m] = f32x4(0.f);
      continue;
    }
    const int col = state_col<NT>(m, wave, lane);
    const StateAt x(job.s_in, job, head, w.col0 + col, col < w.cols, lane);
#pragma unroll
    for (int t = 0; t < DKP / 16; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        S[t][m][r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(x.rsrc, x.at(t, r), 0, kPlain));
  }
}

// Split sequences.  Slot i of a sequence holds the state that segment i leaves by
// itself (segment 0: from the initial state), or after the scan the sequence's
// state after segment i; the last slot holds the initial state, if there is one,
// which the launch that needs it may overwrite in its own place.  (A sequence of
// one segment has one workgroup for each of its columns, which reads them before
// it writes them.)
template <int KT, int NT>
__device__ __forceinline__ f32x4* slot_at(const Where& w, int slot, int wave, int lane) {
  return reinterpret_cast<f32x4*>(w.states + slot * w.slot) + wave * (KT * NT * 64) + lane;
}

// The state a segment starts from.
template <int DKP, int NT>
__device__ __forceinline__ void first_state(f32x4 (&S)[DKP / 16][NT], const AttnArgs& a, const AttnJob& job,
                                            const Where& w, size_t head, int wave, int lane) {
  constexpr int KT = DKP / 16;
  if (w.states == nullptr || (w.seg == 0 && w.initial < 0)) {
    initial_state<DKP, NT>(S, job, w, head, wave, lane);
    return;
  }
  const bool scanned = a.segments >= kScanFrom;
  const f32x4* p = slot_at<KT, NT>(w, w.seg == 0 ? w.initial : scanned ? w.seg - 1 : 0, wave, lane);
#pragma unroll
  for (int t = 0; t < KT; ++t)
#pragma unroll
    for (int m = 0; m < NT; ++m) S[t][m] = p[(t * NT + m) * 64];
  if (scanned) return;
  const float whole = uniform(decay_power(w.log_decay, a.seg_tokens)), one = uniform(decay_power(w.log_decay, 1));
  for (int i = 1; i < w.seg; ++i) {
    const f32x4* own = slot_at<KT, NT>(w, i, wave, lane);
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int m = 0; m < NT; ++m) {
        const f32x4 x = own[(t * NT + m) * 64];
#pragma unroll
        for (int r = 0; r < 4; ++r) S[t][m][r] = carried(S[t][m][r], x[r], whole, one);
      }
  }
}
template <int DKP, int NT>
__device__ __forceinline__ void last_state(const f32x4 (&S)[DKP / 16][NT], const AttnJob& job, const Where& w, size_t head,
                                           int wave, int lane) {
#pragma unroll
  for (int m = 0; m < NT; ++m) {
    const int col = state_col<NT>(m, wave, lane);
    const StateAt x(job.s_out, job, head, w.col0 + col, col < w.cols, lane);
#pragma unroll
    for (int t = 0; t < DKP / 16; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[t][m][r]), x.rsrc, x.at(t, r), 0, kPlain);
  }
}

// The slots of every segment but the last: grid tiles x H x pieces (without the last segments), jobs.  The chunks
// are taken from a segment's last to its first, each weighted for the tokens
// behind it: the state itself is not touched between products, and the main
// kernel, which starts where this one ends, finds the tokens it reads first in
// the caches.  Measured: 32768 bf16 tokens of 32 heads of 128, 537 MB, 112 us (4.8
// TB/s; 122 from first to last).
template <class E, int DKP, int NT, int WAVES, bool VEC>
__global__ void __launch_bounds__(64 * WAVES, 2) attention_state_kernel(AttnArgs a) {
  typedef Shape<E, DKP, NT, WAVES> Sh;
  constexpr int C = Sh::C;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  char *const kt = lds, *const vt = lds + Sh::kTile * DKP;
  float* const weights = reinterpret_cast<float*>(lds + Sh::kTile * (DKP + Sh::DVT));
  const AttnJob& job = a.job[blockIdx.y];
  Where w;
  if (!where<E, DKP, NT, WAVES>(a, job, a.segments, w)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lo = w.seg * a.seg_tokens, hi = min(w.s.len, lo + a.seg_tokens);
  const int p = job.reverse ? 0 : 1;
  const uint32_t ks = (uint32_t)job.k.token * (uint32_t)sizeof(typename E::raw),
                 vs = (uint32_t)job.v.token * (uint32_t)sizeof(typename E::raw);

  Rows<E, C, DKP, 64 * WAVES, VEC> rk(ks, job.Dk, job.reverse);
  Rows<E, C, Sh::DVT, 64 * WAVES, VEC> rv(vs, w.cols, job.reverse);
  auto fetch = [&](int i) {
    const int n = i < lo ? 0 : min(C, hi - i);
    const int64_t t0 = n == 0 ? 0 : job.reverse ? w.s.len - i - n : i;
    rk.load(w.k, t0, n, ks, job.Dk, job.reverse);
    rv.load(w.v, t0, n, vs, w.cols, job.reverse);
  };
  if (hi >= w.s.len) return;  // no segment follows
  const int end = lo + (hi - lo - 1) / C * C;  // the last chunk's first token
  fetch(end);
  w.log_decay = uniform(a.log_decay[w.h]);
  const float decay = uniform(decay_power(w.log_decay, C));
  const float weight = (int)threadIdx.x < C ? state_weight(job, w.log_decay, C, p, threadIdx.x) : 0.f;
  const size_t head = (size_t)w.b * a.H + w.h;
  f32x4 S[Sh::KT][NT];
  auto start = [&]() {
    if (w.seg == 0) {
      initial_state<DKP, NT>(S, job, w, head, wave, lane);
    } else {
#pragma unroll
      for (int t = 0; t < Sh::KT; ++t)
#pragma unroll
        for (int m = 0; m < NT; ++m) S[t][m] = f32x4(0.f);
    }
  };
  auto put = [&](int slot) {
    f32x4* to = slot_at<Sh::KT, NT>(w, slot, wave, lane);
#pragma unroll
    for (int t = 0; t < Sh::KT; ++t)
#pragma unroll
      for (int m = 0; m < NT; ++m) to[(t * NT + m) * 64] = S[t][m];
  };
  start();
  if (w.seg == 0) {
    if (w.initial >= 0) put(w.initial);
    const float whole = uniform(decay_power(w.log_decay, hi - lo)), one = uniform(decay_power(w.log_decay, 1));
#pragma unroll
    for (int t = 0; t < Sh::KT; ++t)
#pragma unroll
      for (int m = 0; m < NT; ++m)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[t][m][r] = carried(S[t][m][r], 0.f, whole, one);
  }
  float after = 1.f;  // decay of the tokens behind the chunk
  for (int i = end; i >= lo; i -= C) {
    const int n = min(C, hi - i);
    if ((int)threadIdx.x < C)
      weights[threadIdx.x] = n == C ? weight * after : state_weight(job, w.log_decay, n, p, threadIdx.x);
    after = n == C ? after * decay : uniform(decay_power(w.log_decay, n));
    rk.store(kt);
    rv.store(vt);
    __syncthreads();
    fetch(i - C);
    b16x8 D[C / 32][NT][kFull];
#pragma unroll
    for (int j = 0; j < C / 32; ++j) decayed_values<E, NT, Sh::DVT, C>(D[j], vt, weights, wave, lane, j);
    const int base = row_at<DKP>(8 * (lane >> 4) + ((lane & 15) >> 2)) ^ ((lane & 3) << 4);
#pragma unroll
    for (int t = 0; t < Sh::KT; ++t) {
      b16x8 K[C / 32][Parts<E>::kIn];
      read_keys<E, DKP, C>(K, kt, base, t);
      update_tile<E, NT, C>(S[t], D, K);
    }
    __syncthreads();
  }
  float z = 0.f;
  watch(z, S);
  if (wave_any(z != 0.f)) {
    start();
    attention_tokens<E, DKP, NT, false>(job, w, lo, hi, wave, lane, S);
  }
  put(w.seg);
}

// Turns the segments' own states into the sequence's states after them, 4
// elements a thread, the loads of 8 slots ahead (15 slots of 32 heads of 128 x
// 128, 62 MB, 12 us).  grid: tiles x B H x (DKP DVT /
// 1024) workgroups, jobs.  (Slots that a sequence does not reach stay as they are:
// no one reads them.)
template <int DKP, int NT, int WAVES>
__global__ void __launch_bounds__(256) attention_scan_kernel(AttnArgs a) {
  constexpr int DVT = 16 * NT * WAVES, kBlocks = DKP * DVT / 1024, kAhead = 8;
  const AttnJob& job = a.job[blockIdx.y];
  const int id = blockIdx.x / kBlocks, bh = id / a.tiles, tile = id - bh * a.tiles, b = bh / a.H, h = bh - b * a.H;
  if (tile * DVT >= job.Dv) return;
  const Span s = span_of(a, b);
  const int reached = (s.len - 1) / a.seg_tokens;  // slots that are read
  if (reached < 2) return;
  const float whole = decay_power(a.log_decay[h], a.seg_tokens), one = decay_power(a.log_decay[h], 1);
  const int64_t slot = first_slot(a, job, b, (uint32_t)s.first / (uint32_t)a.seg_tokens);
  f32x4* p = reinterpret_cast<f32x4*>(job.segments) + ((slot * a.H + h) * a.tiles + tile) * (DKP * DVT / 4) +
             (blockIdx.x % kBlocks) * 256 + threadIdx.x;
  const int64_t step = (int64_t)a.H * a.tiles * (DKP * DVT / 4);
  f32x4 S = *p;
  for (int i0 = 1; i0 < reached; i0 += kAhead) {
    f32x4 own[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) own[i] = i0 + i < reached ? p[(i0 + i) * step] : f32x4(0.f);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (i0 + i >= reached) break;
#pragma unroll
      for (int r = 0; r < 4; ++r) S[r] = carried(S[r], own[i][r], whole, one);
      p[(i0 + i) * step] = S;
    }
  }
}

// Stores the chunk's rows of o, element type or fp32: a lane has 4 NT
// neighbouring columns of token 16 t + l.  Nontemporal, so that the caches keep q,
// k and v: backward of 8 x 2048 tokens of 16 bf16 heads of 128, operands not in the
// caches, 247 us, 251 with plain stores; with heads that share k and v in fours,
// whose fp32 rows the next launch reads, 316 and 319; the forward pass and the norm
// of each head after it, which reads o, 148 and 147.
constexpr int kStream = 2;
template <class E, int IT, int NT, bool WIDE>
__device__ __forceinline__ void put_rows(const Out& x, const Where& w, const f32x4 (&O)[IT][NT], int64_t t0, int n,
                                         bool reverse, int wave, int lane) {
  typedef typename E::raw raw;
  constexpr int kSize = WIDE ? 4 : 2;
  const int stride = x.token * kSize, c0 = 16 * NT * wave + 4 * NT * (lane >> 4);
  const __amdgpu_buffer_rsrc_t out = make_rsrc(x.p + (w.o + t0 * x.token) * kSize,
                                               (uint32_t)(n - 1) * (uint32_t)stride + (uint32_t)(w.cols * kSize));
  const int row = lane & 15;
  const int first = (reverse ? n - 1 - row : row) * stride + c0 * kSize, step = (reverse ? -16 : 16) * stride;
  if (x.vec) {
    const int live = c0 < w.cols ? n - row : 0;  // rows from this one on
#pragma unroll
    for (int t = 0; t < IT; ++t) {
      const uint32_t to = 16 * t < live ? (uint32_t)(first + t * step) : kOutside;
      if constexpr (WIDE) {
#pragma unroll
        for (int m = 0; m < NT; ++m)
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, O[t][m]), out, to + 16 * m, 0, kStream);
      } else {
        typedef raw vec __attribute__((ext_vector_type(4 * NT)));
        vec y;
#pragma unroll
        for (int e = 0; e < 4 * NT; ++e) y[e] = E::put(O[t][e / 4][e % 4]);
        if constexpr (NT == 2)
          __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, y), out, to, 0, kStream);
        else
          __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, y), out, to, 0, kStream);
      }
    }
    return;
  }
#pragma unroll
  for (int t = 0; t < IT; ++t)
#pragma unroll
    for (int e = 0; e < 4 * NT; ++e) {
      const uint32_t to = row + 16 * t < n && c0 + e < w.cols ? (uint32_t)(first + t * step + e * kSize) : kOutside;
      const float f = O[t][e / 4][e % 4];
      if constexpr (WIDE)
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(f), out, to, 0, kStream);
      else
        __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, E::put(f)), out, to, 0, kStream);
    }
}

// The attention: grid tiles x H x pieces, jobs.
template <class E, int DKP, int NT, int WAVES, bool VEC>
__global__ void __launch_bounds__(64 * WAVES, 2) attention_chunk_kernel(AttnArgs a) {
  typedef Shape<E, DKP, NT, WAVES> Sh;
  typedef typename E::raw raw;
  constexpr int C = Sh::C, IT = C / 16, IN = Parts<E>::kIn;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  char *const qt = lds + Sh::kQ, *const kt = lds + Sh::kK, *const vt = lds + Sh::kV, *const pt = lds + Sh::kP;
  float *const weights = reinterpret_cast<float*>(lds + Sh::kW), *const decays = reinterpret_cast<float*>(lds + Sh::kD);
  const AttnJob& job = a.job[blockIdx.y];
  Where w;
  if (!where<E, DKP, NT, WAVES>(a, job, a.segments, w)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = lane & 15;
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

  constexpr int kRaw = (int)sizeof(raw);
  const uint32_t qs = pinned((int)job.q.token * kRaw), ks = pinned((int)job.k.token * kRaw),
                 vs = pinned((int)job.v.token * kRaw);
  const int dk = pinned(job.Dk);
  const int flags = pinned((job.o_vec ? 1 : 0) | (job.o_f32 ? 2 : 0));
  const Out out = {static_cast<char*>(const_cast<void*>(job.o.p)), pinned((int)job.o.token), (flags & 1) != 0,
                   (flags & 2) != 0};
  Rows<E, C, DKP, 64 * WAVES, VEC> rq(qs, dk, reverse), rk(ks, dk, reverse);
  Rows<E, C, Sh::DVT, 64 * WAVES, VEC> rv(vs, w.cols, reverse);
  auto fetch = [&](int i) {
    const int n = max(0, min(C, hi - i));
    const int64_t t0 = n == 0 ? 0 : reverse ? w.s.len - i - n : i;
    rq.load(w.q, t0, n, qs, dk, reverse);
    rk.load(w.k, t0, n, ks, dk, reverse);
  };
  auto fetch_v = [&](int i) {
    const int n = max(0, min(C, hi - i));
    const int64_t t0 = n == 0 ? 0 : reverse ? w.s.len - i - n : i;
    rv.load(w.v, t0, n, vs, w.cols, reverse);
  };
  // The next chunk's loads start as soon as the tiles are in LDS where there
  // are registers for them through the whole chunk, else once the products with
  // the state are done (v after those with the scores).
  constexpr bool kEarly = C == 32 && !(DKP == 256 && IN == 3);
  fetch(lo);
  fetch_v(lo);
  w.log_decay = uniform(a.log_decay[w.h]);
  if ((int)threadIdx.x < C) weights[threadIdx.x] = state_weight(job, w.log_decay, C, p, threadIdx.x);
  if ((int)threadIdx.x < C + 16) {
    const int x = threadIdx.x;
    decays[x] = x <= C ? job.oscale * job.kscale * decay_power(w.log_decay, C - x) : 0.f;
  }
  // Score tiles above the diagonal that the products read: zero throughout.
  for (int x = threadIdx.x; x < kFull * Sh::kPPart / 4; x += 64 * WAVES) reinterpret_cast<uint32_t*>(pt)[x] = 0u;
  const float d16 = uniform(decay_power(w.log_decay, 16)), decay = uniform(decay_power(w.log_decay, C));
  const float from_state = job.oscale * decay_power(w.log_decay, l + p);  // of i = l

  f32x4 S[Sh::KT][NT];
  const size_t head = (size_t)w.b * a.H + w.h;
  first_state<DKP, NT>(S, a, job, w, head, wave, lane);
  bool broken = false;  // a value was not finite

  for (int i0 = lo; i0 < hi; i0 += C) {
    const int n = min(C, hi - i0);
    int lane = threadIdx.x & 63;
    keep(lane);
    const int g = lane >> 4, l = lane & 15;
    if (n < C && (int)threadIdx.x < C) weights[threadIdx.x] = state_weight(job, w.log_decay, n, p, threadIdx.x);
    rq.store(qt);
    rk.store(kt);
    rv.store(vt);
    __syncthreads();
    if (kEarly) {
      fetch(i0 + C);
      fetch_v(i0 + C);
    }

    const int rows = row_at<DKP>(l) ^ (g << 4);  // row l of a tile of 16, unit g

    // Scores, as P^T = k q^T, so that a lane has 4 tokens j of one i.  C = 64:
    // a wave takes the tiles of 16 tokens i up to the diagonal; C = 32: one of
    // the three tiles.  Which ones moves on from chunk to chunk, since they
    // differ and a wave's number is its SIMD's.
    const int turn = (wave + i0 / C) % 4, ti = C == 64 ? turn : (turn + 1) / 2, tj0 = C == 64 ? 0 : turn / 2;
    if (C == 64 || turn < 3) {
      constexpr int kTiles = C == 64 ? 4 : 1;
      f32x4 acc[kTiles];
#pragma unroll
      for (int x = 0; x < kTiles; ++x) acc[x] = f32x4(0.f);
#pragma unroll
      for (int s = 0; s < DKP / 32; ++s) {
        b16x8 Q[IN], K[kTiles][1][IN];
#pragma unroll
        for (int c = 0; c < IN; ++c) {
          Q[c] = read_row(qt, ti * (32 * DKP) + (rows ^ (64 * s)) + c * (C * DKP * 2));
#pragma unroll
          for (int x = 0; x < kTiles; ++x)
            if (tj0 + x <= ti) K[x][0][c] = read_row(kt, tj0 * (32 * DKP) + (rows ^ (64 * s)) + c * (C * DKP * 2) + x * (32 * DKP));
        }
#pragma unroll
        for (int x = 0; x < kTiles; ++x)
          if (tj0 + x <= ti) {
            f32x4 y[1] = {acc[x]};
            products<IN, IN, 1>(y, K[x], Q);
            acc[x] = y[0];
          }
      }
#pragma unroll
      for (int x = 0; x < kTiles; ++x) {
        const int tj = tj0 + x;
        if (tj > ti) break;
        const float* const d = decays + (C - 16 * (ti - tj) - l + 4 * g);  // of i - j; zeros above the diagonal
        float f[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) f[r] = acc[x][r] * d[r];
        uint32_t words[kFull][2];
        split<kFull, 4>(f, words);
#pragma unroll
        for (int c = 0; c < kFull; ++c)
          *reinterpret_cast<u32x2*>(pt + c * Sh::kPPart + 2 * ((16 * ti + l) * Sh::kPRow + 16 * tj + 4 * g)) =
              u32x2{words[c][0], words[c][1]};
      }
    }

    // o^T = S^T q^T, 32 rows of the state at a time, which then take the
    // chunk's tokens.  The reads of a step's operands are issued one product
    // ahead.
    const float dn = n == C ? decay : uniform(decay_power(w.log_decay, n));
    b16x8 D[C / 32][NT][kFull];
#pragma unroll
    for (int j = 0; j < C / 32; ++j) decayed_values<E, NT, Sh::DVT, C>(D[j], vt, weights, wave, lane, j);
    const int columns = row_at<DKP>(8 * g + (l >> 2)) ^ ((l & 3) << 4);
    f32x4 O[IT][NT];
#pragma unroll
    for (int t = 0; t < IT; ++t)
#pragma unroll
      for (int m = 0; m < NT; ++m) O[t][m] = f32x4(0.f);
    b16x8 Q[2][IT][IN];
    auto read_queries = [&](int s) {
#pragma unroll
      for (int t = 0; t < IT; ++t)
#pragma unroll
        for (int c = 0; c < IN; ++c) Q[s % 2][t][c] = read_row(qt, (rows ^ (64 * s)) + c * (C * DKP * 2) + t * (32 * DKP));
    };
    read_queries(0);
#pragma unroll
    for (int s = 0; s < DKP / 32; ++s) {
      b16x8 K[2][C / 32][IN];
#pragma unroll
      for (int y = 0; y < 2; ++y) read_keys<E, DKP, C>(K[y], kt, columns, 2 * s + y);
      if (s + 1 < DKP / 32) read_queries(s + 1);
      b16x8 A[NT][kFull];
#pragma unroll
      for (int m = 0; m < NT; ++m) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = S[2 * s + e / 4][m][e % 4];
        uint32_t words[kFull][4];
        split<kFull, 8>(x, words);
#pragma unroll
        for (int c = 0; c < kFull; ++c) A[m][c] = operand(words[c]);
      }
#pragma unroll
      for (int t = 0; t < IT; ++t) products<kFull, IN, NT>(O[t], A, Q[s % 2][t]);
#pragma unroll
      for (int y = 0; y < 2; ++y) {
#pragma unroll
        for (int m = 0; m < NT; ++m) S[2 * s + y][m] *= dn;
        update_tile<E, NT, C>(S[2 * s + y], D, K[y]);
      }
    }
    // times d^(i + p)
    float f = from_state;
#pragma unroll
    for (int t = 0; t < IT; ++t, f *= d16)
#pragma unroll
      for (int m = 0; m < NT; ++m) O[t][m] *= f;
    __syncthreads();  // the scores are in LDS
    if (!kEarly) fetch(i0 + C);

    // o^T += v^T P^T
#pragma unroll
    for (int j = 0; j < C / 32; ++j) {
      b16x8 V[NT][IN], P[IT][kFull];
      read_values<E, NT, Sh::DVT, C>(V, vt, wave, lane, j);
#pragma unroll
      for (int t = 2 * j; t < IT; ++t)
#pragma unroll
        for (int c = 0; c < kFull; ++c)
          P[t][c] = read_row(pt, c * Sh::kPPart + 2 * ((16 * t + l) * Sh::kPRow + 32 * j + 8 * g));
#pragma unroll
      for (int t = 2 * j; t < IT; ++t) products<IN, kFull, NT>(O[t], V, P[t]);
    }
    if (!kEarly) fetch_v(i0 + C);
    float z = 0.f;
    watch(z, O);
    broken = broken || wave_any(z != 0.f);
    const int64_t t0 = reverse ? w.s.len - i0 - n : i0;
    if constexpr (sizeof(raw) == 2) {
      if (!out.wide)
        put_rows<E, IT, NT, false>(out, w, O, t0, n, reverse, wave, lane);
      else
        put_rows<E, IT, NT, true>(out, w, O, t0, n, reverse, wave, lane);
    } else {
      put_rows<E, IT, NT, true>(out, w, O, t0, n, reverse, wave, lane);
    }

    __syncthreads();  // before the next chunk's tiles
  }
  float z = 0.f;
  watch(z, S);
  const bool ends = last && job.s_out != nullptr;
  int after = threadIdx.x & 63;  // (its products would else be held through the loop)
  keep(after);
  if (broken || wave_any(z != 0.f)) {
    first_state<DKP, NT>(S, a, job, w, head, wave, after);
    attention_tokens<E, DKP, NT, true>(job, w, lo, hi, wave, after, S);
  }
  if (ends) last_state<DKP, NT>(S, job, w, head, wave, after);
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

template <class E, int DKP, int NT, int WAVES, bool VEC>
hipError_t launch_shape(const AttnArgs& a, hipStream_t stream) {
  typedef Shape<E, DKP, NT, WAVES> Sh;
  const unsigned columns = (unsigned)a.tiles * a.H, states = columns * a.B;
  if (a.segments > 1) {
    const unsigned inner = a.units > 0 ? a.units : a.B * (a.segments - 1);  // (by number: the last segments, too)
    hipError_t e = launch_wide(attention_state_kernel<E, DKP, NT, WAVES, VEC>, dim3(columns * inner, a.jobs), 64 * WAVES,
                               Sh::kLdsState, a, stream);
    if (e != hipSuccess) return e;
    if (a.segments >= kScanFrom) {
      e = launch_wide(attention_scan_kernel<DKP, NT, WAVES>, dim3(states * (DKP * Sh::DVT / 1024), a.jobs), 256, 0, a, stream);
      if (e != hipSuccess) return e;
    }
  }
  const dim3 grid(columns * (unsigned)pieces(a), a.jobs);
  return launch_wide(attention_chunk_kernel<E, DKP, NT, WAVES, VEC>, grid, 64 * WAVES, Sh::kLds, a, stream);
}

template <class E, bool VEC>
hipError_t launch_vec(const AttnArgs& a, hipStream_t stream) {
  if (a.dkp == 64) return a.nt == 1 ? launch_shape<E, 64, 1, 4, VEC>(a, stream) : launch_shape<E, 64, 2, 4, VEC>(a, stream);
  if (a.dkp == 128) return a.nt == 1 ? launch_shape<E, 128, 1, 4, VEC>(a, stream) : launch_shape<E, 128, 2, 4, VEC>(a, stream);
  return launch_shape<E, 256, 1, 4, VEC>(a, stream);
}

template <class E>
hipError_t launch_type(const AttnArgs& a, hipStream_t stream) {
  return a.vec ? launch_vec<E, true>(a, stream) : launch_vec<E, false>(a, stream);
}

}  // namespace attn
}  // namespace prnn
