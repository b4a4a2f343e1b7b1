// Host side of linear attention and layer norm: argument checks, the jobs of
// a launch and the workspace.
#include "sequence.h"

#include <algorithm>
#include <cstdio>
#include <cstring>

using namespace prnn;

namespace {

size_t size_of(prnnDataType_t t) { return t == PRNN_DATA_FLOAT ? 4 : 2; }
bool known(prnnDataType_t t) { return t == PRNN_DATA_FLOAT || t == PRNN_DATA_HALF || t == PRNN_DATA_BFLOAT; }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// The bytes a buffer touches: rows of `row` bytes at multiples of the strides
// below (bytes; counts of 1 have no stride).
struct Region {
  uintptr_t base = 0;
  uint64_t row = 0;  // 0: touches nothing
  struct Axis {
    uint64_t stride, count;
  } axis[3] = {};
};

// `e` and the bytes from an axis' first row to its last.  No memory reaches
// kFar: what does counts as that, so that the sums stay in 64 bits.
constexpr uint64_t kFar = 1ull << 60;
uint64_t along(uint64_t e, const Region::Axis& x) {
  if (x.count <= 1) return e;
  const unsigned __int128 far = (unsigned __int128)x.stride * (x.count - 1) + e;
  return far < kFar ? (uint64_t)far : kFar;
}

uint64_t extent(const Region& r) {
  uint64_t e = r.row;
  for (const auto& x : r.axis) e = along(e, x);
  return e;
}

uint64_t gcd(uint64_t a, uint64_t b) {
  while (b != 0) {
    const uint64_t t = a % b;
    a = b;
    b = t;
  }
  return a;
}

// Whether two regions can share a byte.  Ranges that meet are still disjoint
// when both repeat with one period (slices of one fused buffer) and their
// places inside that period do not meet: the axes whose strides are at least
// the period only move by whole periods.
bool overlap(const Region& a, const Region& b) {
  if (a.row == 0 || b.row == 0) return false;
  if (a.base >= b.base + extent(b) || b.base >= a.base + extent(a)) return false;
  // candidate periods: the strides of either region
  for (int from = 0; from < 6; ++from) {
    const auto& pick = from < 3 ? a.axis[from] : b.axis[from - 3];
    if (pick.count <= 1 || pick.stride == 0) continue;
    uint64_t period = pick.stride;
    for (const Region* r : {&a, &b})
      for (const auto& x : r->axis)
        if (x.count > 1 && x.stride >= pick.stride) period = gcd(period, x.stride);
    uint64_t foot[2];
    int i = 0;
    for (const Region* r : {&a, &b}) {
      foot[i] = r->row;
      for (const auto& x : r->axis)
        if (x.stride < pick.stride) foot[i] = along(foot[i], x);
      ++i;
    }
    const uint64_t d = a.base <= b.base ? (b.base - a.base) % period : (period - (a.base - b.base) % period) % period;
    if (d >= foot[0] && d + foot[1] <= period) return false;
  }
  return true;
}

// Whether every element of a region lies apart from the others.
bool distinct(const Region& r) {
  Region::Axis x[3] = {r.axis[0], r.axis[1], r.axis[2]};
  std::sort(x, x + 3, [](const Region::Axis& p, const Region::Axis& q) { return p.stride < q.stride; });
  uint64_t e = r.row;
  for (const auto& y : x) {
    if (y.count <= 1) continue;
    if (y.stride < e) return false;
    e = along(e, y);
  }
  return true;
}

Region flat(const void* p, uint64_t bytes) {
  Region r;
  r.base = reinterpret_cast<uintptr_t>(p);
  r.row = p != nullptr ? bytes : 0;
  return r;
}

Region rows_of(const void* p, int64_t M, int N, int64_t ld, size_t e) {
  Region r = flat(p, p != nullptr && M > 0 ? (uint64_t)N * e : 0);
  r.axis[0] = {(uint64_t)ld * e, (uint64_t)M};
  return r;
}

// Strides beyond this cannot address memory.
constexpr int64_t kMaxStride = 1ll << 40;
constexpr int64_t kMaxTokenStride = 1ll << 23;
// Tokens of a sequence: the segments that cover them, and a chunk more, stay in
// 31 bits (of at most 768 segments each is rounded up to 64 tokens).
constexpr int64_t kMaxTokens = 0x7fffffffll - (1 << 17) + 1;

struct Problem {
  prnnAttention_t d;
  int64_t tokens;  // rows of the token axis
  size_t esize;
};

bool seq_ok(const Problem& p, const prnnSequence_t* s, bool step) {
  if (s == nullptr || s->batch < 0 || s->head < 0 || (!step && s->token < 0)) return false;
  if (s->batch > kMaxStride || s->head > kMaxStride || (!step && s->token > kMaxStride)) return false;
  if (p.tokens == 0) return true;
  return s->data != nullptr && aligned(s->data, p.esize);
}

Region region(const Problem& p, const prnnSequence_t* s, int heads, int D, bool step) {
  Region r = flat(s->data, p.tokens > 0 ? (uint64_t)D * p.esize : 0);
  r.axis[0] = {(uint64_t)s->head * p.esize, (uint64_t)heads};
  if (!step) r.axis[1] = {(uint64_t)s->token * p.esize, (uint64_t)p.tokens};
  if (step || p.d.offsets == nullptr) r.axis[2] = {(uint64_t)s->batch * p.esize, (uint64_t)p.d.B};
  return r;
}

// The descriptor's own checks.
prnnStatus_t check_attention(prnnContext* h, const prnnAttention_t* d, bool step, Problem* p) {
  if (h == nullptr || d == nullptr) return PRNN_STATUS_BAD_PARAM;
  if (handle_failed(h)) return PRNN_STATUS_EXECUTION_FAILED;
  if (d->B < 0 || d->H < 1 || d->Hkv < 1 || d->H % d->Hkv != 0) return PRNN_STATUS_BAD_PARAM;
  if (d->Dk < 1 || d->Dv < 1 || d->Dk > PRNN_ATTENTION_MAX_D || d->Dv > PRNN_ATTENTION_MAX_D) return PRNN_STATUS_BAD_PARAM;
  if (!known(d->type)) return PRNN_STATUS_BAD_PARAM;
  p->d = *d;
  p->esize = size_of(d->type);
  if (step) {
    p->d.T = 1;
    p->d.lengths = p->d.offsets = nullptr;
    p->tokens = 1;
  } else {
    if (d->T < 0 || (d->lengths != nullptr && d->offsets != nullptr)) return PRNN_STATUS_BAD_PARAM;
    if (!aligned(d->lengths, 4) || !aligned(d->offsets, 4)) return PRNN_STATUS_BAD_PARAM;
    if (d->offsets != nullptr && d->rows < 0) return PRNN_STATUS_BAD_PARAM;
    p->tokens = d->offsets != nullptr ? d->rows : d->T;
    if (d->T == 0) p->tokens = 0;
    if (p->tokens > 0x7fffffffll) return PRNN_STATUS_NOT_SUPPORTED;
    p->d.T = (int)std::min<int64_t>(d->T, p->tokens);  // (packed: no sequence is longer than the rows)
    if (p->d.T > kMaxTokens) return PRNN_STATUS_NOT_SUPPORTED;
  }
  if (d->B == 0) return PRNN_STATUS_SUCCESS;
  if (d->log_decay == nullptr || !aligned(d->log_decay, 4)) return PRNN_STATUS_BAD_PARAM;
  if ((int64_t)d->B * d->H > (1ll << 24)) return PRNN_STATUS_NOT_SUPPORTED;
  return PRNN_STATUS_SUCCESS;
}

bool token_strides_fit(std::initializer_list<const prnnSequence_t*> all) {
  for (const prnnSequence_t* s : all)
    if (s->token > kMaxTokenStride) return false;
  return true;
}

AttnOperand operand(const prnnSequence_t* s, int group) { return {s->data, s->token, s->batch, s->head, group}; }

AttnArgs base_args(const Problem& p, int jobs) {
  AttnArgs a;
  std::memset(&a, 0, sizeof(a));
  a.log_decay = p.d.log_decay;
  a.lengths = p.d.lengths;
  a.offsets = p.d.offsets;
  a.rows = p.d.offsets != nullptr ? p.d.rows : 0;
  a.jobs = jobs;
  a.B = p.d.B;
  a.T = p.tokens > 0 ? p.d.T : 0;
  a.H = p.d.H;
  return a;
}

uint64_t state_bytes(const prnnAttention_t& d) { return 4ull * d.B * d.H * d.Dk * d.Dv; }

// A state output may be the state input itself, nothing else.
bool state_pair_ok(const prnnAttention_t& d, const float* in, const float* out) {
  return in == out || !overlap(flat(in, state_bytes(d)), flat(out, state_bytes(d)));
}

prnnStatus_t launched(hipError_t e) {
  if (e == hipSuccess) return PRNN_STATUS_SUCCESS;
  (void)hipGetLastError();
  return PRNN_STATUS_INTERNAL_ERROR;
}

void log_call(const prnnContext* h, const char* what, const Problem& p) {
  if (!handle_logs(h)) return;
  std::fprintf(stderr, "prnn: %s B=%d T=%d H=%d Hkv=%d Dk=%d Dv=%d type=%d%s\n", what, p.d.B, p.d.T, p.d.H, p.d.Hkv,
               p.d.Dk, p.d.Dv, (int)p.d.type, p.d.offsets != nullptr ? " packed" : p.d.lengths != nullptr ? " padded" : "");
}

}  // namespace

extern "C" {

prnnStatus_t prnn_linear_attention(prnnHandle_t h, const prnnAttention_t* d, const prnnSequence_t* q,
                                   const prnnSequence_t* k, const prnnSequence_t* v, const float* S0,
                                   const prnnSequence_t* o, float* S1, hipStream_t stream) {
  Problem p;
  prnnStatus_t st = check_attention(h, d, false, &p);
  if (st != PRNN_STATUS_SUCCESS || d->B == 0) return st;
  for (const prnnSequence_t* s : {q, k, v, o})
    if (!seq_ok(p, s, false)) return PRNN_STATUS_BAD_PARAM;
  if (!aligned(S0, 4) || !aligned(S1, 4) || !state_pair_ok(*d, S0, S1)) return PRNN_STATUS_BAD_PARAM;
  const Region rq = region(p, q, d->H, d->Dk, false), rk = region(p, k, d->Hkv, d->Dk, false),
               rv = region(p, v, d->Hkv, d->Dv, false), ro = region(p, o, d->H, d->Dv, false);
  const Region s0 = flat(S0, state_bytes(*d)), s1 = flat(S1, state_bytes(*d)), ld = flat(d->log_decay, 4ull * d->H),
               sp = flat(d->offsets != nullptr ? d->offsets : d->lengths, 4ull * (d->B + (d->offsets != nullptr)));
  if (!distinct(ro) || overlap(ro, s1)) return PRNN_STATUS_BAD_PARAM;
  for (const Region& in : {rq, rk, rv, ld, sp})
    if (overlap(ro, in) || overlap(s1, in)) return PRNN_STATUS_BAD_PARAM;
  if (overlap(ro, s0)) return PRNN_STATUS_BAD_PARAM;
  if (!token_strides_fit({q, k, v, o})) return PRNN_STATUS_NOT_SUPPORTED;
  if (p.tokens == 0 && S1 == nullptr) return PRNN_STATUS_SUCCESS;

  AttnArgs a = base_args(p, 1);
  AttnJob& j = a.job[0];
  const int group = d->H / d->Hkv;
  j.q = operand(q, 1);
  j.k = operand(k, group);
  j.v = operand(v, group);
  j.o = operand(o, 1);
  j.s_in = S0;
  j.s_out = S1;
  j.Dk = d->Dk;
  j.Dv = d->Dv;
  j.s_row = d->Dv;
  j.s_col = 1;
  j.kscale = 1.f;
  j.oscale = d->scale;
  const size_t floats = plan_attention(&a, d->type, handle_compute_units(h));
  if (!grid_fits(a)) return PRNN_STATUS_NOT_SUPPORTED;
  if (floats > 0) {
    void* mem = nullptr;
    st = handle_workspace(h, floats * 4, stream, &mem);
    if (st != PRNN_STATUS_SUCCESS) return st;
    j.segments = static_cast<float*>(mem);
  }
  st = launched(launch_attention(a, d->type, stream));
  if (st == PRNN_STATUS_SUCCESS) log_call(h, "linear attention", p);
  return st;
}

prnnStatus_t prnn_linear_attention_backward(prnnHandle_t h, const prnnAttention_t* d, const prnnSequence_t* q,
                                            const prnnSequence_t* k, const prnnSequence_t* v, const float* S0,
                                            const prnnSequence_t* do_, const float* dS1, const prnnSequence_t* dq,
                                            const prnnSequence_t* dk, const prnnSequence_t* dv, float* dS0,
                                            hipStream_t stream) {
  Problem p;
  prnnStatus_t st = check_attention(h, d, false, &p);
  if (st != PRNN_STATUS_SUCCESS || d->B == 0) return st;
  for (const prnnSequence_t* s : {q, k, v, do_, dq, dk, dv})
    if (!seq_ok(p, s, false)) return PRNN_STATUS_BAD_PARAM;
  if (!aligned(S0, 4) || !aligned(dS1, 4) || !aligned(dS0, 4) || !state_pair_ok(*d, dS1, dS0)) return PRNN_STATUS_BAD_PARAM;
  const Region in[] = {region(p, q, d->H, d->Dk, false),
                       region(p, k, d->Hkv, d->Dk, false),
                       region(p, v, d->Hkv, d->Dv, false),
                       region(p, do_, d->H, d->Dv, false),
                       flat(S0, state_bytes(*d)),
                       flat(d->log_decay, 4ull * d->H),
                       flat(d->offsets != nullptr ? d->offsets : d->lengths, 4ull * (d->B + (d->offsets != nullptr)))};
  const Region out[] = {region(p, dq, d->H, d->Dk, false), region(p, dk, d->Hkv, d->Dk, false),
                        region(p, dv, d->Hkv, d->Dv, false), flat(dS0, state_bytes(*d))};
  const Region ds1 = flat(dS1, state_bytes(*d));
  for (int i = 0; i < 4; ++i) {
    if (i < 3 && (!distinct(out[i]) || overlap(out[i], ds1))) return PRNN_STATUS_BAD_PARAM;
    for (const Region& r : in)
      if (overlap(out[i], r)) return PRNN_STATUS_BAD_PARAM;
    for (int m = 0; m < i; ++m)
      if (overlap(out[i], out[m])) return PRNN_STATUS_BAD_PARAM;
  }
  if (!token_strides_fit({q, k, v, do_, dq, dk, dv})) return PRNN_STATUS_NOT_SUPPORTED;
  if (p.tokens == 0 && dS0 == nullptr) return PRNN_STATUS_SUCCESS;

  const int group = d->H / d->Hkv;
  const int64_t rows = d->offsets != nullptr ? p.tokens : p.tokens * d->B;
  // A shared head's gradient: every head's own in fp32 first, then their sum.
  // Heads outermost, so that a row is D elements whatever their number (the
  // kernels count a chunk's rows in 32 bits).
  if (group > 1 && (double)rows * d->H * (d->Dk + d->Dv) > 1e15) return PRNN_STATUS_ALLOC_FAILED;  // no memory holds it
  const size_t wide_k = group > 1 ? ((size_t)rows * d->H * d->Dk * 4 + 255) / 256 * 256 : 0;
  const size_t wide_v = group > 1 ? ((size_t)rows * d->H * d->Dv * 4 + 255) / 256 * 256 : 0;
  auto dense = [&](float* mem, int D) {
    AttnOperand x = {mem, D, 0, p.tokens * D, 1};
    if (d->offsets == nullptr) x.batch = d->H * x.head;
    return x;
  };
  AttnArgs a = base_args(p, 3);
  AttnJob& jq = a.job[0];
  jq.q = operand(do_, 1);
  jq.k = operand(v, group);
  jq.v = operand(k, group);
  jq.o = operand(dq, 1);
  jq.s_in = S0;
  jq.Dk = d->Dv;
  jq.Dv = d->Dk;
  jq.s_row = 1;
  jq.s_col = d->Dv;
  jq.kscale = 1.f;
  jq.oscale = d->scale;
  AttnJob& jk = a.job[1];
  jk.q = operand(v, group);
  jk.k = operand(do_, 1);
  jk.v = operand(q, 1);
  jk.o = group > 1 ? dense(nullptr, d->Dk) : operand(dk, 1);
  jk.o_f32 = group > 1;
  jk.s_in = dS1;
  jk.Dk = d->Dv;
  jk.Dv = d->Dk;
  jk.s_row = 1;
  jk.s_col = d->Dv;
  jk.kscale = d->scale;
  jk.oscale = 1.f;
  jk.reverse = 1;
  AttnJob& jv = a.job[2];
  jv.q = operand(k, group);
  jv.k = operand(q, 1);
  jv.v = operand(do_, 1);
  jv.o = group > 1 ? dense(nullptr, d->Dv) : operand(dv, 1);
  jv.o_f32 = group > 1;
  jv.s_in = dS1;
  jv.s_out = dS0;
  jv.Dk = d->Dk;
  jv.Dv = d->Dv;
  jv.s_row = d->Dv;
  jv.s_col = 1;
  jv.kscale = d->scale;
  jv.oscale = 1.f;
  jv.reverse = 1;
  const size_t floats = plan_attention(&a, d->type, handle_compute_units(h));
  if (!grid_fits(a)) return PRNN_STATUS_NOT_SUPPORTED;
  // dS0 in the place of dS1: dk's job reads dS1, dv's writes dS0, and nothing
  // orders the workgroups of one launch, so dk's reads a copy.
  const size_t kept = dS0 != nullptr && dS0 == dS1 ? (size_t)state_bytes(*d) : 0;
  float* work = nullptr;  // the heads' gradients, the segments of the three jobs, the kept state
  if (wide_k + wide_v + floats + kept > 0) {
    void* mem = nullptr;
    st = handle_workspace(h, wide_k + wide_v + 12 * floats + kept, stream, &mem);
    if (st != PRNN_STATUS_SUCCESS) return st;
    work = static_cast<float*>(mem);
    if (kept > 0) {
      a.keep_from = dS1;
      a.keep_to = work + (wide_k + wide_v) / 4 + 3 * floats;
      a.keep = (int64_t)(kept / 4);
      jk.s_in = a.keep_to;
    }
    if (group > 1) {
      jk.o.p = work;
      jv.o.p = work + wide_k / 4;
    }
    for (int i = 0; i < 3 && floats > 0; ++i) a.job[i].segments = work + (wide_k + wide_v) / 4 + i * floats;
  }
  st = launched(launch_attention(a, d->type, stream));
  if (st == PRNN_STATUS_SUCCESS && group > 1 && p.tokens > 0) {
    AttnReduceArgs r;
    std::memset(&r, 0, sizeof(r));
    r.lengths = d->lengths;
    r.offsets = d->offsets;
    r.rows = a.rows;
    r.B = d->B;
    r.T = a.T;
    r.groups = d->Hkv;
    r.per_group = group;
    r.grad[0].src = jk.o;
    r.grad[0].dst = operand(dk, 1);
    r.grad[0].D = d->Dk;
    r.grad[1].src = jv.o;
    r.grad[1].dst = operand(dv, 1);
    r.grad[1].D = d->Dv;
    st = launched(launch_attention_reduce(r, d->type, stream));
  }
  if (st == PRNN_STATUS_SUCCESS) log_call(h, "linear attention backward", p);
  return st;
}

prnnStatus_t prnn_linear_attention_step(prnnHandle_t h, const prnnAttention_t* d, const prnnSequence_t* q,
                                        const prnnSequence_t* k, const prnnSequence_t* v, const float* S0,
                                        const prnnSequence_t* o, float* S1, hipStream_t stream) {
  Problem p;
  prnnStatus_t st = check_attention(h, d, true, &p);
  if (st != PRNN_STATUS_SUCCESS || d->B == 0) return st;
  for (const prnnSequence_t* s : {q, k, v, o})
    if (!seq_ok(p, s, true)) return PRNN_STATUS_BAD_PARAM;
  if (S0 == nullptr || S1 == nullptr || !aligned(S0, 4) || !aligned(S1, 4) || !state_pair_ok(*d, S0, S1))
    return PRNN_STATUS_BAD_PARAM;
  const Region ro = region(p, o, d->H, d->Dv, true), s1 = flat(S1, state_bytes(*d));
  if (!distinct(ro) || overlap(ro, s1) || overlap(ro, flat(S0, state_bytes(*d)))) return PRNN_STATUS_BAD_PARAM;
  for (const Region& in : {region(p, q, d->H, d->Dk, true), region(p, k, d->Hkv, d->Dk, true),
                           region(p, v, d->Hkv, d->Dv, true), flat(d->log_decay, 4ull * d->H)})
    if (overlap(ro, in) || overlap(s1, in)) return PRNN_STATUS_BAD_PARAM;
  const int group = d->H / d->Hkv;
  AttnStepArgs a;
  std::memset(&a, 0, sizeof(a));
  a.tiles = (d->Dv + 31) / 32;
  if ((int64_t)a.tiles * d->B * d->H > kMaxWorkgroups) return PRNN_STATUS_NOT_SUPPORTED;
  a.q = operand(q, 1);
  a.k = operand(k, group);
  a.v = operand(v, group);
  a.o = operand(o, 1);
  a.log_decay = d->log_decay;
  a.s_in = S0;
  a.s_out = S1;
  a.B = d->B;
  a.H = d->H;
  a.Dk = d->Dk;
  a.Dv = d->Dv;
  a.scale = d->scale;
  st = launched(launch_attention_step(a, d->type, stream));
  if (st == PRNN_STATUS_SUCCESS) log_call(h, "linear attention step", p);
  return st;
}

// The checks both directions share.
static prnnStatus_t check_norm(prnnContext* h, int64_t M, int N, prnnDataType_t type, prnnDataType_t ptype) {
  if (h == nullptr) return PRNN_STATUS_BAD_PARAM;
  if (handle_failed(h)) return PRNN_STATUS_EXECUTION_FAILED;
  if (M < 0 || N < 1 || !known(type) || !known(ptype)) return PRNN_STATUS_BAD_PARAM;
  if (ptype != PRNN_DATA_FLOAT && ptype != type) return PRNN_STATUS_BAD_PARAM;
  // (columns are counted in 31 bits, in steps of up to 1024)
  return M > 0x7fffffffll || N > 0x7fffffff - 1023 ? PRNN_STATUS_NOT_SUPPORTED : PRNN_STATUS_SUCCESS;
}

static bool ld_ok(int64_t ld, int N) { return ld >= N && ld <= kMaxStride; }

prnnStatus_t prnn_layer_norm(prnnHandle_t h, int64_t M, int N, prnnDataType_t type, const void* x, int64_t ldx,
                             prnnDataType_t ptype, const void* weight, const void* bias, float eps, void* y,
                             int64_t ldy, float* mean, float* rstd, hipStream_t stream) {
  const prnnStatus_t st = check_norm(h, M, N, type, ptype);
  if (st != PRNN_STATUS_SUCCESS) return st;
  if (!(eps >= 0.f) || !ld_ok(ldx, N) || !ld_ok(ldy, N)) return PRNN_STATUS_BAD_PARAM;
  if (M == 0) return PRNN_STATUS_SUCCESS;
  const size_t e = size_of(type), pe = size_of(ptype);
  if (x == nullptr || y == nullptr || !aligned(x, e) || !aligned(y, e) || !aligned(weight, pe) || !aligned(bias, pe) ||
      !aligned(mean, 4) || !aligned(rstd, 4))
    return PRNN_STATUS_BAD_PARAM;
  const Region rx = rows_of(x, M, N, ldx, e), ry = rows_of(y, M, N, ldy, e), rm = flat(mean, 4ull * M),
               rr = flat(rstd, 4ull * M);
  if (!(x == y && ldx == ldy) && overlap(rx, ry)) return PRNN_STATUS_BAD_PARAM;
  if (overlap(ry, rm) || overlap(ry, rr) || overlap(rm, rr) || overlap(rx, rm) || overlap(rx, rr))
    return PRNN_STATUS_BAD_PARAM;
  for (const Region& in : {flat(weight, pe * N), flat(bias, pe * N)})
    if (overlap(ry, in) || overlap(rm, in) || overlap(rr, in)) return PRNN_STATUS_BAD_PARAM;
  NormArgs a;
  std::memset(&a, 0, sizeof(a));
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  a.M = M;
  a.N = N;
  a.ldx = ldx;
  a.ldy = ldy;
  a.eps = eps;
  a.compute_units = handle_compute_units(h);
  return launched(launch_layer_norm(a, type, ptype, stream));
}

prnnStatus_t prnn_layer_norm_backward(prnnHandle_t h, int64_t M, int N, prnnDataType_t type, const void* dy,
                                      int64_t lddy, const void* x, int64_t ldx, const float* mean, const float* rstd,
                                      prnnDataType_t ptype, const void* weight, void* dx, int64_t lddx, void* dweight,
                                      void* dbias, hipStream_t stream) {
  prnnStatus_t st = check_norm(h, M, N, type, ptype);
  if (st != PRNN_STATUS_SUCCESS) return st;
  if (!ld_ok(ldx, N) || !ld_ok(lddy, N) || (dx != nullptr && !ld_ok(lddx, N))) return PRNN_STATUS_BAD_PARAM;
  const size_t e = size_of(type), pe = size_of(ptype);
  if (M > 0 && (x == nullptr || dy == nullptr || mean == nullptr || rstd == nullptr)) return PRNN_STATUS_BAD_PARAM;
  if (!aligned(x, e) || !aligned(dy, e) || !aligned(dx, e) || !aligned(mean, 4) || !aligned(rstd, 4) ||
      !aligned(weight, pe) || !aligned(dweight, pe) || !aligned(dbias, pe))
    return PRNN_STATUS_BAD_PARAM;
  const Region rx = rows_of(x, M, N, ldx, e), rdy = rows_of(dy, M, N, lddy, e), rdx = rows_of(dx, M, N, lddx, e),
               rw = flat(dweight, pe * N), rb = flat(dbias, pe * N);
  if (!(dx == x && lddx == ldx) && overlap(rdx, rx)) return PRNN_STATUS_BAD_PARAM;
  if (!(dx == dy && lddx == lddy) && overlap(rdx, rdy)) return PRNN_STATUS_BAD_PARAM;
  if (overlap(rdx, rw) || overlap(rdx, rb) || overlap(rw, rb)) return PRNN_STATUS_BAD_PARAM;
  for (const Region& in : {flat(mean, 4ull * M), flat(rstd, 4ull * M), flat(weight, pe * N)})
    if (overlap(rdx, in) || overlap(rw, in) || overlap(rb, in)) return PRNN_STATUS_BAD_PARAM;
  for (const Region& in : {rx, rdy})
    if (overlap(rw, in) || overlap(rb, in)) return PRNN_STATUS_BAD_PARAM;
  if (dx == nullptr && dweight == nullptr && dbias == nullptr) return PRNN_STATUS_SUCCESS;
  if (M == 0 && dweight == nullptr && dbias == nullptr) return PRNN_STATUS_SUCCESS;
  NormArgs a;
  std::memset(&a, 0, sizeof(a));
  a.x = x;
  a.dy = dy;
  a.weight = weight;
  a.y = dx;
  a.mean_in = mean;
  a.rstd_in = rstd;
  a.dweight = dweight;
  a.dbias = dbias;
  a.M = M;
  a.N = N;
  a.ldx = ldx;
  a.ldy = lddx;
  a.lddy = lddy;
  const int grid = layer_norm_backward_grid(a, type, handle_compute_units(h));
  if (grid > 0 && (dweight != nullptr || dbias != nullptr)) {
    void* mem = nullptr;
    st = handle_workspace(h, (size_t)grid * 2 * N * 4, stream, &mem);
    if (st != PRNN_STATUS_SUCCESS) return st;
    a.partial = static_cast<float*>(mem);
  }
  return launched(launch_layer_norm_backward(a, type, ptype, grid, stream));
}

}  // extern "C"
