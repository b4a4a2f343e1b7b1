// Host side of the gated delta rule: argument checks, the plan and the workspace.
#include "delta_rule.h"

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <initializer_list>

#include "regions.h"

using namespace prnn;

namespace {

constexpr int64_t kMaxTokenStride = 1ll << 23;
constexpr int64_t kMaxTokens = 0x7fffffffll - (1 << 17) + 1;

struct Problem {
  prnnDeltaRule_t d;
  int64_t tokens;  // rows of the token axis
  size_t esize;
};

prnnStatus_t check_rule(prnnContext* h, const prnnDeltaRule_t* d, bool step, Problem* p) {
  if (h == nullptr || d == nullptr) return PRNN_STATUS_BAD_PARAM;
  if (handle_failed(h)) return PRNN_STATUS_EXECUTION_FAILED;
  if (d->B < 0 || d->H < 1 || d->Hk < 1 || d->H % d->Hk != 0) return PRNN_STATUS_BAD_PARAM;
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
  if ((int64_t)d->B * d->H > (1ll << 24)) return PRNN_STATUS_NOT_SUPPORTED;
  return PRNN_STATUS_SUCCESS;
}

// A sequence operand with elements of e bytes (null: absent, where it may be).
struct Tensor {
  const prnnSequence_t* s;
  int heads, D;
  size_t e;
};

bool tensor_ok(const Problem& p, const Tensor& t, bool step) {
  const prnnSequence_t* s = t.s;
  if (s == nullptr || s->batch < 0 || s->head < 0 || (!step && s->token < 0)) return false;
  if (s->batch > kMaxStride || s->head > kMaxStride || (!step && s->token > kMaxStride)) return false;
  return p.tokens == 0 || (s->data != nullptr && aligned(s->data, t.e));
}

Region region(const Problem& p, const Tensor& t, bool step) {
  Region r = flat(t.s->data, p.tokens > 0 ? (uint64_t)t.D * t.e : 0);
  r.axis[0] = {(uint64_t)t.s->head * t.e, (uint64_t)t.heads};
  if (!step) r.axis[1] = {(uint64_t)t.s->token * t.e, (uint64_t)p.tokens};
  if (step || p.d.offsets == nullptr) r.axis[2] = {(uint64_t)t.s->batch * t.e, (uint64_t)p.d.B};
  return r;
}

uint64_t state_bytes(const prnnDeltaRule_t& d) { return 4ull * d.B * d.H * d.Dk * d.Dv; }

// The buffers of a call: no output overlaps an input or another output, or itself.
// `s_in` and `s_out` may be one buffer.
prnnStatus_t check_buffers(const Problem& p, std::initializer_list<Tensor> ins, std::initializer_list<Tensor> outs,
                           std::initializer_list<const float*> states, const float* s_in, const float* s_out, bool step) {
  const prnnDeltaRule_t& d = p.d;
  Region in[16], out[8];
  int ni = 0, no = 0;
  bool far = false;
  for (const auto* list : {&ins, &outs})
    for (const Tensor& t : *list) {
      if (!tensor_ok(p, t, step)) return PRNN_STATUS_BAD_PARAM;
      far = far || (!step && t.s->token > kMaxTokenStride);
      (list == &ins ? in[ni++] : out[no++]) = region(p, t, step);
    }
  for (const float* s : states) {
    if (!aligned(s, 4)) return PRNN_STATUS_BAD_PARAM;
    in[ni++] = flat(s, state_bytes(d));
  }
  if (!aligned(s_in, 4) || !aligned(s_out, 4)) return PRNN_STATUS_BAD_PARAM;
  if (d.offsets != nullptr) in[ni++] = flat(d.offsets, 4ull * (d.B + 1));
  if (d.lengths != nullptr) in[ni++] = flat(d.lengths, 4ull * d.B);
  for (int i = 0; i < no; ++i)
    if (!distinct(out[i])) return PRNN_STATUS_BAD_PARAM;
  const Region from = flat(s_in, state_bytes(d)), to = flat(s_out, state_bytes(d));
  if (s_in != s_out && overlap(from, to)) return PRNN_STATUS_BAD_PARAM;
  out[no++] = to;
  for (int i = 0; i < no; ++i) {
    if (i + 1 < no && overlap(out[i], from)) return PRNN_STATUS_BAD_PARAM;
    for (int j = 0; j < ni; ++j)
      if (overlap(out[i], in[j])) return PRNN_STATUS_BAD_PARAM;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return PRNN_STATUS_BAD_PARAM;
  }
  return far ? PRNN_STATUS_NOT_SUPPORTED : PRNN_STATUS_SUCCESS;
}

AttnOperand operand(const prnnSequence_t* s, int group) {
  if (s == nullptr) return {nullptr, 0, 0, 0, 1, inverse_of(1)};
  return {s->data, s->token, s->batch, s->head, group, inverse_of(group)};
}

DeltaArgs base_args(const Problem& p, const prnnSequence_t* q, const prnnSequence_t* k, const prnnSequence_t* v,
                    const prnnSequence_t* g, const prnnSequence_t* beta, const prnnSequence_t* o) {
  DeltaArgs a;
  std::memset(&a, 0, sizeof(a));
  const int group = p.d.H / p.d.Hk;
  a.q = operand(q, group);
  a.k = operand(k, group);
  a.v = operand(v, 1);
  a.g = operand(g, 1);
  a.beta = operand(beta, 1);
  a.o = operand(o, 1);
  a.lengths = p.d.lengths;
  a.offsets = p.d.offsets;
  a.rows = p.d.offsets != nullptr ? p.tokens : 0;
  a.B = p.d.B;
  a.T = p.tokens > 0 ? p.d.T : 0;
  a.H = p.d.H;
  a.Dk = p.d.Dk;
  a.Dv = p.d.Dv;
  a.scale = p.d.scale;
  return a;
}

// Whether the launches' workgroups fit a grid (prepare: a wave for each chunk
// and head; the gradients: a workgroup for each group of chunks and head, which may have more
// than the 256 threads that kMaxWorkgroups counts).
bool grids_fit(const DeltaArgs& a, bool backward) {
  if ((double)a.slots * a.H > 4. * kMaxWorkgroups) return false;
  const int64_t blocks = a.slots * a.H;
  if (backward && a.group_slots * a.H * delta_grad_waves(a.dkp) > 4 * kMaxWorkgroups) return false;
  const double pieces = a.units > 0 ? (double)a.units * a.H : (double)a.B * a.H * a.segments;
  return (backward ? blocks : (blocks + 3) / 4) <= kMaxWorkgroups &&
         pieces * (a.tiles + (a.segments > 1 ? a.move_tiles : 0)) <= kMaxWorkgroups && (a.segments < 3 || (double)a.B * a.H * ((a.pitch + 15) / 16) <= kMaxWorkgroups);
}

void log_call(const prnnContext* h, const char* what, const Problem& p) {
  if (!handle_logs(h)) return;
  std::fprintf(stderr, "prnn: %s B=%d T=%d H=%d Hk=%d Dk=%d Dv=%d type=%d%s\n", what, p.d.B, p.d.T, p.d.H, p.d.Hk,
               p.d.Dk, p.d.Dv, (int)p.d.type, p.d.offsets != nullptr ? " packed" : p.d.lengths != nullptr ? " padded" : "");
}

size_t rounded(size_t bytes) { return (bytes + 255) / 256 * 256; }

// The workspace of split sequences, from `at` on (null: only its size).
size_t segment_memory(DeltaArgs* a, char* at) {
  const size_t parts = (size_t)a->seg_slots * a->H, states = rounded(parts * a->Dk * a->pitch * 4),
               moves = rounded(parts * a->Dk * a->move_pitch * 4);
  if (at != nullptr && parts > 0) {
    a->ends = reinterpret_cast<float*>(at);
    a->firsts = reinterpret_cast<float*>(at + states);
    a->moves = reinterpret_cast<float*>(at + 2 * states);
  }
  return 2 * states + moves;
}

}  // namespace

namespace prnn {

void plan_delta(DeltaArgs* a, prnnDataType_t type, bool backward, int compute_units) {
  const int e = type == PRNN_DATA_FLOAT ? 4 : 2;
  // whether every row starts at a multiple of `per` elements of `size` bytes and has a multiple of them
  auto vectors = [&](const AttnOperand& x, int D, int size, int per) {
    return D % per == 0 && (uintptr_t)x.p % (per * size) == 0 && (a->T <= 1 || x.token % per == 0) &&
           (a->offsets != nullptr ? x.token % per == 0 : a->B <= 1 || x.batch % per == 0) &&
           (a->H / x.group <= 1 || x.head % per == 0);
  };
  const int in = 16 / e, wide = a->qk_f32 ? 4 : e;
  a->vec = vectors(a->q, a->Dk, e, in) && vectors(a->k, a->Dk, e, in) && (backward || vectors(a->v, a->Dv, e, in)) &&
           (!backward || (vectors(a->v, a->Dv, e, in) && vectors(a->o, a->Dv, e, in)));
  if (!backward && vectors(a->o, a->Dv, e, 4)) a->vec |= 2;
  if (backward && vectors(a->dv, a->Dv, e, 4)) a->vec |= 4;
  if (backward && vectors(a->dq, a->Dk, wide, 4) && vectors(a->dk, a->Dk, wide, 4)) a->vec |= 8;
  a->dkp = a->Dk <= 64 ? 64 : a->Dk <= 128 ? 128 : 256;
  a->tiles = (a->Dv + 63) / 64;
  a->chunks = (int)(((int64_t)a->T + kDeltaChunk - 1) / kDeltaChunk);
  a->slots = a->T == 0 ? 0 : a->offsets != nullptr ? a->rows / kDeltaChunk + a->B : (int64_t)a->B * a->chunks;
  a->group = a->dkp == 128 && type != PRNN_DATA_FLOAT ? 2 : 1;  // (group_chunks)
  a->groups = (a->chunks + a->group - 1) / a->group;
  a->group_slots = a->T == 0 ? 0 : a->offsets != nullptr ? a->rows / (a->group * kDeltaChunk) + a->B : (int64_t)a->B * a->groups;
  a->pitch = (a->Dv + 3) / 4 * 4;
  a->move_pitch = (a->Dk + 3) / 4 * 4;
  a->move_tiles = (a->Dk + 63) / 64;
  // Segments: as many as give each compute unit 2 workgroups, of at least 4 chunks, and
  // no more than the root of the chunks (64 rows: twice that), since a step of the scan costs about
  // as much as a chunk.  A split in 2 gains nothing.  Measured in 1 / 4 / 6 / 8 / 10 / 12 / 16
  // segments: 32768 bf16 tokens of 32 heads of 128 (the rule: 8) 2481 / 1250 / 1126 / 1059 / 1134 /
  // 1088 / 1142 us; gradients of 3 x 1531 fp16 tokens of 6 heads of 96 x 80 (the rule: 6) 342 / 238 / 204 /
  // 218 / - / 210 / 243; 3001 packed fp16 rows of 16 heads of 64, the longest sequence 1463 (the rule:
  // 10) 123 / 81 / 73 / 71 / 68; 4 x 256 fp32 tokens of 14 heads of 128 (the rule: 1) 48 / 64.
  const int64_t sequences = a->offsets != nullptr && a->T > 0 ? std::max<int64_t>(1, std::min<int64_t>(a->B, a->rows / a->T)) : a->B;
  const int64_t states = std::max<int64_t>(1, sequences * a->H * a->tiles);
  int64_t segments = std::min<int64_t>(2 * compute_units / states, (int64_t)(std::sqrt((double)a->chunks) * (a->dkp == 64 ? 2 : 1)));
  segments = std::min<int64_t>(segments, a->chunks / 4);
  if (segments < 3) segments = 1;
  a->seg_chunks = std::max(1, (int)((a->chunks + segments - 1) / segments));
  a->segments = std::max(1, (a->chunks + a->seg_chunks - 1) / a->seg_chunks);
  const int64_t tokens = (int64_t)a->seg_chunks * kDeltaChunk;
  a->units = 0;
  a->seg_slots = 0;
  if (a->segments > 1) {
    a->seg_slots = a->offsets != nullptr ? a->rows / tokens + 1 : (int64_t)a->B * a->segments;
    if (a->offsets != nullptr) a->units = (int)(a->rows / tokens + a->B);
  }
  a->pieces = a->units > 0 ? a->units : a->B * a->segments;
  a->by_tiles = inverse_of(a->tiles);
  a->by_all_tiles = inverse_of(a->tiles + a->move_tiles);
  a->by_heads = inverse_of(a->H);
  a->by_chunks = inverse_of(std::max(1, a->chunks));
  a->by_groups = inverse_of(std::max(1, a->groups));
  a->by_group_tokens = inverse_of(a->group * kDeltaChunk);
  a->by_segments = inverse_of(a->segments);
  a->by_seg_chunks = inverse_of(a->seg_chunks);
  a->by_seg_tokens = inverse_of((int)tokens);
  a->by_pieces = inverse_of(a->pieces);
}

}  // namespace prnn

extern "C" {

prnnStatus_t prnn_gated_delta_rule(prnnHandle_t h, const prnnDeltaRule_t* d, const prnnSequence_t* q,
                                   const prnnSequence_t* k, const prnnSequence_t* v, const prnnSequence_t* log_decay,
                                   const prnnSequence_t* beta, const float* S0, const prnnSequence_t* o, float* S1,
                                   hipStream_t stream) {
  Problem p;
  prnnStatus_t st = check_rule(h, d, false, &p);
  if (st != PRNN_STATUS_SUCCESS || d->B == 0) return st;
  const Tensor tq = {q, d->Hk, d->Dk, p.esize}, tk = {k, d->Hk, d->Dk, p.esize}, tv = {v, d->H, d->Dv, p.esize},
               tb = {beta, d->H, 1, 4}, tg = {log_decay != nullptr ? log_decay : beta, d->H, 1, 4},
               to = {o, d->H, d->Dv, p.esize};
  st = check_buffers(p, {tq, tk, tv, tb, tg}, {to}, {}, S0, S1, false);
  if (st != PRNN_STATUS_SUCCESS) return st;
  if (p.tokens == 0 && S1 == nullptr) return PRNN_STATUS_SUCCESS;
  DeltaArgs a = base_args(p, q, k, v, log_decay, beta, o);
  a.s_in = S0;
  a.s_out = S1;
  plan_delta(&a, d->type, false, handle_compute_units(h));
  if (!grids_fit(a, false)) return PRNN_STATUS_NOT_SUPPORTED;
  if (a.slots > 0) {
    void* mem = nullptr;
    const size_t blocks = rounded((size_t)a.slots * a.H * kDeltaBlock);
    st = handle_workspace(h, blocks + segment_memory(&a, nullptr), stream, &mem);
    if (st != PRNN_STATUS_SUCCESS) return st;
    a.blocks = static_cast<char*>(mem);
    segment_memory(&a, a.blocks + blocks);
  }
  st = launched(launch_delta(a, d->type, false, stream));
  if (st == PRNN_STATUS_SUCCESS) log_call(h, "gated delta rule", p);
  return st;
}

prnnStatus_t prnn_gated_delta_rule_backward(prnnHandle_t h, const prnnDeltaRule_t* d, const prnnSequence_t* q,
                                            const prnnSequence_t* k, const prnnSequence_t* v,
                                            const prnnSequence_t* log_decay, const prnnSequence_t* beta, const float* S0,
                                            const prnnSequence_t* do_, const float* dS1, const prnnSequence_t* dq,
                                            const prnnSequence_t* dk, const prnnSequence_t* dv,
                                            const prnnSequence_t* dlog_decay, const prnnSequence_t* dbeta, float* dS0,
                                            hipStream_t stream) {
  Problem p;
  prnnStatus_t st = check_rule(h, d, false, &p);
  if (st != PRNN_STATUS_SUCCESS || d->B == 0) return st;
  const Tensor tq = {q, d->Hk, d->Dk, p.esize}, tk = {k, d->Hk, d->Dk, p.esize}, tv = {v, d->H, d->Dv, p.esize},
               tb = {beta, d->H, 1, 4}, tg = {log_decay != nullptr ? log_decay : beta, d->H, 1, 4},
               tdo = {do_, d->H, d->Dv, p.esize}, tdq = {dq, d->Hk, d->Dk, p.esize}, tdk = {dk, d->Hk, d->Dk, p.esize},
               tdv = {dv, d->H, d->Dv, p.esize}, tdb = {dbeta, d->H, 1, 4}, tdg = {dlog_decay, d->H, 1, 4};
  if (dlog_decay != nullptr)
    st = check_buffers(p, {tq, tk, tv, tb, tg, tdo}, {tdq, tdk, tdv, tdb, tdg}, {S0}, dS1, dS0, false);
  else
    st = check_buffers(p, {tq, tk, tv, tb, tg, tdo}, {tdq, tdk, tdv, tdb}, {S0}, dS1, dS0, false);
  if (st != PRNN_STATUS_SUCCESS) return st;
  if (p.tokens == 0 && dS0 == nullptr) return PRNN_STATUS_SUCCESS;
  DeltaArgs a = base_args(p, q, k, v, log_decay, beta, do_);
  const int group = d->H / d->Hk;
  const int64_t rows = d->offsets != nullptr ? p.tokens : p.tokens * d->B;
  if ((double)rows * d->H * (d->Dk + d->Dv) > 1e15) return PRNN_STATUS_ALLOC_FAILED;  // no memory holds it
  a.dq = operand(dq, 1);
  a.dk = operand(dk, 1);
  a.dv = operand(dv, 1);
  a.dg = operand(dlog_decay, 1);
  a.dbeta = operand(dbeta, 1);
  a.s_in = S0;
  a.ds_in = dS1;
  a.ds_out = dS0;
  // A shared head's gradient: every head's own in fp32 first, heads outermost, then their sum.
  const size_t heads = group > 1 ? rounded((size_t)rows * d->H * d->Dk * 4) : 0;
  if (group > 1) {
    for (AttnOperand* x : {&a.dq, &a.dk}) {
      *x = {nullptr, d->Dk, 0, p.tokens * d->Dk, 1, inverse_of(1)};
      if (d->offsets == nullptr) x->batch = d->H * x->head;
    }
    a.qk_f32 = 1;
  }
  plan_delta(&a, d->type, true, handle_compute_units(h));
  if (!grids_fit(a, true)) return PRNN_STATUS_NOT_SUPPORTED;
  if (a.slots > 0) {
    const size_t blocks = (size_t)a.slots * a.H, groups = (size_t)a.group_slots * a.H, pitch = a.pitch,
                 tokens = rounded(groups * a.group * kDeltaChunk * pitch * 4), states = rounded(groups * d->Dk * pitch * 4);
    void* mem = nullptr;
    const size_t segments = segment_memory(&a, nullptr);
    st = handle_workspace(h, rounded(blocks * kDeltaBlock) + 2 * (tokens + states + heads) + segments, stream, &mem);
    if (st != PRNN_STATUS_SUCCESS) return st;
    char* at = static_cast<char*>(mem);
    auto take = [&](size_t bytes) {
      char* const p0 = at;
      at += bytes;
      return p0;
    };
    a.blocks = take(rounded(blocks * kDeltaBlock));
    a.x = reinterpret_cast<float*>(take(tokens));
    a.w = reinterpret_cast<float*>(take(tokens));
    a.S = reinterpret_cast<float*>(take(states));
    a.R = reinterpret_cast<float*>(take(states));
    segment_memory(&a, take(segments));
    if (group > 1) {
      a.dq.p = take(heads);
      a.dk.p = take(heads);
    }
  }
  st = launched(launch_delta(a, d->type, true, stream));
  if (st == PRNN_STATUS_SUCCESS && group > 1 && p.tokens > 0) {
    AttnReduceArgs r;
    std::memset(&r, 0, sizeof(r));
    r.lengths = d->lengths;
    r.offsets = d->offsets;
    r.rows = a.rows;
    r.B = d->B;
    r.T = a.T;
    r.groups = d->Hk;
    r.per_group = group;
    r.grad[0].src = a.dq;
    r.grad[0].dst = operand(dq, 1);
    r.grad[1].src = a.dk;
    r.grad[1].dst = operand(dk, 1);
    r.grad[0].D = r.grad[1].D = d->Dk;
    st = launched(launch_attention_reduce(r, d->type, stream));
  }
  if (st == PRNN_STATUS_SUCCESS) log_call(h, "gated delta rule backward", p);
  return st;
}

prnnStatus_t prnn_gated_delta_rule_step(prnnHandle_t h, const prnnDeltaRule_t* d, const prnnSequence_t* q,
                                        const prnnSequence_t* k, const prnnSequence_t* v, const prnnSequence_t* log_decay,
                                        const prnnSequence_t* beta, const float* S0, const prnnSequence_t* o, float* S1,
                                        hipStream_t stream) {
  Problem p;
  prnnStatus_t st = check_rule(h, d, true, &p);
  if (st != PRNN_STATUS_SUCCESS || d->B == 0) return st;
  if (S0 == nullptr || S1 == nullptr) return PRNN_STATUS_BAD_PARAM;
  const Tensor tq = {q, d->Hk, d->Dk, p.esize}, tk = {k, d->Hk, d->Dk, p.esize}, tv = {v, d->H, d->Dv, p.esize},
               tb = {beta, d->H, 1, 4}, tg = {log_decay != nullptr ? log_decay : beta, d->H, 1, 4},
               to = {o, d->H, d->Dv, p.esize};
  st = check_buffers(p, {tq, tk, tv, tb, tg}, {to}, {}, S0, S1, true);
  if (st != PRNN_STATUS_SUCCESS) return st;
  const int group = d->H / d->Hk;
  DeltaStepArgs a;
  std::memset(&a, 0, sizeof(a));
  a.tiles = (d->Dv + 31) / 32;
  if ((int64_t)a.tiles * d->B * d->H > kMaxWorkgroups) return PRNN_STATUS_NOT_SUPPORTED;
  a.q = operand(q, group);
  a.k = operand(k, group);
  a.v = operand(v, 1);
  a.o = operand(o, 1);
  a.g = operand(log_decay, 1);
  a.beta = operand(beta, 1);
  a.s_in = S0;
  a.s_out = S1;
  a.B = d->B;
  a.H = d->H;
  a.Dk = d->Dk;
  a.Dv = d->Dv;
  a.scale = d->scale;
  st = launched(launch_delta_step(a, d->type, stream));
  if (st == PRNN_STATUS_SUCCESS) log_call(h, "gated delta rule step", p);
  return st;
}

}  // extern "C"
