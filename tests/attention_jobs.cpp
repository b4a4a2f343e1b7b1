// Calls linear attention with stand-ins for the handle and the launches, and
// checks what would have been launched (see test_attention_jobs.py).  Device
// pointers are numbers: nothing here reads them.
#include <algorithm>
#include <cstdio>
#include <cstring>
#include <vector>

#include "sequence.h"

struct prnnContext {};

static const uintptr_t kWork = 0x700000000000ull;
static size_t workspace = 0;  // bytes asked for by the last call
static prnn::AttnArgs args;   // of the last launch
static prnn::AttnReduceArgs reduced;
static int launches = 0, steps = 0, reductions = 0;

namespace prnn {
bool handle_failed(prnnContext*) { return false; }
int handle_compute_units(const prnnContext*) { return 256; }
bool handle_logs(const prnnContext*) { return false; }
prnnStatus_t handle_workspace(prnnContext*, size_t bytes, hipStream_t, void** out) {
  workspace = bytes;
  *out = reinterpret_cast<void*>(kWork);
  return PRNN_STATUS_SUCCESS;
}
hipError_t launch_attention(const AttnArgs& a, prnnDataType_t, hipStream_t) {
  args = a;
  ++launches;
  return hipSuccess;
}
hipError_t launch_attention_reduce(const AttnReduceArgs& a, prnnDataType_t, hipStream_t) {
  reduced = a;
  ++reductions;
  return hipSuccess;
}
hipError_t launch_attention_step(const AttnStepArgs&, prnnDataType_t, hipStream_t) {
  ++steps;
  return hipSuccess;
}
hipError_t launch_layer_norm(const NormArgs&, prnnDataType_t, prnnDataType_t, hipStream_t) { return hipSuccess; }
int layer_norm_backward_grid(const NormArgs&, prnnDataType_t, int) { return 0; }
hipError_t launch_layer_norm_backward(const NormArgs&, prnnDataType_t, prnnDataType_t, int, hipStream_t) { return hipSuccess; }
}  // namespace prnn
extern "C" hipError_t hipGetLastError() { return hipSuccess; }

static int failures = 0;
#define CHECK(ok, ...)                          \
  do {                                          \
    if (!(ok)) {                                \
      std::printf("%s: ", #ok);                 \
      std::printf(__VA_ARGS__);                 \
      std::printf("\n");                        \
      ++failures;                               \
    }                                           \
  } while (0)

// Operands of a problem, dense and far apart, time first or batch first.
struct Problem {
  prnnAttention_t d = {};
  prnnSequence_t q, k, v, o, dq, dk, dv;
  prnnContext h;
  float *S0 = nullptr, *S1 = nullptr, *dS1 = nullptr, *dS0 = nullptr;
  static float* state(int i) { return reinterpret_cast<float*>(0x100000000000ull + 0x10000000000ull * i); }
  Problem(int B, int T, int H, int Hkv, int Dk, int Dv, prnnDataType_t type, bool batch_first = false) {
    d.B = B;
    d.T = T;
    d.H = H;
    d.Hkv = Hkv;
    d.Dk = Dk;
    d.Dv = Dv;
    d.type = type;
    d.scale = 1.f;
    d.log_decay = reinterpret_cast<float*>(0x1000);
    prnnSequence_t* all[] = {&q, &k, &v, &o, &dq, &dk, &dv};
    const int heads[] = {H, Hkv, Hkv, H, H, Hkv, Hkv}, size[] = {Dk, Dk, Dv, Dv, Dk, Dk, Dv};
    for (int i = 0; i < 7; ++i) {
      const int64_t row = (int64_t)heads[i] * size[i];
      all[i]->data = reinterpret_cast<void*>(0x200000000000ull + 0x40000000000ull * i);
      all[i]->head = size[i];
      all[i]->token = batch_first ? row : row * B;
      all[i]->batch = batch_first ? row * T : row;
    }
  }
  void packed(int64_t rows, int max_len) {
    d.offsets = reinterpret_cast<int32_t*>(0x2000);
    d.rows = rows;
    d.T = max_len;
    prnnSequence_t* all[] = {&q, &k, &v, &o, &dq, &dk, &dv};
    for (prnnSequence_t* s : all) s->token = s->head * (s == &k || s == &v || s == &dk || s == &dv ? d.Hkv : d.H);
  }
  prnnStatus_t forward() { return prnn_linear_attention(&h, &d, &q, &k, &v, S0, &o, S1, nullptr); }
  prnnStatus_t backward() {
    return prnn_linear_attention_backward(&h, &d, &q, &k, &v, S0, &o, dS1, &dq, &dk, &dv, dS0, nullptr);
  }
};

// The segments of a launch cover its sequences, in the integers the kernels use.
static void check_segments(const char* what) {
  const prnn::AttnArgs& a = args;
  CHECK(a.segments >= 1 && a.seg_tokens >= 64 && a.seg_tokens % 64 == 0, "%s: %d of %d", what, a.segments, a.seg_tokens);
  CHECK((int64_t)a.segments * a.seg_tokens >= a.T, "%s: %d of %d tokens for %d", what, a.segments, a.seg_tokens, a.T);
  CHECK((int64_t)a.segments * a.seg_tokens + 64 <= 0x7fffffffll, "%s: %d of %d tokens", what, a.segments, a.seg_tokens);
}

static void long_sequences() {
  const prnnDataType_t type = PRNN_DATA_BFLOAT;
  // a length beyond the rows there are is the rows
  for (int H : {1, 2, 16, 64, 256, 1000})
    for (int64_t rows : {200ll, 5000ll, 100000ll})
      for (int call = 0; call < 2; ++call) {
        int segments = 0, seg_tokens = 0;
        for (int max_len : {(int)rows, 0x7fffffff, 0x7fffffff - 63, 0x7ffe0000}) {
          Problem p(3, 1, H, H, 128, 128, type);
          p.packed(rows, max_len);
          const prnnStatus_t st = call == 0 ? p.forward() : p.backward();
          CHECK(st == PRNN_STATUS_SUCCESS, "%d heads, max_len %d: %d", H, max_len, (int)st);
          check_segments("packed");
          if (max_len == rows) {
            segments = args.segments;
            seg_tokens = args.seg_tokens;
          }
          CHECK(args.T == rows && args.segments == segments && args.seg_tokens == seg_tokens,
                "%d heads, %lld rows, max_len %d: T %d, %d segments of %d", H, (long long)rows, max_len, args.T,
                args.segments, args.seg_tokens);
        }
      }
  // the longest that a launch counts, and what is refused
  for (int T : {100, 1 << 20, 1 << 30, 0x7ffe0000})
    for (int H : {1, 3, 256}) {
      Problem p(1, T, H, H, 1, 1, type);
      CHECK(p.forward() == PRNN_STATUS_SUCCESS, "%d tokens", T);
      check_segments("whole");
    }
  for (int T : {0x7ffe0001, 0x7fffffff}) {
    Problem p(1, T, 1, 1, 1, 1, type);
    launches = 0;
    CHECK(p.forward() == PRNN_STATUS_NOT_SUPPORTED && launches == 0, "%d tokens", T);
    CHECK(p.backward() == PRNN_STATUS_NOT_SUPPORTED && launches == 0, "%d tokens", T);
  }
}

// Whether [p, p + bytes) lies in the workspace, apart from what else is there.
struct Piece {
  uint64_t at, bytes;
  const char* what;
};
static void check_pieces(const std::vector<Piece>& pieces) {
  for (size_t i = 0; i < pieces.size(); ++i) {
    CHECK(pieces[i].at >= kWork && pieces[i].at + pieces[i].bytes <= kWork + workspace, "%s", pieces[i].what);
    for (size_t j = 0; j < i; ++j)
      CHECK(pieces[i].at >= pieces[j].at + pieces[j].bytes || pieces[j].at >= pieces[i].at + pieces[i].bytes,
            "%s and %s", pieces[i].what, pieces[j].what);
  }
}

// dS0 in the place of dS1: one launch's jobs run in any order, so none may read
// what another one writes.
static void gradients_in_place() {
  for (int T : {0, 1, 200, 9000})
    for (int B : {1, 4, 64})
      for (int group : {1, 4})
        for (bool packed : {false, true})
          for (bool same : {false, true}) {
            Problem p(B, T, 8, 8 / group, 64, 96, PRNN_DATA_HALF);
            if (packed) p.packed(T, T);
            p.S0 = Problem::state(0);
            p.dS1 = Problem::state(1);
            p.dS0 = same ? p.dS1 : Problem::state(2);
            CHECK(p.backward() == PRNN_STATUS_SUCCESS, "%d tokens", T);
            for (int i = 0; i < 3; ++i)
              for (int j = 0; j < 3; ++j)
                CHECK(i == j || args.job[j].s_out == nullptr || args.job[i].s_in != args.job[j].s_out,
                      "%d tokens: job %d reads what job %d writes", T, i, j);
            CHECK(args.job[2].s_in == p.dS1 && args.job[2].s_out == p.dS0 && args.job[0].s_in == p.S0, "%d tokens", T);
            if (!same) {
              CHECK(args.keep == 0 && args.job[1].s_in == p.dS1, "%d tokens", T);
              continue;
            }
            const size_t n = (size_t)B * 8 * 64 * 96;
            CHECK(args.keep_from == p.dS1 && args.keep_to == args.job[1].s_in && args.keep == (int64_t)n, "%d tokens", T);
            std::vector<Piece> pieces = {{(uint64_t)args.keep_to, 4 * n, "states"}};
            if (group > 1 && T > 0) {
              const size_t rows = (size_t)T * (packed ? 1 : B) * 8;
              pieces.push_back({(uint64_t)args.job[1].o.p, rows * 64 * 4, "dk"});
              pieces.push_back({(uint64_t)args.job[2].o.p, rows * 96 * 4, "dv"});
            }
            check_pieces(pieces);
          }
}

// Shared heads: every head's own gradient lies in the workspace.  The kernels
// count a chunk's rows in 32 bits, below 2^30 bytes for up to 64 tokens, whatever
// number of heads and sequences there is.
static void shared_heads() {
  const struct {
    int B, T, H, Hkv, Dk, Dv;
  } shapes[] = {{2, 5, 4, 2, 8, 16},        {1, 300, 8, 1, 64, 64},     {2048, 64, 64, 32, 128, 96}, {4096, 64, 64, 32, 128, 128},
                {8192, 64, 32, 8, 128, 128}, {1024, 3, 1024, 1, 256, 1}, {1, 64, 1 << 20, 1 << 19, 256, 256}};
  for (const auto& s : shapes)
    for (bool packed : {false, true}) {
      Problem p(s.B, s.T, s.H, s.Hkv, s.Dk, s.Dv, PRNN_DATA_BFLOAT, true);
      for (prnnSequence_t* x : {&p.q, &p.k, &p.v, &p.o, &p.dq, &p.dk, &p.dv}) {  // heads outermost: any number of them
        x->token = x->head;
        x->batch = x->token * s.T;
        x->head = x->batch * s.B;
      }
      if (packed) {
        p.d.offsets = reinterpret_cast<int32_t*>(0x2000);
        p.d.rows = (int64_t)s.T * s.B;
      }
      const prnnStatus_t st = p.backward();
      CHECK(st == PRNN_STATUS_SUCCESS, "%d x %d heads: %d", s.B, s.H, (int)st);
      if (st != PRNN_STATUS_SUCCESS) continue;
      const uint64_t all = (uint64_t)s.T * s.B * s.H;
      check_pieces({{(uint64_t)args.job[1].o.p, all * s.Dk * 4, "dk"}, {(uint64_t)args.job[2].o.p, all * s.Dv * 4, "dv"}});
      for (int i : {1, 2}) {
        const prnn::AttnOperand& o = args.job[i].o;
        const int64_t D = i == 1 ? s.Dk : s.Dv;
        CHECK(args.job[i].o_f32 && o.group == 1 && o.token >= D, "%d x %d heads", s.B, s.H);
        CHECK(64 * o.token * 4 < 1ll << 30, "%d x %d heads: rows of %lld elements", s.B, s.H, (long long)o.token);
        // the last element is the last of the piece, and the axes do not meet
        const int64_t tokens = packed ? (int64_t)s.T * s.B : s.T, sequences = packed ? 1 : s.B;
        CHECK((tokens - 1) * o.token + (sequences - 1) * o.batch + (s.H - 1) * o.head + D == (int64_t)all * D,
              "%d x %d heads", s.B, s.H);
        // and the sums read what the job writes
        const prnn::AttnOperand& r = reduced.grad[i - 1].src;
        CHECK(r.p == o.p && r.token == o.token && (packed || r.batch == o.batch) && r.head == o.head, "%d x %d heads", s.B, s.H);
      }
    }
}

// Packed sequences: the workspace follows the rows there are, not the number of
// sequences times the longest one's segments.
static void packed_workspace() {
  const struct {
    int B;
    int64_t rows;
    int max_len, H, Hkv, D;
  } shapes[] = {{512, 32768, 32768, 16, 16, 128}, {512, 32768, 16384, 16, 16, 128}, {4096, 4096, 4096, 16, 4, 128},
                {4096, 4096, 1, 16, 16, 128},     {100000, 100000, 100000, 1, 1, 64}, {7, 3001, 1200, 16, 4, 64},
                {60, 60000, 60000, 4, 2, 256},    {1 << 22, 1 << 22, 1 << 22, 1, 1, 16}, {1 << 20, 900, 900, 1, 1, 64}, {3, 130, 130, 2, 2, 200}};
  for (const auto& s : shapes)
    for (bool states : {false, true})
      for (int call = 0; call < 2; ++call) {
        Problem p(s.B, 1, s.H, s.Hkv, s.D, s.D, PRNN_DATA_BFLOAT);
        p.packed(s.rows, s.max_len);
        if (states) {
          p.S0 = Problem::state(0);
          p.S1 = p.dS1 = Problem::state(1);
          p.dS0 = Problem::state(2);
        }
        workspace = 0;
        const prnnStatus_t st = call == 0 ? p.forward() : p.backward();
        CHECK(st == PRNN_STATUS_SUCCESS, "%d sequences: %d", s.B, (int)st);
        check_segments("packed");
        // q, k, v and o, or those with the gradients; fp32 gradients of shared heads
        const double row = s.D * 2.0, operands = s.rows * row * (call == 0 ? 2 * s.H + 2 * s.Hkv : 3 * s.H + 4 * s.Hkv);
        const double wide = call == 1 && s.H != s.Hkv ? 4.0 * s.rows * s.H * s.D * 2 + 512 : 0;
        CHECK(workspace - wide <= 8 * operands + 4096, "%d sequences of %lld rows: workspace of %zu bytes for %.0f", s.B,
              (long long)s.rows, workspace, operands);
        CHECK((int64_t)args.tiles * s.H * prnn::pieces(args) < 1ll << 24, "%d sequences: %d segments", s.B, args.segments);
        if (args.segments == 1) continue;
        // workgroups for a small multiple of the segments there can be
        CHECK(prnn::pieces(args) <= 4 * (s.rows / args.seg_tokens + s.B), "%d sequences: %lld pieces of %lld rows in segments of %d",
              s.B, (long long)prnn::pieces(args), (long long)s.rows, args.seg_tokens);
        // slots of sequences of any lengths that add up to the rows: apart, and inside
        for (int pattern = 0; pattern < 4; ++pattern)
          for (int i = 0; i < args.jobs; ++i) {
            const prnn::AttnJob& job = args.job[i];
            int64_t first = 0, next = 0, next_unit = 0;
            uint32_t seed = 1;
            for (int b = 0; b < s.B; ++b) {
              seed = seed * 1664525u + 1013904223u;
              const int64_t left = s.rows - first;
              int64_t len = pattern == 0 ? (b == s.B / 2 ? left : 0) : pattern == 1 ? args.seg_tokens * (seed >> 30)
                          : pattern == 2 ? args.seg_tokens + 1 : seed % (2 * s.rows / s.B + 2);
              len = std::min(len, std::min<int64_t>(left, args.T));
              const int64_t count = len > 0 ? (len - 1) / args.seg_tokens + 1 : 0;
              const int64_t used = count < 2 ? 0 : count - (job.s_in == nullptr ? 1 : 0);
              const int64_t at = prnn::first_slot(args, job, b, (uint32_t)(first / args.seg_tokens));
              CHECK(used == 0 || (at >= next && at + used <= prnn::slots(args)), "slots %lld + %lld of sequence %d",
                    (long long)at, (long long)used, b);
              if (used > 0) next = at + used;
              // found by their number, every segment has one of its own
              if (args.units > 0 && i == 0) {
                const int64_t unit = first / args.seg_tokens + b;
                CHECK(unit >= next_unit && unit + std::max<int64_t>(count, 1) <= args.units, "sequence %d", b);
                next_unit = unit + std::max<int64_t>(count, 1);
              }
              first += len;
            }
          }
        CHECK(prnn::slots(args) * s.H * args.tiles * args.dkp * 64 * args.nt * 4 * args.jobs <= (int64_t)workspace,
              "%d sequences", s.B);
      }
}

// Launches of more threads than 32 bits count are refused.
static void grids() {
  const struct {
    int B, H, Dk, Dv;
    bool step, whole;
  } shapes[] = {{64, 32, 128, 128, true, true},      {1 << 18, 63, 1, 1, true, true}, {1 << 19, 32, 1, 32, false, false},
                {1 << 18, 32, 1, 33, false, true},   {1 << 19, 15, 1, 64, true, true}, {1 << 19, 16, 1, 64, false, true},
                {1 << 16, 256, 1, 1, false, false},  {1 << 15, 255, 1, 256, false, true}};
  for (const auto& s : shapes) {
    Problem p(s.B, 1, s.H, s.H, s.Dk, s.Dv, PRNN_DATA_BFLOAT, true);
    p.S0 = Problem::state(0);
    p.S1 = Problem::state(1);
    launches = steps = 0;
    const bool step = prnn_linear_attention_step(&p.h, &p.d, &p.q, &p.k, &p.v, p.S0, &p.o, p.S1, nullptr) == PRNN_STATUS_SUCCESS;
    CHECK(step == s.step && steps == (s.step ? 1 : 0), "a step of %d x %d heads of %d", s.B, s.H, s.Dv);
    const prnnStatus_t st = p.forward();
    CHECK(st == (s.whole ? PRNN_STATUS_SUCCESS : PRNN_STATUS_NOT_SUPPORTED) && launches == (s.whole ? 1 : 0),
          "%d x %d heads of %d: %d", s.B, s.H, s.Dv, (int)st);
  }
}

// Spans past 64 bits do not wrap into small ones: an output in the place of a far
// row of an input, or the other way round, is refused.
static void spans() {
  const int B = (1 << 23) + 1;
  const int64_t stride = 1ll << 40;  // (B - 1) strides are 2^64 bytes
  for (int which = 0; which < 3; ++which) {
    Problem p(B, 1, 1, 1, 8, 8, PRNN_DATA_HALF, true);
    p.S0 = Problem::state(0);
    p.S1 = Problem::state(1);
    prnnSequence_t *far = which == 0 ? &p.q : which == 1 ? &p.v : &p.o, *near = which == 2 ? &p.k : &p.o;
    far->batch = stride;
    far->data = reinterpret_cast<void*>(0x10000);
    near->data = static_cast<char*>(far->data) + 5 * 2 * stride;
    CHECK(p.forward() == PRNN_STATUS_BAD_PARAM, "forward %d", which);
    CHECK(prnn_linear_attention_step(&p.h, &p.d, &p.q, &p.k, &p.v, p.S0, &p.o, p.S1, nullptr) == PRNN_STATUS_BAD_PARAM,
          "step %d", which);
  }
  prnnContext h;
  float *x = reinterpret_cast<float*>(0x10000), *y = x + 5 * stride;
  for (const int M : {4, 6, (1 << 22) + 1}) {
    const prnnStatus_t want = M > 5 ? PRNN_STATUS_BAD_PARAM : PRNN_STATUS_SUCCESS;
    CHECK(prnn_layer_norm(&h, M, 4, PRNN_DATA_FLOAT, x, stride, PRNN_DATA_FLOAT, nullptr, nullptr, 0.f, y, 4, nullptr, nullptr,
                          nullptr) == want, "%d rows", M);
  }
}

// Layer norm counts columns in 31 bits.
static void wide_norms() {
  prnnContext h;
  float *x = Problem::state(0), *y = Problem::state(1), *m = Problem::state(2), *w = Problem::state(3);
  const prnnDataType_t f = PRNN_DATA_FLOAT;
  for (int N : {1, 12345, 0x7fffffff - 1023, 0x7fffffff - 1022, 0x7fffffff - 255, 0x7fffffff}) {
    const prnnStatus_t want = N > 0x7fffffff - 1023 ? PRNN_STATUS_NOT_SUPPORTED : PRNN_STATUS_SUCCESS;
    CHECK(prnn_layer_norm(&h, 1, N, f, x, N, f, nullptr, nullptr, 0.f, y, N, nullptr, nullptr, nullptr) == want, "%d columns", N);
    CHECK(prnn_layer_norm_backward(&h, 1, N, f, y, N, x, N, m, m + 1, f, nullptr, w, N, nullptr, nullptr, nullptr) == want,
          "%d columns", N);
  }
}

int main(int argc, char** argv) {
  const char* const which = argc > 1 ? argv[1] : "";
  if (!std::strcmp(which, "long sequences")) long_sequences();
  else if (!std::strcmp(which, "gradients in place")) gradients_in_place();
  else if (!std::strcmp(which, "shared heads")) shared_heads();
  else if (!std::strcmp(which, "packed workspace")) packed_workspace();
  else if (!std::strcmp(which, "wide norms")) wide_norms();
  else if (!std::strcmp(which, "grids")) grids();
  else if (!std::strcmp(which, "spans")) spans();
  else ++failures;
  if (failures == 0) std::printf("all checks passed\n");
  return failures == 0 ? 0 : 1;
}
