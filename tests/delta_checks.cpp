// Calls the gated delta rule and rms norm with stand-ins for the handle and the
// launches: invalid arguments must be refused, and what would have been launched
// must fit its grids and its workspace (see test_delta_checks.py).  Device
// pointers are numbers: nothing here reads them.
#include <algorithm>
#include <cstdio>
#include <cstring>
#include <random>
#include <vector>

#include "delta_rule.h"
#include "rms_norm.h"

struct prnnContext {
  bool failed = false;
  bool no_memory = false;
};

using namespace prnn;

static const uintptr_t kWork = 0x700000000000ull;
static int launches = 0, reductions = 0;
static size_t workspace = 0;
static DeltaArgs args;  // of the last launch

namespace prnn {
bool handle_failed(prnnContext* h) {
  const bool f = h->failed;
  h->failed = false;
  return f;
}
int handle_compute_units(const prnnContext*) { return 256; }
bool handle_logs(const prnnContext*) { return false; }
prnnStatus_t handle_workspace(prnnContext* h, size_t bytes, hipStream_t, void** out) {
  if (h->no_memory) return PRNN_STATUS_ALLOC_FAILED;
  workspace = bytes;
  *out = reinterpret_cast<void*>(kWork);
  return PRNN_STATUS_SUCCESS;
}
hipError_t launch_delta(const DeltaArgs& a, prnnDataType_t, bool, hipStream_t) {
  args = a;
  ++launches;
  return hipSuccess;
}
hipError_t launch_delta_step(const DeltaStepArgs&, prnnDataType_t, hipStream_t) {
  ++launches;
  return hipSuccess;
}
hipError_t launch_attention_reduce(const AttnReduceArgs&, prnnDataType_t, hipStream_t) {
  ++reductions;
  return hipSuccess;
}
hipError_t launch_rms_norm(const RmsArgs&, prnnDataType_t, prnnDataType_t, bool, hipStream_t) {
  ++launches;
  return hipSuccess;
}
int rms_norm_backward_grid(const RmsArgs& a, prnnDataType_t, int) { return a.M > 0 ? 4 : 0; }
hipError_t launch_rms_norm_backward(const RmsArgs&, prnnDataType_t, prnnDataType_t, int, hipStream_t) {
  ++launches;
  return hipSuccess;
}
}  // namespace prnn
extern "C" hipError_t hipGetLastError() { return hipSuccess; }

static int failures = 0;
static void expect(prnnStatus_t got, prnnStatus_t want, bool enqueued, const char* what) {
  if (got != want || (launches > 0) != enqueued) {
    std::printf("%s: status %d, want %d; %d launches\n", what, (int)got, (int)want, launches);
    ++failures;
  }
  launches = 0;
}
#define CHECK(ok, ...)            \
  do {                            \
    if (!(ok)) {                  \
      std::printf("%s: ", #ok);   \
      std::printf(__VA_ARGS__);   \
      std::printf("\n");          \
      ++failures;                 \
    }                             \
  } while (0)

template <class T>
static T* at(uintptr_t p) {
  return reinterpret_cast<T*>(p);
}

// A valid problem, from which each check departs.  Dense, time first, far apart.
struct Case {
  prnnContext h;
  prnnDeltaRule_t d;
  prnnSequence_t q, k, v, g, beta, o, dq, dk, dv, dg, dbeta;
  float *S0, *S1;
  explicit Case(int B = 3, int T = 5, int H = 4, int Hk = 2, int Dk = 8, int Dv = 6, prnnDataType_t type = PRNN_DATA_HALF) {
    std::memset(&d, 0, sizeof(d));
    d.B = B;
    d.T = T;
    d.H = H;
    d.Hk = Hk;
    d.Dk = Dk;
    d.Dv = Dv;
    d.type = type;
    d.scale = 0.5f;
    prnnSequence_t* x[] = {&q, &k, &v, &g, &beta, &o, &dq, &dk, &dv, &dg, &dbeta};
    const int heads[] = {Hk, Hk, H, H, H, H, Hk, Hk, H, H, H}, size[] = {Dk, Dk, Dv, 1, 1, Dv, Dk, Dk, Dv, 1, 1};
    for (int i = 0; i < 11; ++i) {
      const int64_t row = (int64_t)heads[i] * size[i];
      *x[i] = {at<void>(0x200000000000ull + 0x40000000000ull * i), row * B, row, size[i]};
    }
    S0 = at<float>(0x100000000000ull);
    S1 = at<float>(0x110000000000ull);
  }
  void packed(int64_t rows) {
    d.offsets = at<int32_t>(0x1000);
    d.rows = rows;
    for (prnnSequence_t* x : {&q, &k, &v, &g, &beta, &o, &dq, &dk, &dv, &dg, &dbeta}) x->token = x->batch;
  }
  prnnStatus_t forward() { return prnn_gated_delta_rule(&h, &d, &q, &k, &v, &g, &beta, S0, &o, S1, nullptr); }
  prnnStatus_t step() { return prnn_gated_delta_rule_step(&h, &d, &q, &k, &v, &g, &beta, S0, &o, S1, nullptr); }
  prnnStatus_t backward() {
    return prnn_gated_delta_rule_backward(&h, &d, &q, &k, &v, &g, &beta, nullptr, &o, S0, &dq, &dk, &dv, &dg, &dbeta, S1, nullptr);
  }
};

// Departs by `change`; the forward, backward and (where it applies) step calls
// must all answer `want`.
template <class F>
static void all(const char* what, prnnStatus_t want, F change, bool step = true, bool enqueued = false) {
  for (int call = 0; call < (step ? 3 : 2); ++call) {
    Case c;
    change(c);
    expect(call == 0 ? c.forward() : call == 1 ? c.backward() : c.step(), want, enqueued, what);
  }
}

static void delta_refusals() {
  const prnnStatus_t ok = PRNN_STATUS_SUCCESS, bad = PRNN_STATUS_BAD_PARAM, no = PRNN_STATUS_NOT_SUPPORTED;
  all("as it is", ok, [](Case&) {}, true, true);
  {
    Case c;
    expect(prnn_gated_delta_rule(nullptr, &c.d, &c.q, &c.k, &c.v, &c.g, &c.beta, c.S0, &c.o, c.S1, nullptr), bad, false, "no handle");
    expect(prnn_gated_delta_rule(&c.h, nullptr, &c.q, &c.k, &c.v, &c.g, &c.beta, c.S0, &c.o, c.S1, nullptr), bad, false, "no rule");
    expect(prnn_gated_delta_rule(&c.h, &c.d, nullptr, &c.k, &c.v, &c.g, &c.beta, c.S0, &c.o, c.S1, nullptr), bad, false, "no q");
    expect(prnn_gated_delta_rule(&c.h, &c.d, &c.q, &c.k, &c.v, &c.g, nullptr, c.S0, &c.o, c.S1, nullptr), bad, false, "no beta");
    expect(prnn_gated_delta_rule(&c.h, &c.d, &c.q, &c.k, &c.v, nullptr, &c.beta, c.S0, &c.o, c.S1, nullptr), ok, true, "no decay");
    expect(prnn_gated_delta_rule_backward(&c.h, &c.d, &c.q, &c.k, &c.v, nullptr, &c.beta, nullptr, &c.o, nullptr, &c.dq, &c.dk,
                                          &c.dv, nullptr, &c.dbeta, nullptr, nullptr), ok, true, "gradients without decay");
    expect(prnn_gated_delta_rule_backward(&c.h, &c.d, &c.q, &c.k, &c.v, &c.g, &c.beta, nullptr, &c.o, nullptr, &c.dq, &c.dk,
                                          nullptr, &c.dg, &c.dbeta, nullptr, nullptr), bad, false, "no dv");
  }
  all("failed run", PRNN_STATUS_EXECUTION_FAILED, [](Case& c) { c.h.failed = true; });
  all("B < 0", bad, [](Case& c) { c.d.B = -1; });
  all("B = 0", ok, [](Case& c) { c.d.B = 0; });
  all("T < 0", bad, [](Case& c) { c.d.T = -1; }, false);
  all("H = 0", bad, [](Case& c) { c.d.H = 0; });
  all("Hk = 0", bad, [](Case& c) { c.d.Hk = 0; });
  all("H not a multiple of Hk", bad, [](Case& c) { c.d.Hk = 3; });
  all("Dk = 0", bad, [](Case& c) { c.d.Dk = 0; });
  all("Dk = 257", bad, [](Case& c) { c.d.Dk = 257; });
  all("Dv = -3", bad, [](Case& c) { c.d.Dv = -3; });
  all("Dv = 257", bad, [](Case& c) { c.d.Dv = 257; });
  all("8-bit values", bad, [](Case& c) { c.d.type = PRNN_DATA_E4M3; });
  all("type", bad, [](Case& c) { c.d.type = PRNN_DATA_MAX_ENUM; });
  all("no k", bad, [](Case& c) { c.k.data = nullptr; });
  all("q at an odd byte", bad, [](Case& c) { c.q.data = at<void>(0x200000000001ull); });
  all("beta at 2 bytes", bad, [](Case& c) { c.beta.data = at<void>(0x300000000002ull); });
  all("fp32 at 2 bytes", bad, [](Case& c) {
    c.d.type = PRNN_DATA_FLOAT;
    c.v.data = at<void>(0x280000000002ull);
  });
  all("negative head stride", bad, [](Case& c) { c.q.head = -8; });
  all("negative token stride", bad, [](Case& c) { c.k.token = -8; }, false);
  all("negative batch stride", bad, [](Case& c) { c.beta.batch = -1; });
  all("a stride past every memory", bad, [](Case& c) { c.q.head = 1ll << 50; });
  all("state at 2 bytes", bad, [](Case& c) { c.S0 = at<float>(0x100000000002ull); });
  all("states overlap in part", bad, [](Case& c) { c.S1 = c.S0 + 4; });
  all("states in place", ok, [](Case& c) { c.S1 = c.S0; }, true, true);
  all("lengths and offsets", bad, [](Case& c) {
    c.packed(15);
    c.d.lengths = at<int32_t>(0x2000);
  }, false);
  all("rows < 0", bad, [](Case& c) { c.packed(-1); }, false);
  all("offsets at 2 bytes", bad, [](Case& c) {
    c.packed(15);
    c.d.offsets = at<int32_t>(0x1002);
  }, false);
  all("packed", ok, [](Case& c) { c.packed(11); }, false, true);
  all("lengths", ok, [](Case& c) { c.d.lengths = at<int32_t>(0x2000); }, false, true);
  all("o's heads overlap", bad, [](Case& c) { c.dv.head = c.o.head = 5; });
  all("o's batch rows coincide", bad, [](Case& c) { c.dv.batch = c.o.batch = 0; });
  all("token stride past 2^23", no, [](Case& c) { c.q.token = (1 << 23) + 1; }, false);
  all("too many states", no, [](Case& c) { c.d.B = 1 << 23; });
  all("more rows than 31 bits count", no, [](Case& c) { c.packed(1ll << 31); }, false);
  all("an input repeated by strides of 0", ok, [](Case& c) { c.k.batch = c.k.token = c.beta.head = c.g.token = 0; }, true, true);
  {
    Case c;
    c.o.data = c.q.data;
    expect(c.forward(), bad, false, "o over q");
    c = Case();
    c.o.data = c.beta.data;
    expect(c.forward(), bad, false, "o over beta");
    c = Case();
    c.o.data = c.S0;
    expect(c.forward(), bad, false, "o over the states");
    c = Case();
    c.S1 = static_cast<float*>(c.k.data);
    expect(c.forward(), bad, false, "the final states over k");
    expect(c.step(), bad, false, "the final states over k");
    c = Case();
    c.S1 = nullptr;
    expect(c.step(), bad, false, "a step without states");
    c = Case();
    c.S0 = nullptr;
    expect(c.step(), bad, false, "a step without states");
    c = Case();
    c.dk.data = c.dq.data;
    expect(c.backward(), bad, false, "dk over dq");
    c = Case();
    c.dg.data = c.dbeta.data;
    expect(c.backward(), bad, false, "dlog_decay over dbeta");
    c = Case();
    c.dbeta.data = c.beta.data;
    expect(c.backward(), bad, false, "dbeta over beta");
    c = Case();
    c.d.offsets = at<int32_t>(0x100000000000ull);
    c.d.rows = 15;
    expect(c.backward(), ok, true, "offsets and dS1 read from one place");
    c.S1 = c.S0;
    expect(c.backward(), bad, false, "dS0 over the offsets");
    c = Case();
    c.h.no_memory = true;
    expect(c.forward(), PRNN_STATUS_ALLOC_FAILED, false, "no memory");
    expect(c.backward(), PRNN_STATUS_ALLOC_FAILED, false, "no memory");
    // q, k, v and o as slices of the rows of one buffer, fp16: 16 + 16 + 24 + 24 elements
    c = Case();
    prnnSequence_t* slices[] = {&c.q, &c.k, &c.v, &c.o};
    const int offset[] = {0, 16, 32, 56};
    for (int i = 0; i < 4; ++i) {
      slices[i]->data = at<void>(0x200000000000ull + 2 * offset[i]);
      slices[i]->batch = 80;
      slices[i]->token = 80 * 3;
    }
    expect(c.forward(), ok, true, "slices of one buffer");
    c.o.data = at<void>(0x200000000000ull + 2 * 55);
    expect(c.forward(), bad, false, "slices that meet");
    c = Case();
    c.d.T = 0;
    c.q.data = c.k.data = c.v.data = c.g.data = c.beta.data = c.o.data = nullptr;
    expect(c.forward(), ok, true, "T = 0 passes the states on");
    c.S1 = nullptr;
    expect(c.forward(), ok, false, "T = 0 without final states");
  }
}

// Whether [p, p + bytes) lies in the workspace.
static bool inside(const void* p, size_t bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(p);
  return bytes == 0 || (x >= kWork && x + bytes <= kWork + workspace);
}

// What sequences [first, first + len) use of the workspace, as the kernels number it:
// no two share a chunk, a group or a segment whose state is kept, and all are inside.
static void check_plan(Case& c, const std::vector<int64_t>& offsets, bool backward) {
  const prnnStatus_t st = backward ? c.backward() : c.forward();
  CHECK(st == PRNN_STATUS_SUCCESS, "status %d", (int)st);
  if (st != PRNN_STATUS_SUCCESS) return;
  const DeltaArgs& a = args;
  const bool packed = c.d.offsets != nullptr;
  int64_t chunk = 0, group = 0, part = 0, unit = 0;
  const int64_t tokens = (int64_t)a.seg_chunks * kDeltaChunk;
  for (int b = 0; b < a.B; ++b) {
    const int64_t first = packed ? offsets[b] : 0, len = packed ? std::min<int64_t>(a.T, offsets[b + 1] - first) : a.T;
    const int64_t n = (len + kDeltaChunk - 1) / kDeltaChunk, groups = (n + a.group - 1) / a.group,
                  segments = std::max<int64_t>(1, (n + a.seg_chunks - 1) / a.seg_chunks);
    const int64_t c0 = packed ? first / kDeltaChunk + b : (int64_t)b * a.chunks;
    const int64_t g0 = packed ? first / (a.group * kDeltaChunk) + b : (int64_t)b * a.groups;
    if (n > 0) {
      CHECK(c0 >= chunk && c0 + n <= a.slots, "chunks of sequence %d", b);
      CHECK(g0 >= group && g0 + groups <= a.group_slots, "groups of sequence %d", b);
      chunk = c0 + n;
      group = g0 + groups;
    }
    CHECK(segments <= a.segments, "segments of sequence %d", b);
    if (a.seg_slots > 0) {
      // (the states behind all but the last segment are kept, and the first one's start at the
      // first one's place)
      const int64_t p0 = packed ? first / tokens : (int64_t)b * a.segments;
      if (segments > 1) {
        CHECK(p0 >= part && p0 + segments <= a.seg_slots, "segments of sequence %d", b);
        part = p0 + segments - 1;
      }
      if (packed) {
        const int64_t u0 = first / tokens + b;
        CHECK(u0 >= unit && u0 + segments <= a.units, "units of sequence %d", b);
        unit = u0 + segments;
      }
    } else {
      CHECK(a.units == 0 && segments == 1, "sequence %d", b);
    }
  }
  CHECK(inside(a.blocks, (size_t)a.slots * a.H * kDeltaBlock), "blocks");
  const size_t parts = (size_t)a.seg_slots * a.H;
  CHECK(a.pitch >= a.Dv && a.pitch % 4 == 0 && a.move_pitch >= a.Dk && a.move_pitch % 4 == 0, "pitches");
  if (parts > 0) {
    CHECK(inside(a.ends, parts * a.Dk * a.pitch * 4) && inside(a.firsts, parts * a.Dk * a.pitch * 4) &&
              inside(a.moves, parts * a.Dk * a.move_pitch * 4), "segments");
    CHECK(a.firsts >= a.ends + parts * a.Dk * a.pitch && a.moves >= a.firsts + parts * a.Dk * a.pitch, "segments");
  }
  if (backward && a.slots > 0) {
    const size_t groups = (size_t)a.group_slots * a.H, rows = groups * a.group * kDeltaChunk * a.pitch,
                 states = groups * a.Dk * a.pitch;
    CHECK(inside(a.x, rows * 4) && inside(a.w, rows * 4) && inside(a.S, states * 4) && inside(a.R, states * 4), "gradients");
    CHECK((char*)a.x >= a.blocks + (size_t)a.slots * a.H * kDeltaBlock && a.w >= a.x + rows && a.S >= a.w + rows &&
              a.R >= a.S + states, "gradients");
    CHECK(parts == 0 || a.ends >= a.R + states, "gradients");
    if (a.H > c.d.Hk) {
      const size_t heads = (size_t)(packed ? a.rows : (int64_t)a.T * a.B) * a.H * a.Dk;
      const float *dq = static_cast<const float*>(a.dq.p), *dk = static_cast<const float*>(a.dk.p);
      CHECK(a.qk_f32 && inside(dq, heads * 4) && inside(dk, heads * 4) && dk >= dq + heads, "shared heads");
      CHECK(dq >= a.R + states && (parts == 0 || dq >= a.moves + parts * a.Dk * a.move_pitch), "shared heads");
    }
  }
}

static void delta_plans() {
  std::mt19937 rng(5);
  const prnnDataType_t types[] = {PRNN_DATA_FLOAT, PRNN_DATA_HALF, PRNN_DATA_BFLOAT};
  int split = 0, splits = 0;
  for (int i = 0; i < 4000; ++i) {
    const int B = 1 + rng() % 9, Hk = 1 + rng() % 4, H = Hk * (1 + rng() % 3), Dk = 1 + rng() % 256, Dv = 1 + rng() % 256;
    const int T = rng() % 2 ? rng() % 300 : rng() % 40000;
    Case c(B, T, H, Hk, Dk, Dv, types[rng() % 3]);
    std::vector<int64_t> offsets(1, rng() % 70);
    if (rng() % 2) {
      for (int b = 0; b < B; ++b) offsets.push_back(offsets.back() + (rng() % 4 == 0 ? rng() % 3 : rng() % (T + 1)));
      c.packed(offsets.back() + rng() % 50);
    }
    for (int back = 0; back < 2; ++back) {
      check_plan(c, offsets, back);
      splits += args.segments > 1;
      split += args.seg_slots > 0 && args.units > 0;
    }
  }
  CHECK(splits > 500 && split > 200, "%d calls split, %d of packed rows", splits, split);
  // the longest sequences and the most of them: refused, or within the grids
  for (int type = 0; type < 2; ++type)
    for (int64_t T : {1ll << 20, 1ll << 24, 1ll << 28, 0x7ffe0000ll})
      for (int B : {1, 7, 4096, 1 << 20})
        for (int H : {1, 16}) {
          Case c(B, (int)T, H, 1, 64, 256, types[type]);
          for (prnnSequence_t* x : {&c.q, &c.k, &c.v, &c.g, &c.beta, &c.o, &c.dq, &c.dk, &c.dv, &c.dg, &c.dbeta}) x->batch = x->token, x->token /= B;
          c.d.B = B;
          for (prnnSequence_t* x : {&c.q, &c.k, &c.v, &c.g, &c.beta, &c.o, &c.dq, &c.dk, &c.dv, &c.dg, &c.dbeta}) x->batch = x->token * T;
          launches = 0;
          const prnnStatus_t st = c.forward();
          if (st != PRNN_STATUS_SUCCESS) {
            CHECK(launches == 0 && (st == PRNN_STATUS_NOT_SUPPORTED || st == PRNN_STATUS_BAD_PARAM), "T %lld B %d: %d", (long long)T, B, (int)st);
            continue;
          }
          const double pieces = args.units > 0 ? (double)args.units * H : (double)B * H * args.segments;
          CHECK((double)args.slots * H <= 4. * kMaxWorkgroups && pieces * args.tiles <= kMaxWorkgroups, "T %lld B %d", (long long)T, B);
        }
}

static void rms_refusals() {
  const prnnStatus_t ok = PRNN_STATUS_SUCCESS, bad = PRNN_STATUS_BAD_PARAM, no = PRNN_STATUS_NOT_SUPPORTED;
  struct Norm {
    prnnContext h;
    int64_t M = 5;
    int N = 200;
    prnnDataType_t type = PRNN_DATA_HALF, ptype = PRNN_DATA_FLOAT, ytype = PRNN_DATA_HALF;
    char *x = at<char>(0x100000), *res = at<char>(0x200000), *w = at<char>(0x300000), *sum = at<char>(0x400000), *y = at<char>(0x500000);
    int64_t ldx = 200, ldr = 200, lds = 200, ldy = 200;
    float *scales = nullptr, *rstd = at<float>(0x610000), eps = 1e-6f;
    int group = 0;
    prnnStatus_t run() {
      return prnn_rms_norm(&h, M, N, type, x, ldx, res, ldr, ptype, w, eps, sum, lds, ytype, y, ldy, scales, group, rstd, nullptr);
    }
    void eight(int g) {
      ytype = PRNN_DATA_E4M3;
      scales = at<float>(0x600000);
      group = g;
    }
  };
  auto norm = [&](const char* what, prnnStatus_t want, bool enqueued, auto change) {
    Norm n;
    change(n);
    expect(n.run(), want, enqueued, what);
  };
  norm("norm", ok, true, [](Norm&) {});
  norm("norm: x alone", ok, true, [](Norm& n) {
    n.res = n.w = n.sum = nullptr;
    n.rstd = nullptr;
  });
  norm("norm: 8 bits, 128 columns a scale", ok, true, [](Norm& n) { n.eight(128); });
  norm("norm: 8 bits, a row a scale", ok, true, [](Norm& n) { n.eight(0); });
  norm("norm: 8 bits at odd bytes", ok, true, [](Norm& n) {
    n.eight(0);
    ++n.y;
  });
  norm("norm: sum over the residual, y over x", ok, true, [](Norm& n) {
    n.sum = n.res;
    n.y = n.x;
  });
  norm("norm: sum over x, y over the residual", ok, true, [](Norm& n) {
    n.sum = n.x;
    n.y = n.res;
  });
  norm("norm: halves of one buffer", ok, true, [](Norm& n) {
    n.y = n.x + 400;
    n.ldx = n.ldy = 400;
  });
  norm("norm: no rows", ok, false, [](Norm& n) {
    n.M = 0;
    n.x = n.y = nullptr;
  });
  norm("norm: M < 0", bad, false, [](Norm& n) { n.M = -1; });
  norm("norm: N = 0", bad, false, [](Norm& n) { n.N = 0; });
  norm("norm: too many rows", no, false, [](Norm& n) { n.M = 1ll << 31; });
  norm("norm: too many columns", no, false, [](Norm& n) {
    n.N = 0x7fffffff;
    n.ldx = n.ldy = n.ldr = n.lds = 1ll << 31;
  });
  norm("norm: no x", bad, false, [](Norm& n) { n.x = nullptr; });
  norm("norm: no y", bad, false, [](Norm& n) { n.y = nullptr; });
  norm("norm: ldx < N", bad, false, [](Norm& n) { n.ldx = 199; });
  norm("norm: ldr < N", bad, false, [](Norm& n) { n.ldr = 199; });
  norm("norm: lds < N", bad, false, [](Norm& n) { n.lds = 199; });
  norm("norm: ldy < N", bad, false, [](Norm& n) { n.ldy = 199; });
  norm("norm: type", bad, false, [](Norm& n) { n.type = n.ytype = PRNN_DATA_E4M3; });
  norm("norm: another type's y", bad, false, [](Norm& n) { n.ytype = PRNN_DATA_BFLOAT; });
  norm("norm: bf16 weights of fp16", bad, false, [](Norm& n) { n.ptype = PRNN_DATA_BFLOAT; });
  norm("norm: eps < 0", bad, false, [](Norm& n) { n.eps = -1.f; });
  norm("norm: eps NaN", bad, false, [](Norm& n) { n.eps = __builtin_nanf(""); });
  norm("norm: x at an odd byte", bad, false, [](Norm& n) { ++n.x; });
  norm("norm: weights at 2 bytes", bad, false, [](Norm& n) { n.w += 2; });
  norm("norm: scales without 8 bits", bad, false, [](Norm& n) { n.scales = at<float>(0x600000); });
  norm("norm: 8 bits without scales", bad, false, [](Norm& n) {
    n.eight(0);
    n.scales = nullptr;
  });
  norm("norm: groups without 8 bits", bad, false, [](Norm& n) { n.group = 128; });
  norm("norm: groups of 64", bad, false, [](Norm& n) { n.eight(64); });
  norm("norm: 8 bits over x", bad, false, [](Norm& n) {
    n.eight(0);
    n.y = n.x;
  });
  norm("norm: y over x in part", bad, false, [](Norm& n) { n.y = n.x + 2; });
  norm("norm: y over x at another stride", bad, false, [](Norm& n) {
    n.y = n.x;
    n.ldy = 201;
  });
  norm("norm: y over the sum", bad, false, [](Norm& n) { n.y = n.sum; });
  norm("norm: y over the weights", bad, false, [](Norm& n) { n.y = n.w; });
  norm("norm: rstd over x", bad, false, [](Norm& n) { n.rstd = at<float>(0x100000); });
  norm("norm: rstd over the scales", bad, false, [](Norm& n) {
    n.eight(128);
    n.rstd = n.scales + 9;
  });
  norm("norm: the last row's second scale over rstd", bad, false, [](Norm& n) {
    n.eight(128);
    n.scales = n.rstd - 9;
  });
  norm("norm: failed run", PRNN_STATUS_EXECUTION_FAILED, false, [](Norm& n) { n.h.failed = true; });
  expect(prnn_rms_norm(nullptr, 5, 8, PRNN_DATA_FLOAT, at<void>(0x1000), 8, nullptr, 0, PRNN_DATA_FLOAT, nullptr, 0.f, nullptr, 0,
                       PRNN_DATA_FLOAT, at<void>(0x2000), 8, nullptr, 0, nullptr, nullptr), bad, false, "norm: no handle");

  struct Back {
    prnnContext h;
    int64_t M = 5, lddy = 7, ldx = 7, ldds = 7, lddx = 7;
    int N = 7;
    prnnDataType_t type = PRNN_DATA_FLOAT, ptype = PRNN_DATA_FLOAT;
    float *dy = at<float>(0x100000), *x = at<float>(0x200000), *rstd = at<float>(0x300000), *w = at<float>(0x400000),
          *ds = at<float>(0x500000), *dx = at<float>(0x600000), *dw = at<float>(0x700000);
    prnnStatus_t run() { return prnn_rms_norm_backward(&h, M, N, type, dy, lddy, x, ldx, rstd, ptype, w, ds, ldds, dx, lddx, dw, nullptr); }
  };
  auto back = [&](const char* what, prnnStatus_t want, bool enqueued, auto change) {
    Back n;
    change(n);
    expect(n.run(), want, enqueued, what);
  };
  back("backward", ok, true, [](Back&) {});
  back("backward over dy", ok, true, [](Back& n) { n.dx = n.dy; });
  back("backward over x", ok, true, [](Back& n) { n.dx = n.x; });
  back("backward over dsum", ok, true, [](Back& n) { n.dx = n.ds; });
  back("backward: weights only", ok, true, [](Back& n) { n.dx = nullptr; });
  back("backward: dx only", ok, true, [](Back& n) { n.dw = nullptr; });
  back("backward of nothing", ok, false, [](Back& n) { n.dw = n.dx = nullptr; });
  back("backward of no rows", ok, true, [](Back& n) {
    n.M = 0;
    n.dy = n.x = n.rstd = nullptr;
  });
  back("backward: no dy", bad, false, [](Back& n) { n.dy = nullptr; });
  back("backward: no rstd", bad, false, [](Back& n) { n.rstd = nullptr; });
  back("backward: lddy < N", bad, false, [](Back& n) { n.lddy = 6; });
  back("backward: lddx < N", bad, false, [](Back& n) { n.lddx = 6; });
  back("backward: ldds < N", bad, false, [](Back& n) { n.ldds = 6; });
  back("backward: fp16 weights of fp32", bad, false, [](Back& n) { n.ptype = PRNN_DATA_HALF; });
  back("backward: dx over x in part", bad, false, [](Back& n) { n.dx = n.x + 1; });
  back("backward: dx over rstd", bad, false, [](Back& n) { n.dx = n.rstd; });
  back("backward: dweight over x", bad, false, [](Back& n) { n.dw = n.x; });
  back("backward: dweight over dx", bad, false, [](Back& n) { n.dw = n.dx; });
  back("backward: dweight over the weights", bad, false, [](Back& n) { n.dw = n.w; });
  back("backward: no memory", PRNN_STATUS_ALLOC_FAILED, false, [](Back& n) { n.h.no_memory = true; });
  back("backward: failed run", PRNN_STATUS_EXECUTION_FAILED, false, [](Back& n) { n.h.failed = true; });
}

int main(int argc, char** argv) {
  const char* what = argc > 1 ? argv[1] : "";
  if (!std::strcmp(what, "delta refusals")) delta_refusals();
  else if (!std::strcmp(what, "delta plans")) delta_plans();
  else if (!std::strcmp(what, "rms refusals")) rms_refusals();
  else return 2;
  if (failures == 0) std::printf("all checks passed\n");
  return failures == 0 ? 0 : 1;
}
