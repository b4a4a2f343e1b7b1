// Calls the linear-attention and layer-norm entry points with stand-ins for
// the handle and the launches (see test_sequence_checks.py).  Device pointers
// are numbers: nothing here reads them.
#include <cstdio>
#include <cstdlib>

#include "sequence.h"

struct prnnContext {
  bool failed = false;
  bool no_memory = false;
};

static int launches = 0;
static size_t workspace = 0;

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
  *out = reinterpret_cast<void*>(0x7000000000ull);
  return PRNN_STATUS_SUCCESS;
}
static hipError_t count() {
  ++launches;
  return hipSuccess;
}
size_t plan_attention(AttnArgs* a, prnnDataType_t, int) {
  a->tiles = a->segments = 2;
  return 1000;
}
hipError_t launch_attention(const AttnArgs&, prnnDataType_t, hipStream_t) { return count(); }
hipError_t launch_attention_reduce(const AttnReduceArgs&, prnnDataType_t, hipStream_t) { return count(); }
hipError_t launch_attention_step(const AttnStepArgs&, prnnDataType_t, hipStream_t) { return count(); }
hipError_t launch_layer_norm(const NormArgs&, prnnDataType_t, prnnDataType_t, hipStream_t) { return count(); }
int layer_norm_backward_grid(const NormArgs& a, prnnDataType_t, int) { return a.M > 0 ? 4 : 0; }
hipError_t launch_layer_norm_backward(const NormArgs&, prnnDataType_t, prnnDataType_t, int, hipStream_t) { return count(); }
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

template <class T>
static T* at(uintptr_t p) {
  return reinterpret_cast<T*>(p);
}

// A valid problem, from which each check departs.
struct Case {
  prnnAttention_t d;
  prnnSequence_t q, k, v, o, dq, dk, dv;
  float *S0, *S1;
  Case() {
    d = {3, 5, 4, 2, 8, 6, PRNN_DATA_HALF, 0.5f, at<float>(0x100000), nullptr, nullptr, 0};
    q = {at<void>(0x200000), 3 * 32, 32, 8};
    k = {at<void>(0x300000), 3 * 16, 16, 8};
    v = {at<void>(0x400000), 3 * 12, 12, 6};
    o = {at<void>(0x500000), 3 * 24, 24, 6};
    dq = q;
    dk = k;
    dv = v;
    dq.data = at<void>(0x600000);
    dk.data = at<void>(0x700000);
    dv.data = at<void>(0x800000);
    S0 = at<float>(0x900000);
    S1 = at<float>(0xa00000);
  }
  prnnContext h;
  prnnStatus_t forward() { return prnn_linear_attention(&h, &d, &q, &k, &v, S0, &o, S1, nullptr); }
  prnnStatus_t step() { return prnn_linear_attention_step(&h, &d, &q, &k, &v, S0, &o, S1, nullptr); }
  prnnStatus_t backward() {
    return prnn_linear_attention_backward(&h, &d, &q, &k, &v, nullptr, &o, S0, &dq, &dk, &dv, S1, nullptr);
  }
};

// Departs by `change`; the forward, backward and (where it applies) step calls
// must all answer `want`.
template <class F>
static void all(const char* what, prnnStatus_t want, F change, bool step = true) {
  const bool enqueued = false;
  for (int call = 0; call < (step ? 3 : 2); ++call) {
    Case c;
    change(c);
    expect(call == 0 ? c.forward() : call == 1 ? c.backward() : c.step(), want, enqueued, what);
  }
}

int main() {
  const prnnStatus_t ok = PRNN_STATUS_SUCCESS, bad = PRNN_STATUS_BAD_PARAM, no = PRNN_STATUS_NOT_SUPPORTED;
  {
    Case c;
    expect(c.forward(), ok, true, "forward");
    expect(c.step(), ok, true, "step");
    expect(c.backward(), ok, true, "backward");
    expect(prnn_linear_attention(nullptr, &c.d, &c.q, &c.k, &c.v, c.S0, &c.o, c.S1, nullptr), bad, false, "no handle");
    expect(prnn_linear_attention(&c.h, nullptr, &c.q, &c.k, &c.v, c.S0, &c.o, c.S1, nullptr), bad, false, "no descriptor");
    expect(prnn_linear_attention(&c.h, &c.d, nullptr, &c.k, &c.v, c.S0, &c.o, c.S1, nullptr), bad, false, "no q");
  }
  all("failed run", PRNN_STATUS_EXECUTION_FAILED, [](Case& c) { c.h.failed = true; });
  all("B < 0", bad, [](Case& c) { c.d.B = -1; });
  all("T < 0", bad, [](Case& c) { c.d.T = -1; }, false);
  all("H = 0", bad, [](Case& c) { c.d.H = 0; });
  all("Hkv = 0", bad, [](Case& c) { c.d.Hkv = 0; });
  all("H not a multiple of Hkv", bad, [](Case& c) { c.d.Hkv = 3; });
  all("Dk = 0", bad, [](Case& c) { c.d.Dk = 0; });
  all("Dk = 257", bad, [](Case& c) { c.d.Dk = 257; });
  all("Dv = -3", bad, [](Case& c) { c.d.Dv = -3; });
  all("Dv = 257", bad, [](Case& c) { c.d.Dv = 257; });
  all("type", bad, [](Case& c) { c.d.type = (prnnDataType_t)3; });
  all("type", bad, [](Case& c) { c.d.type = PRNN_DATA_MAX_ENUM; });
  all("no decays", bad, [](Case& c) { c.d.log_decay = nullptr; });
  all("decays at 2 bytes", bad, [](Case& c) { c.d.log_decay = at<float>(0x100002); });
  all("no k", bad, [](Case& c) { c.k.data = nullptr; });
  all("q at an odd byte", bad, [](Case& c) { c.q.data = at<void>(0x200001); });
  all("fp32 at 2 bytes", bad, [](Case& c) {
    c.d.type = PRNN_DATA_FLOAT;
    c.v.data = at<void>(0x400002);
  });
  all("negative head stride", bad, [](Case& c) { c.q.head = -8; });
  all("negative token stride", bad, [](Case& c) { c.k.token = -8; }, false);
  all("negative batch stride", bad, [](Case& c) { c.v.batch = -8; });
  all("a stride past every memory", bad, [](Case& c) { c.q.head = 1ll << 50; });
  all("state at 2 bytes", bad, [](Case& c) { c.S0 = at<float>(0x900002); });
  all("states overlap in part", bad, [](Case& c) { c.S1 = c.S0 + 4; });
  all("lengths and offsets", bad, [](Case& c) {
    c.d.lengths = at<int32_t>(0xb00000);
    c.d.offsets = at<int32_t>(0xb10000);
    c.d.rows = 15;
  }, false);
  all("rows < 0", bad, [](Case& c) {
    c.d.offsets = at<int32_t>(0xb10000);
    c.d.rows = -1;
  }, false);
  all("offsets at 2 bytes", bad, [](Case& c) {
    c.d.offsets = at<int32_t>(0xb10002);
    c.d.rows = 15;
  }, false);
  all("o's heads overlap", bad, [](Case& c) { c.dq.head = c.o.head = 5; });
  all("o's batch rows coincide", bad, [](Case& c) { c.dv.batch = c.o.batch = 0; });
  all("token stride past 2^23", no, [](Case& c) { c.q.token = (1 << 23) + 1; }, false);
  all("too many states", no, [](Case& c) {
    c.d.B = 1 << 23;
    c.q.batch = c.k.batch = c.v.batch = c.o.batch = c.dq.batch = c.dk.batch = c.dv.batch = 1 << 20;
  });
  {
    Case c;
    c.o.data = c.q.data;
    expect(c.forward(), bad, false, "o over q");
    c = Case();
    c.o.data = c.S0;
    expect(c.forward(), bad, false, "o over the states");
    c = Case();
    c.S1 = at<float>(0x300010);
    expect(c.forward(), bad, false, "the final states over k");
    c = Case();
    c.S1 = c.S0 = nullptr;
    expect(c.step(), bad, false, "a step without states");
    c = Case();
    c.dk.data = c.dq.data;
    expect(c.backward(), bad, false, "dk over dq");
    c = Case();
    c.dq.data = c.q.data;
    expect(c.backward(), bad, false, "dq over q");
    c = Case();
    c.h.no_memory = true;
    expect(c.backward(), PRNN_STATUS_ALLOC_FAILED, false, "no memory for the shared heads");
    c = Case();
    c.S1 = c.S0;
    expect(c.forward(), ok, true, "states in place");
    expect(c.step(), ok, true, "states in place");
    expect(c.backward(), ok, true, "states in place");
    c = Case();
    c.k.batch = c.k.token = 0;
    expect(c.forward(), ok, true, "an input repeated by strides of 0");
    // q, k, v and o as slices of the rows of one buffer, fp16: 32 + 16 + 12 + 24 elements
    c = Case();
    prnnSequence_t* all4[] = {&c.q, &c.k, &c.v, &c.o};
    const int offset[] = {0, 32, 48, 60};
    for (int i = 0; i < 4; ++i) {
      all4[i]->data = at<void>(0x200000 + 2 * offset[i]);
      all4[i]->batch = 84;
      all4[i]->token = 84 * 3;
    }
    expect(c.forward(), ok, true, "slices of one buffer");
    c.o.data = at<void>(0x200000 + 2 * 59);
    expect(c.forward(), bad, false, "slices that meet");
    c = Case();
    c.d.B = 0;
    expect(c.forward(), ok, false, "B = 0");
    c = Case();
    c.d.T = 0;
    c.q.data = c.k.data = c.v.data = c.o.data = nullptr;
    expect(c.forward(), ok, true, "T = 0 passes the states on");
    c.S1 = nullptr;
    expect(c.forward(), ok, false, "T = 0 without final states");
    c = Case();
    c.d.offsets = at<int32_t>(0xb10000);
    c.d.rows = 11;
    c.q.token = 32;
    c.k.token = 16;
    c.v.token = 12;
    c.o.token = 24;
    expect(c.forward(), ok, true, "packed");
    workspace = 0;
    c.dq.token = 32;
    c.dk.token = 16;
    c.dv.token = 12;
    expect(c.backward(), ok, true, "packed");
    if (workspace < 11u * 4 * (8 + 6) * 4 + 3 * 1000 * 4) {
      std::printf("workspace of %zu bytes\n", workspace);
      ++failures;
    }
  }

  prnnContext h;
  float *x = at<float>(0x100000), *y = at<float>(0x200000), *w = at<float>(0x300000), *b = at<float>(0x310000),
        *m = at<float>(0x400000), *r = at<float>(0x410000), *z = at<float>(0x500000), *dw = at<float>(0x600000),
        *db = at<float>(0x610000);
  const prnnDataType_t f = PRNN_DATA_FLOAT, half = PRNN_DATA_HALF;
  auto norm = [&](prnnContext* hh, int64_t M, int N, prnnDataType_t t, const void* xx, int64_t ldx, prnnDataType_t pt,
                  const void* ww, float eps, void* yy, int64_t ldy, float* mm) {
    return prnn_layer_norm(hh, M, N, t, xx, ldx, pt, ww, b, eps, yy, ldy, mm, r, nullptr);
  };
  expect(norm(&h, 5, 7, f, x, 7, f, w, 1e-5f, y, 9, m), ok, true, "norm");
  expect(norm(&h, 5, 7, f, x, 7, f, w, 1e-5f, x, 7, m), ok, true, "norm in place");
  expect(norm(&h, 5, 7, half, x, 7, half, w, 0.f, y, 7, m), ok, true, "norm of fp16");
  expect(norm(&h, 0, 7, f, nullptr, 7, f, w, 1e-5f, nullptr, 7, m), ok, false, "norm of no rows");
  expect(norm(nullptr, 5, 7, f, x, 7, f, w, 1e-5f, y, 7, m), bad, false, "norm: no handle");
  expect(norm(&h, -1, 7, f, x, 7, f, w, 1e-5f, y, 7, m), bad, false, "norm: M < 0");
  expect(norm(&h, 5, 0, f, x, 7, f, w, 1e-5f, y, 7, m), bad, false, "norm: N = 0");
  expect(norm(&h, 5, 7, f, x, 6, f, w, 1e-5f, y, 7, m), bad, false, "norm: ldx < N");
  expect(norm(&h, 5, 7, f, x, 7, f, w, 1e-5f, y, 6, m), bad, false, "norm: ldy < N");
  expect(norm(&h, 5, 7, f, x, 7, half, w, 1e-5f, y, 7, m), bad, false, "norm: fp16 parameters of fp32 rows");
  expect(norm(&h, 5, 7, half, x, 7, PRNN_DATA_BFLOAT, w, 1e-5f, y, 7, m), bad, false, "norm: bf16 parameters of fp16");
  expect(norm(&h, 5, 7, (prnnDataType_t)5, x, 7, f, w, 1e-5f, y, 7, m), bad, false, "norm: type");
  expect(norm(&h, 5, 7, f, x, 7, f, w, -1e-5f, y, 7, m), bad, false, "norm: eps < 0");
  expect(norm(&h, 5, 7, f, x, 7, f, w, __builtin_nanf(""), y, 7, m), bad, false, "norm: eps NaN");
  expect(norm(&h, 5, 7, f, nullptr, 7, f, w, 1e-5f, y, 7, m), bad, false, "norm: no x");
  expect(norm(&h, 5, 7, f, at<void>(0x100002), 7, f, w, 1e-5f, y, 7, m), bad, false, "norm: x at 2 bytes");
  expect(norm(&h, 5, 7, f, x, 7, f, w, 1e-5f, x + 3, 7, m), bad, false, "norm: y over x in part");
  expect(norm(&h, 5, 7, f, x, 7, f, w, 1e-5f, x, 9, m), bad, false, "norm: y over x at another stride");
  expect(norm(&h, 5, 7, f, x, 7, f, w, 1e-5f, y, 7, r), bad, false, "norm: mean over rstd");
  expect(norm(&h, 5, 7, f, x, 7, f, w, 1e-5f, w, 7, m), bad, false, "norm: y over weight");
  expect(norm(&h, 1ll << 31, 7, f, x, 7, f, w, 1e-5f, y, 7, nullptr), no, false, "norm: too many rows");
  // x and y as halves of the rows of one buffer
  expect(norm(&h, 5, 8, f, x, 16, f, w, 1e-5f, x + 8, 16, m), ok, true, "norm: halves of one buffer");
  h.failed = true;
  expect(norm(&h, 5, 7, f, x, 7, f, w, 1e-5f, y, 7, m), PRNN_STATUS_EXECUTION_FAILED, false, "norm: failed run");

  auto back = [&](int64_t M, int N, const void* dy, int64_t lddy, const void* xx, const float* mm, void* dx,
                  int64_t lddx, void* dww, void* dbb) {
    return prnn_layer_norm_backward(&h, M, N, f, dy, lddy, xx, N, mm, r, f, w, dx, lddx, dww, dbb, nullptr);
  };
  expect(back(5, 7, y, 7, x, m, z, 7, dw, db), ok, true, "norm backward");
  expect(back(5, 7, y, 7, x, m, y, 7, dw, db), ok, true, "norm backward over dy");
  expect(back(5, 7, y, 7, x, m, x, 7, dw, db), ok, true, "norm backward over x");
  expect(back(5, 7, y, 7, x, m, nullptr, 0, dw, db), ok, true, "norm backward: parameters only");
  expect(back(5, 7, y, 7, x, m, z, 7, nullptr, nullptr), ok, true, "norm backward: dx only");
  expect(back(5, 7, y, 7, x, m, nullptr, 0, nullptr, nullptr), ok, false, "norm backward of nothing");
  expect(back(0, 7, nullptr, 7, nullptr, nullptr, nullptr, 7, dw, db), ok, true, "norm backward of no rows");
  expect(back(5, 7, nullptr, 7, x, m, z, 7, dw, db), bad, false, "norm backward: no dy");
  expect(back(5, 7, y, 7, x, nullptr, z, 7, dw, db), bad, false, "norm backward: no mean");
  expect(back(5, 7, y, 6, x, m, z, 7, dw, db), bad, false, "norm backward: lddy < N");
  expect(back(5, 7, y, 7, x, m, z, 5, dw, db), bad, false, "norm backward: lddx < N");
  expect(back(5, 7, y, 7, x, m, z, 7, dw, dw), bad, false, "norm backward: dweight over dbias");
  expect(back(5, 7, y, 7, x, m, z, 7, x, db), bad, false, "norm backward: dweight over x");
  expect(back(5, 7, y, 7, x, m, x + 1, 7, dw, db), bad, false, "norm backward: dx over x in part");
  expect(back(5, 7, y, 7, x, m, m, 7, dw, db), bad, false, "norm backward: dx over mean");
  h.no_memory = true;
  expect(back(5, 7, y, 7, x, m, z, 7, dw, db), PRNN_STATUS_ALLOC_FAILED, false, "norm backward: no memory");

  if (failures == 0) std::printf("all checks passed\n");
  return failures == 0 ? 0 : 1;
}
