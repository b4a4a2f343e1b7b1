// Host side of rms norm: argument checks and the workspace.
#include "rms_norm.h"

#include <cstring>

#include "regions.h"

using namespace prnn;

namespace {

// The checks both directions share.
prnnStatus_t check_norm(prnnContext* h, int64_t M, int N, prnnDataType_t type, prnnDataType_t ptype) {
  if (h == nullptr) return PRNN_STATUS_BAD_PARAM;
  if (handle_failed(h)) return PRNN_STATUS_EXECUTION_FAILED;
  if (M < 0 || N < 1 || !known(type) || !known(ptype)) return PRNN_STATUS_BAD_PARAM;
  if (ptype != PRNN_DATA_FLOAT && ptype != type) return PRNN_STATUS_BAD_PARAM;
  // (columns are counted in 31 bits, in steps of up to 1024)
  return M > 0x7fffffffll || N > 0x7fffffff - 1023 ? PRNN_STATUS_NOT_SUPPORTED : PRNN_STATUS_SUCCESS;
}

}  // namespace

extern "C" {

prnnStatus_t prnn_rms_norm(prnnHandle_t h, int64_t M, int N, prnnDataType_t type, const void* x, int64_t ldx,
                           const void* residual, int64_t ldr, prnnDataType_t ptype, const void* weight, float eps,
                           void* sum, int64_t lds, prnnDataType_t ytype, void* y, int64_t ldy, float* scales, int group,
                           float* rstd, hipStream_t stream) {
  const prnnStatus_t st = check_norm(h, M, N, type, ptype);
  if (st != PRNN_STATUS_SUCCESS) return st;
  const bool eight = ytype == PRNN_DATA_E4M3;
  if (!eight && ytype != type) return PRNN_STATUS_BAD_PARAM;
  if (!(eps >= 0.f) || !ld_ok(ldx, N) || !ld_ok(ldy, N) || (residual != nullptr && !ld_ok(ldr, N)) ||
      (sum != nullptr && !ld_ok(lds, N)))
    return PRNN_STATUS_BAD_PARAM;
  if (group != 0 && (!eight || group != kRmsGroup)) return PRNN_STATUS_BAD_PARAM;
  if (M == 0) return PRNN_STATUS_SUCCESS;
  const size_t e = size_of(type), pe = size_of(ptype), ye = eight ? 1 : e;
  if (x == nullptr || y == nullptr || (scales != nullptr) != eight) return PRNN_STATUS_BAD_PARAM;
  if (!aligned(x, e) || !aligned(residual, e) || !aligned(sum, e) || !aligned(y, ye) || !aligned(weight, pe) ||
      !aligned(scales, 4) || !aligned(rstd, 4))
    return PRNN_STATUS_BAD_PARAM;
  const uint64_t groups = group > 0 ? ((uint64_t)N + group - 1) / group : 1;
  const Region rx = rows_of(x, M, N, ldx, e), rr = rows_of(residual, M, N, ldr, e), rs = rows_of(sum, M, N, lds, e),
               ry = rows_of(y, M, N, ldy, ye), rw = flat(weight, pe * N), rc = flat(scales, 4ull * M * groups),
               rd = flat(rstd, 4ull * M);
  // sum may be x or the residual, and y of their type too (each in place)
  auto apart = [](const Region& a, int64_t lda, const Region& b, int64_t ldb) {
    return (a.base == b.base && lda == ldb) || !overlap(a, b);
  };
  if (!apart(rs, lds, rx, ldx) || !apart(rs, lds, rr, ldr)) return PRNN_STATUS_BAD_PARAM;
  if (eight ? overlap(ry, rx) || overlap(ry, rr) : !apart(ry, ldy, rx, ldx) || !apart(ry, ldy, rr, ldr))
    return PRNN_STATUS_BAD_PARAM;
  const Region* outs[] = {&rs, &ry, &rc, &rd};
  for (int i = 0; i < 4; ++i) {
    if (overlap(*outs[i], rw)) return PRNN_STATUS_BAD_PARAM;
    if (i >= 2 && (overlap(*outs[i], rx) || overlap(*outs[i], rr))) return PRNN_STATUS_BAD_PARAM;
    for (int j = 0; j < i; ++j)
      if (overlap(*outs[i], *outs[j])) return PRNN_STATUS_BAD_PARAM;
  }
  RmsArgs a;
  std::memset(&a, 0, sizeof(a));
  a.x = x;
  a.residual = residual;
  a.weight = weight;
  a.sum = sum;
  a.y = y;
  a.scales = scales;
  a.rstd = rstd;
  a.M = M;
  a.N = N;
  a.ldx = ldx;
  a.ldr = ldr;
  a.lds = lds;
  a.ldy = ldy;
  a.group = group;
  a.eps = eps;
  a.compute_units = handle_compute_units(h);
  return launched(launch_rms_norm(a, type, ptype, eight, stream));
}

prnnStatus_t prnn_rms_norm_backward(prnnHandle_t h, int64_t M, int N, prnnDataType_t type, const void* dy, int64_t lddy,
                                    const void* x, int64_t ldx, const float* rstd, prnnDataType_t ptype,
                                    const void* weight, const void* dsum, int64_t ldds, void* dx, int64_t lddx,
                                    void* dweight, hipStream_t stream) {
  prnnStatus_t st = check_norm(h, M, N, type, ptype);
  if (st != PRNN_STATUS_SUCCESS) return st;
  if (!ld_ok(ldx, N) || !ld_ok(lddy, N) || (dx != nullptr && !ld_ok(lddx, N)) || (dsum != nullptr && !ld_ok(ldds, N)))
    return PRNN_STATUS_BAD_PARAM;
  const size_t e = size_of(type), pe = size_of(ptype);
  if (M > 0 && (x == nullptr || dy == nullptr || rstd == nullptr)) return PRNN_STATUS_BAD_PARAM;
  if (!aligned(x, e) || !aligned(dy, e) || !aligned(dsum, e) || !aligned(dx, e) || !aligned(rstd, 4) ||
      !aligned(weight, pe) || !aligned(dweight, pe))
    return PRNN_STATUS_BAD_PARAM;
  const Region rx = rows_of(x, M, N, ldx, e), rdy = rows_of(dy, M, N, lddy, e), rds = rows_of(dsum, M, N, ldds, e),
               rdx = rows_of(dx, M, N, lddx, e), rdw = flat(dweight, pe * N);
  if (!(dx == x && lddx == ldx) && overlap(rdx, rx)) return PRNN_STATUS_BAD_PARAM;
  if (!(dx == dy && lddx == lddy) && overlap(rdx, rdy)) return PRNN_STATUS_BAD_PARAM;
  if (!(dx == dsum && lddx == ldds) && overlap(rdx, rds)) return PRNN_STATUS_BAD_PARAM;
  if (overlap(rdx, rdw)) return PRNN_STATUS_BAD_PARAM;
  for (const Region& in : {flat(rstd, 4ull * M), flat(weight, pe * N)})
    if (overlap(rdx, in) || overlap(rdw, in)) return PRNN_STATUS_BAD_PARAM;
  for (const Region& in : {rx, rdy, rds})
    if (overlap(rdw, in)) return PRNN_STATUS_BAD_PARAM;
  if (dx == nullptr && dweight == nullptr) return PRNN_STATUS_SUCCESS;
  if (M == 0 && dweight == nullptr) return PRNN_STATUS_SUCCESS;
  RmsArgs a;
  std::memset(&a, 0, sizeof(a));
  a.x = x;
  a.dy = dy;
  a.dsum = dsum;
  a.weight = weight;
  a.y = dx;
  a.rstd_in = rstd;
  a.dweight = dweight;
  a.M = M;
  a.N = N;
  a.ldx = ldx;
  a.lds = ldds;
  a.ldy = lddx;
  a.lddy = lddy;
  const int grid = rms_norm_backward_grid(a, type, handle_compute_units(h));
  if (grid > 0 && dweight != nullptr) {
    void* mem = nullptr;
    st = handle_workspace(h, (size_t)grid * N * 4, stream, &mem);
    if (st != PRNN_STATUS_SUCCESS) return st;
    a.partial = static_cast<float*>(mem);
  }
  return launched(launch_rms_norm_backward(a, type, ptype, grid, stream));
}

}  // extern "C"
