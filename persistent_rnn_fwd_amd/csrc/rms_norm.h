// Rms norm: kernel arguments and launches.
#pragma once

#include "sequence.h"

namespace prnn {

struct RmsArgs {
  const void* x;
  const void* residual;  // forward: or nullptr
  const void* dy;        // backward
  const void* dsum;      // backward: or nullptr
  const void* weight;    // or nullptr
  void* sum;             // forward: or nullptr
  void* y;               // forward: y; backward: dx, or nullptr
  float* scales;         // forward, 8 bits: [M][groups]
  float* rstd;           // forward: or nullptr
  const float* rstd_in;  // backward
  float* partial;        // backward: [grid][N] sums of dy n, or nullptr
  void* dweight;         // backward: or nullptr
  int64_t M, ldx, ldr, lds, ldy, lddy;
  int N;
  int group;             // 8 bits: columns that share a scale (kRmsGroup), or 0: all of a row
  float eps;
  int compute_units;
};
constexpr int kRmsGroup = 128;
// eight: y is e4m3 with scales.
hipError_t launch_rms_norm(const RmsArgs& a, prnnDataType_t type, prnnDataType_t ptype, bool eight, hipStream_t stream);
// Workgroups of the backward pass (each leaves one partial sum).
int rms_norm_backward_grid(const RmsArgs& a, prnnDataType_t type, int compute_units);
hipError_t launch_rms_norm_backward(const RmsArgs& a, prnnDataType_t type, prnnDataType_t ptype, int grid, hipStream_t stream);

}  // namespace prnn
