// Linear attention and layer norm: kernel arguments, launches and the element
// types they share.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>

#include "prnn.h"

namespace prnn {

// -- pieces of the handle these calls use (prnn.cpp) -----------------------------
bool handle_failed(prnnContext* h);  // an earlier run's failure, reported once
int handle_compute_units(const prnnContext* h);
bool handle_logs(const prnnContext* h);
// At least `bytes` of the handle's workspace.  Grown outside stream capture
// only (NOT_SUPPORTED while capturing); memory that a captured call uses lives
// until the handle is destroyed.
prnnStatus_t handle_workspace(prnnContext* h, size_t bytes, hipStream_t stream, void** out);

// -- linear attention (linear_attention.hip) -------------------------------------

// One operand of a linear attention: strides in elements; head h of the state
// uses head h / group of the operand.
struct AttnOperand {
  const void* p;
  int64_t token, batch, head;
  int group;
  uint32_t inverse;  // of group (set by the launch)
};

// 2^32 / d for the kernels' divisions by d (attn::divide).
inline uint32_t inverse_of(int d) { return d > 1 ? (uint32_t)((1ull << 32) / (uint32_t)d) : 0xffffffffu; }

// One linear attention of a launch, in its own roles: the forward pass is one
// job, the backward pass three.
//   S <- decay S + kscale k v^T,  o = oscale S^T q
// `reverse` walks every sequence from its last token to its first, and takes
// the initial state as decayed already (and leaves the final one decayed).
// State element (row of Dk, column of Dv) lies at row * s_row + col * s_col of
// the [B][H] matrices of Dk Dv elements.
struct AttnJob {
  AttnOperand q, k, v, o;
  const float* s_in;   // or nullptr (zeros)
  float* s_out;        // or nullptr
  float* segments;     // split sequences: a state of each segment ("slots" below), or nullptr
  int Dk, Dv;
  int s_row, s_col;
  float kscale, oscale;
  int reverse;
  int o_f32;           // o is fp32 whatever the element type
  int o_vec;           // 16-byte stores of o (set by plan_attention)
};

constexpr int kMaxAttnJobs = 3;
struct AttnArgs {
  AttnJob job[kMaxAttnJobs];
  const float* log_decay;
  const int32_t* lengths;
  const int32_t* offsets;
  int64_t rows;
  int jobs, B, T, H;
  // A state that a job reads and another one writes: copied ahead of the launch.
  const float* keep_from;
  float* keep_to;
  int64_t keep;  // elements, or 0
  // set by plan_attention
  int dkp, nt;    // kernel instance: rows of the state, tiles of 16 columns a wave
  int vec;        // 16-byte loads of q, k and v
  int tiles;      // workgroups along the columns of the widest job's Dv
  int segments;   // of the longest sequence
  int seg_tokens; // tokens of a segment
  int units;      // packed sequences whose segments are found by number (pieces), or 0
  uint32_t by_tiles, by_heads, by_states, by_seg;  // inverses of tiles, H, B H and seg_tokens
};

// Split sequences keep states in slots of the workspace, [slot][H][tiles] of
// them: a sequence of n > 1 segments the n - 1 that segments leave to the next
// one, and a job with initial states those in one more.  Packed sequences share
// as many slots as their rows can fill, however many sequences there are and
// whatever the longest one is: n - 1 is at most the number of multiples of
// seg_tokens that the sequence's rows pass, so a sequence whose first row is
// `whole` seg_tokens and a rest takes its slots from `whole` (n <= 2 (n - 1): twice
// that, with initial states).  Offsets that decrease make slots coincide, but
// never leave the workspace.
__host__ __device__ inline int64_t first_slot(const AttnArgs& a, const AttnJob& job, int b, uint32_t whole) {
  return a.offsets != nullptr ? (int64_t)whole * (job.s_in != nullptr ? 2 : 1) : (int64_t)b * a.segments;
}
// ... and their number, enough for each of the jobs.
inline int64_t slots(const AttnArgs& a) {
  bool given = false;
  for (int i = 0; i < a.jobs; ++i) given = given || a.job[i].s_in != nullptr;
  return a.offsets != nullptr ? a.rows / a.seg_tokens * (given ? 2 : 1) : (int64_t)a.B * a.segments;
}

// Pieces of the sequences, each with a workgroup for every head and tile of
// columns: the longest one's segments for every sequence, or, where packed
// sequences leave most of those without a token, as many as the rows can fill.
// The segments of a sequence whose first row is `whole` seg_tokens and a rest are
// then the units from whole + b on (n <= the multiples of seg_tokens that its rows
// pass, and one), which a workgroup finds from the offsets.  Measured, 16 bf16 heads
// of 128: 512 sequences in 32768 rows whose longest one is not known 322 us (1141
// with workgroups for each of them as long as the rows), one of 16384 tokens among
// 511 of 32 402 us (1329).
inline int64_t units_of(const AttnArgs& a) { return a.rows / a.seg_tokens + a.B; }
inline int64_t pieces(const AttnArgs& a) { return a.units > 0 ? a.units : (int64_t)a.B * a.segments; }

// Workgroups of 256 threads that a launch takes (it counts threads in 32 bits).
constexpr int64_t kMaxWorkgroups = (1ll << 24) - 1;
constexpr int kScanFrom = 9;  // segments from which a scan between the launches costs less than every segment's own sum

// Whether the widest launch of a plan fits that: the segments', or where their
// states are summed ahead up to 16 workgroups for a state.
inline bool grid_fits(const AttnArgs& a) {
  const int64_t most = a.segments >= kScanFrom ? std::max<int64_t>(pieces(a), 16ll * a.B) : pieces(a);
  return (int64_t)a.tiles * a.H * most <= kMaxWorkgroups;
}

// Chooses the instance and the split, and returns the floats of workspace
// that each job needs for AttnJob::segments (0: none).
size_t plan_attention(AttnArgs* a, prnnDataType_t type, int compute_units);
hipError_t launch_attention(const AttnArgs& a, prnnDataType_t type, hipStream_t stream);
// ... of one element type (attention_f32.hip, attention_f16.hip, attention_bf16.hip).
hipError_t launch_attention_f32(const AttnArgs& a, hipStream_t stream);
hipError_t launch_attention_f16(const AttnArgs& a, hipStream_t stream);
hipError_t launch_attention_bf16(const AttnArgs& a, hipStream_t stream);

// dst(t, b, g) = sum over the heads h of group g of src(t, b, h) (fp32, rows and
// strides multiples of 16 bytes where D is of 4), in head order, for two
// gradients.  Rows as the attention's outputs.
struct AttnReduceArgs {
  struct {
    AttnOperand src, dst;
    int D;
  } grad[2];
  const int32_t* lengths;
  const int32_t* offsets;
  int64_t rows;
  int B, T, groups, per_group;
  int blocks;  // workgroups for each sequence (set by the launch)
};
hipError_t launch_attention_reduce(const AttnReduceArgs& a, prnnDataType_t type, hipStream_t stream);

struct AttnStepArgs {
  AttnOperand q, k, v, o;
  const float* log_decay;
  const float* s_in;
  float* s_out;
  int B, H, Dk, Dv;
  int tiles;  // tiles of 32 columns
  uint32_t by_tiles, by_heads;  // inverses of tiles and H (set by the launch)
  float scale;
};
hipError_t launch_attention_step(const AttnStepArgs& a, prnnDataType_t type, hipStream_t stream);

// -- layer norm (layer_norm.hip) ----------------------------------------------------
struct NormArgs {
  const void* x;
  const void* dy;      // backward
  const void* weight;  // or nullptr
  const void* bias;    // or nullptr
  void* y;             // forward: y; backward: dx, or nullptr
  float* mean;         // forward: or nullptr
  float* rstd;
  const float* mean_in;  // backward
  const float* rstd_in;
  float* partial;      // backward: [grid][2][N] sums of dy n and dy, or nullptr
  void* dweight;       // backward: or nullptr
  void* dbias;
  int64_t M, ldx, ldy, lddy;
  int N;
  float eps;
  int compute_units;   // forward: of the device
};
hipError_t launch_layer_norm(const NormArgs& a, prnnDataType_t type, prnnDataType_t ptype, hipStream_t stream);
// Workgroups of the backward pass (each leaves one partial sum).
int layer_norm_backward_grid(const NormArgs& a, prnnDataType_t type, int compute_units);
hipError_t launch_layer_norm_backward(const NormArgs& a, prnnDataType_t type, prnnDataType_t ptype, int grid,
                                      hipStream_t stream);

#ifdef __HIPCC__
// -- element types ---------------------------------------------------------------------
struct F32 {
  typedef float raw;
  static constexpr int id = PRNN_DATA_FLOAT;
  __device__ static __forceinline__ float get(raw v) { return v; }
  __device__ static __forceinline__ raw put(float f) { return f; }
};
struct F16 {
  typedef _Float16 raw;
  static constexpr int id = PRNN_DATA_HALF;
  __device__ static __forceinline__ float get(raw v) { return (float)v; }
  __device__ static __forceinline__ raw put(float f) { return (_Float16)f; }  // nearest, ties to even
};
struct BF16 {
  typedef __bf16 raw;
  static constexpr int id = PRNN_DATA_BFLOAT;
  __device__ static __forceinline__ float get(raw v) { return (float)v; }
  __device__ static __forceinline__ raw put(float f) { return (__bf16)f; }  // nearest, ties to even
};

#endif

}  // namespace prnn
