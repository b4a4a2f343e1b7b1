// The gated delta rule: kernel arguments and launches.
#pragma once

#include "sequence.h"

namespace prnn {

constexpr int kDeltaChunk = 32;  // tokens of a chunk

// What the chunks' kernels need of a chunk and head besides q, k and v, left by
// the first launch (delta_prepare_kernel), in bytes from the block's start.  T' and P' are three
// bf16 parts of 32 x 32, in the order that delta_at() says.
constexpr int kDeltaT = 0, kDeltaP = 3 * 2048, kDeltaVec = 6 * 2048;
enum DeltaVec { kUp, kScaledUp, kInto, kDown, kBeta };  // 32 floats each
constexpr int kDeltaSums = kDeltaVec + 5 * 128;         // 32 doubles: the decays' sums
constexpr int kDeltaBlock = 13 * 1024;

// Waves of a workgroup of the gradients' launch, by the rows its instance holds (dkp).
constexpr int delta_grad_waves(int dkp) { return dkp == 64 ? 4 : 8; }

struct DeltaArgs {
  AttnOperand q, k, v, o;  // o: the output, or its gradient
  AttnOperand g, beta;     // fp32, one value a token and head; g.p null: no decay
  AttnOperand dq, dk, dv, dg, dbeta;  // dg.p may be null
  const float* s_in;       // or nullptr (zeros)
  float* s_out;            // or nullptr
  const float* ds_in;      // backward: of the final state, or nullptr
  float* ds_out;           // ... and of the initial one, or nullptr
  const int32_t* lengths;
  const int32_t* offsets;
  int64_t rows;
  int B, T, H, Dk, Dv;
  float scale;
  int qk_f32;  // dq and dk are fp32 whatever the element type
  // workspace, by chunk ("slot") and head
  char* blocks;
  // ... backward, by group of chunks (see delta_grad_kernel) and head:
  float *x, *w;   // [tokens][pitch]
  float *S, *R;   // [Dk][pitch], the state that the group starts from and the gradient of the one it ends with
  // ... and by segment of a split sequence (Where::part) and head
  float* ends;    // [Dk][pitch]: the state a segment leaves by itself, then the sequence's; backward then its gradient
  float* firsts;  // [Dk][pitch]: the state, or gradient, that the sequence's first, or last, segment starts from
  float* moves;   // [Dk][Dk], rows `move_pitch` apart: what a segment makes of the identity, without values
  // set by plan_delta
  int64_t slots;      // chunks in the workspace
  int chunks;         // of the longest sequence
  int group, groups;  // chunks of a group; groups of the longest sequence
  int64_t group_slots;  // groups in the workspace
  int64_t seg_slots;  // segments in the workspace, 0: no sequence is split
  int segments;       // of the longest sequence
  int seg_chunks;     // chunks of a segment
  int pieces;         // segments of all sequences, as a launch has workgroups for them
  int units;          // packed: workgroups' sequences and segments are found by number (find_unit), or 0
  int pitch, move_pitch;
  int dkp, tiles, move_tiles, vec;
  uint32_t by_tiles, by_all_tiles, by_heads, by_chunks, by_segments, by_seg_chunks, by_seg_tokens, by_groups,
      by_group_tokens, by_pieces;
};

// Packed sequences as find_unit() takes them: in pieces of seg_tokens.
struct Pieces {
  const int32_t* offsets;
  int64_t rows;
  int B, seg_tokens;
  uint32_t by_seg;
};

// Chunks of all sequences: those of the longest one for each, or as many as
// packed rows can fill (a sequence whose first row is n chunks and a rest has
// the slots from n + b on).
// Long sequences of few heads are split into segments: what a segment makes of
// the state that it starts from is ends + moves S, both computed for all segments
// side by side, and a scan along the sequence gives the states they start from.
void plan_delta(DeltaArgs* a, prnnDataType_t type, bool backward, int compute_units);
hipError_t launch_delta(const DeltaArgs& a, prnnDataType_t type, bool backward, hipStream_t stream);
// ... of one element type (delta_f32.hip, delta_f16.hip, delta_bf16.hip)
hipError_t launch_delta_f32(const DeltaArgs& a, bool backward, hipStream_t stream);
hipError_t launch_delta_f16(const DeltaArgs& a, bool backward, hipStream_t stream);
hipError_t launch_delta_bf16(const DeltaArgs& a, bool backward, hipStream_t stream);

struct DeltaStepArgs {
  AttnOperand q, k, v, o, g, beta;
  const float* s_in;
  float* s_out;
  int B, H, Dk, Dv;
  int tiles;  // tiles of 32 columns
  uint32_t by_tiles, by_heads;
  float scale;
};
hipError_t launch_delta_step(const DeltaStepArgs& a, prnnDataType_t type, hipStream_t stream);

}  // namespace prnn
