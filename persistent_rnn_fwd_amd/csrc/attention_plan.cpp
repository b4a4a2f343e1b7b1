// The plan of a linear attention's launch: the kernel instance and the split of
// the sequences.
#include "sequence.h"

#include <algorithm>

namespace prnn {

size_t plan_attention(AttnArgs* a, prnnDataType_t type, int compute_units) {
  int dk = 0, dv = 0;
  a->vec = 1;
  const int e = type == PRNN_DATA_FLOAT ? 4 : 2;
  // whole 16-byte vectors: the rows' lengths, and every stride that is used
  auto vectors = [&](const AttnOperand& x, int D, int heads, int size) {
    const int per = 16 / size;
    return D % per == 0 && (uintptr_t)x.p % 16 == 0 && (a->T <= 1 || x.token % per == 0) &&
           (a->offsets != nullptr ? x.token % per == 0 : a->B <= 1 || x.batch % per == 0) &&
           (heads <= 1 || x.head % per == 0);
  };
  for (int i = 0; i < a->jobs; ++i) {
    AttnJob& j = a->job[i];
    for (AttnOperand* x : {&j.q, &j.k, &j.v, &j.o}) x->inverse = inverse_of(x->group);
    dk = std::max(dk, j.Dk);
    dv = std::max(dv, j.Dv);
    for (const AttnOperand* x : {&j.q, &j.k, &j.v})
      if (!vectors(*x, x == &j.v ? j.Dv : j.Dk, a->H / x->group, e)) a->vec = 0;
    // (8 columns at a time also where o is fp32)
    j.o_vec = j.Dv % 8 == 0 && vectors(j.o, j.Dv, a->H / j.o.group, j.o_f32 ? 4 : e);
  }
  a->dkp = dk <= 64 ? 64 : dk <= 128 ? 128 : 256;
  // Packed sequences count as so many of the longest's length.
  const int64_t sequences = a->offsets != nullptr && a->T > 0 ? std::max<int64_t>(1, std::min<int64_t>(a->B, a->rows / a->T)) : a->B;
  const int64_t heads = std::max<int64_t>(1, sequences * a->H * a->jobs);
  // 32 columns a wave share its reads of q and k, 16 make twice the workgroups:
  // the narrow form where pieces of 64 tokens of the wide one would not fill the
  // chip.  Measured (32 / 16 columns), fp32 and bf16: 14 heads of 128, 300 tokens
  // 42 / 33 and 26 / 22 us, 56 heads, 256 tokens 30 / 29 and 22 / 21; 128 heads,
  // 1024 tokens 116 / 128 and 65 / 70.
  const int64_t wide = heads * ((dv + 127) / 128) * ((a->T + 63) / 64);
  a->nt = dv > 64 && a->dkp < 256 && wide >= 2 * compute_units ? 2 : 1;
  const int cols = 64 * a->nt;
  a->tiles = (dv + cols - 1) / cols;
  // Segments: as many as give each compute unit 2 workgroups (states of 64 x 64:
  // 3), of at least 128 tokens, or 64 where those would leave units idle.
  // Measured at 32 heads, 64 / 128 tokens: 1024 tokens of 128 x 128 fp32 54 / 49
  // us, bf16 41 / 32, of 64 x 64 bf16 26 / 19.  A split in 2 or 3 costs a short
  // sequence more than it gains: 56 x 3 jobs of 256 tokens of 128 fp32 49 whole, 53
  // in 2; 160 heads of 4096 tokens bf16 383 whole, 347 in 2, 266 in 3.
  const int64_t groups = heads * a->tiles, want = compute_units * (a->dkp == 64 && a->nt == 1 ? 3 : 2) / groups;
  const int64_t least = groups * (a->T / 128) >= compute_units ? 128 : 64;
  const int64_t segments = want < 4 && a->T < 512 ? 1 : std::max<int64_t>(1, std::min<int64_t>(want, a->T / least));
  a->seg_tokens = std::max(64, (int)(((a->T + segments - 1) / segments + 63) / 64 * 64));
  a->segments = std::max(1, (int)(((int64_t)a->T + a->seg_tokens - 1) / a->seg_tokens));
  a->units = 0;
  if (a->offsets != nullptr && a->segments > 1 && pieces(*a) > 4 * units_of(*a)) a->units = (int)units_of(*a);
  if (a->segments > 1 && !grid_fits(*a)) {
    a->segments = 1;
    a->seg_tokens = (a->T + 63) / 64 * 64;
    a->units = 0;
  }
  a->by_tiles = inverse_of(a->tiles);
  a->by_heads = inverse_of(a->H);
  a->by_states = inverse_of((int)std::min<int64_t>((int64_t)a->B * a->H, 0x7fffffff));  // (more do not fit a grid)
  a->by_seg = inverse_of(a->seg_tokens);
  return a->segments > 1 ? (size_t)slots(*a) * a->H * a->tiles * a->dkp * cols : 0;
}

}  // namespace prnn
