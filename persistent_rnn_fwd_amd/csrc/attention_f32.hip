// Linear attention of fp32 operands (attention_chunk.h).
#include "attention_chunk.h"

namespace prnn {

hipError_t launch_attention_f32(const AttnArgs& a, hipStream_t stream) { return attn::launch_type<F32>(a, stream); }

}  // namespace prnn
