// Linear attention of fp16 operands (attention_chunk.h).
#include "attention_chunk.h"

namespace prnn {

hipError_t launch_attention_f16(const AttnArgs& a, hipStream_t stream) { return attn::launch_type<F16>(a, stream); }

}  // namespace prnn
