// Linear attention of bfloat16 operands (attention_chunk.h).
#include "attention_chunk.h"

namespace prnn {

hipError_t launch_attention_bf16(const AttnArgs& a, hipStream_t stream) { return attn::launch_type<BF16>(a, stream); }

}  // namespace prnn
