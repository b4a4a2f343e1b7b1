// The gated delta rule of bf16 operands (delta_chunk.h).
#include "delta_chunk.h"

namespace prnn {

hipError_t launch_delta_bf16(const DeltaArgs& a, bool backward, hipStream_t stream) { return delta::launch_type<BF16>(a, backward, stream); }

}  // namespace prnn
