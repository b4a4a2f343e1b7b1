// The gated delta rule of fp16 operands (delta_chunk.h).
#include "delta_chunk.h"

namespace prnn {

hipError_t launch_delta_f16(const DeltaArgs& a, bool backward, hipStream_t stream) { return delta::launch_type<F16>(a, backward, stream); }

}  // namespace prnn
