// The gated delta rule of fp32 operands (delta_chunk.h).
#include "delta_chunk.h"

namespace prnn {

hipError_t launch_delta_f32(const DeltaArgs& a, bool backward, hipStream_t stream) { return delta::launch_type<F32>(a, backward, stream); }

}  // namespace prnn
