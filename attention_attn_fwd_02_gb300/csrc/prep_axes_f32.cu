// prep_axes_f32.cu -- instances of the step with positions on several axes (prep_axes.cuh).
#include "prep_axes.cuh"

namespace attn {
cudaError_t prep_axes_f32(const Prep& p, bool kv8, cudaStream_t st) { return launch_type<float>(p, kv8, st); }
}  // namespace attn
