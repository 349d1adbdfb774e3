// prep_axes_f16.cu -- instances of the step with positions on several axes (prep_axes.cuh).
#include "prep_axes.cuh"

namespace attn {
cudaError_t prep_axes_f16(const Prep& p, bool kv8, cudaStream_t st) { return launch_type<__half>(p, kv8, st); }
}  // namespace attn
