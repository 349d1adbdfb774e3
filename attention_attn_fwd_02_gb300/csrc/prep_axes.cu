// prep_axes.cu -- the step before attention with positions on several axes (prep.cuh).
#include "prep.cuh"

namespace attn {
cudaError_t prep_axes(const Prep& p, bool kv8, int dtype, cudaStream_t st) {
  return launch_prep<true>(p, kv8, dtype, st);
}
}  // namespace attn
