// shared_tc64.cu -- instances of the shared-prefix kernel (shared_tc.cuh) at head_dim 64.
#include "shared_tc.cuh"

namespace attn {
int shared_tc64(const Problem& p, const Ext& x, const shr::Work& w, cudaStream_t st) {
  return shr::launch_d<64>(p, x, w, st);
}
}  // namespace attn
