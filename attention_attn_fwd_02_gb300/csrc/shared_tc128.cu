// shared_tc128.cu -- instances of the shared-prefix kernel (shared_tc.cuh) at head_dim 128.
#include "shared_tc.cuh"

namespace attn {
int shared_tc128(const Problem& p, const Ext& x, const shr::Work& w, cudaStream_t st) {
  return shr::launch_d<128>(p, x, w, st);
}
}  // namespace attn
