// window_tc64.cu -- the head_dim 64 instances of the windowed tensor-core forward.
#include "window_tc.cuh"

namespace attn {
int window_tc64(const Problem& p, int first, const Split& sp, cudaStream_t st) {
  return win::launch_d<64>(p, first, sp, st);
}
}  // namespace attn
