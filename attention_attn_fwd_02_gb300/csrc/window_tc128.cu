// window_tc128.cu -- the head_dim 128 instances of the windowed tensor-core forward.
#include "window_tc.cuh"

namespace attn {
int window_tc128(const Problem& p, int first, const Split& sp, cudaStream_t st) {
  return win::launch_d<128>(p, first, sp, st);
}
}  // namespace attn
