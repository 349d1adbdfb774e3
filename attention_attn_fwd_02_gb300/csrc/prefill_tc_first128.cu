// prefill_tc_first128.cu -- the head_dim 128 tensor-core prefill's instances for
// windows with first keys.
#include "prefill_tc_fwd.cuh"

namespace attn {
int prefill_tc_first128(const Problem& p, const Split& sp, cudaStream_t st, int first) {
  return tc::launch_d<128, true>(p, sp, st, first);
}
}  // namespace attn
