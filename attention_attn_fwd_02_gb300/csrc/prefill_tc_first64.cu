// prefill_tc_first64.cu -- the head_dim 64 tensor-core prefill's instances for
// windows with first keys.
#include "prefill_tc_fwd.cuh"

namespace attn {
int prefill_tc_first64(const Problem& p, const Split& sp, cudaStream_t st, int first) {
  return tc::launch_d<64, true>(p, sp, st, first);
}
}  // namespace attn
