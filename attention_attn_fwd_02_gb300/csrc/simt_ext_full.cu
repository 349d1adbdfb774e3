// simt_ext_full.cu -- the chunked form (head_dim 32, 64, 128 or 256) of the
// CUDA-core forward for windows with first keys and paged caches.
#include "simt_fwd.cuh"

namespace attn {

cudaError_t launch_simt_ext_full(const Problem& p, const Ext& x, const Split& s, cudaStream_t st) {
  return launch_simt_all<true, true>(p, s, st, x);
}

}  // namespace attn
