// simt_ext.cu -- the CUDA-core forward's instances for windows with first keys
// and paged caches: the general layout here, the chunked form in
// simt_ext_full.cu.
#include "simt_fwd.cuh"

namespace attn {

cudaError_t launch_simt_ext_full(const Problem& p, const Ext& x, const Split& s, cudaStream_t st);

cudaError_t launch_simt_ext(const Problem& p, const Ext& x, const Split& s, cudaStream_t st) {
  if (p.D == 32 || p.D == 64 || p.D == 128 || p.D == 256) return launch_simt_ext_full(p, x, s, st);
  return launch_simt_all<false, true>(p, s, st, x);
}

}  // namespace attn
