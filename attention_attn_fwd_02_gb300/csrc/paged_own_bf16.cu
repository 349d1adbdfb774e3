// paged_own_bf16.cu -- instances of the tensor-core paged decode pass (paged_mma.cuh) over own keys behind a shared prefix.
#include "paged_mma.cuh"

namespace attn {
namespace paged {
template <bool BF16, int D, int NT>
int enqueue_own(const Work& w, cudaStream_t st) {
  return enqueue<BF16, false, D, NT, true>(w, st);
}
template int enqueue_own<true, 64, 1>(const Work&, cudaStream_t);
template int enqueue_own<true, 64, 2>(const Work&, cudaStream_t);
template int enqueue_own<true, 128, 1>(const Work&, cudaStream_t);
template int enqueue_own<true, 128, 2>(const Work&, cudaStream_t);
}  // namespace paged
}  // namespace attn
