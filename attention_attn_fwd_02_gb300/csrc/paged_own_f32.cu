// paged_own_f32.cu -- instances of the paged decode pass over float32 caches (paged_f32.cuh) over own keys behind a shared prefix.
#include "paged_f32.cuh"

namespace attn {
namespace paged {
template <int D, int NH>
int enqueue_own_f32(const Work& w, cudaStream_t st) {
  return enqueue_f32<D, NH, true>(w, st);
}
template int enqueue_own_f32<64, 4>(const Work&, cudaStream_t);
template int enqueue_own_f32<64, 8>(const Work&, cudaStream_t);
template int enqueue_own_f32<128, 4>(const Work&, cudaStream_t);
template int enqueue_own_f32<128, 8>(const Work&, cudaStream_t);
}  // namespace paged
}  // namespace attn
