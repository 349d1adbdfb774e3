// paged_mma_f16.cu -- instances of the tensor-core paged decode pass (paged_mma.cuh).
#include "paged_mma.cuh"

namespace attn {
namespace paged {
bool mma_f16(Work& w, bool launch, cudaStream_t st, int* rc) { return pick<false, false>(w, launch, st, rc); }
}  // namespace paged
}  // namespace attn
