// paged_mma_bf16.cu -- instances of the tensor-core paged decode pass (paged_mma.cuh).
#include "paged_mma.cuh"

namespace attn {
namespace paged {
bool mma_bf16(Work& w, bool launch, cudaStream_t st, int* rc) { return pick<true, false>(w, launch, st, rc); }
}  // namespace paged
}  // namespace attn
