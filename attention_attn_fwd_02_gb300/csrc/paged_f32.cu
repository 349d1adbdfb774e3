// paged_f32.cu -- plans and instances of the paged decode pass over float32 caches (paged_f32.cuh).
#include "paged_f32.cuh"

namespace attn {
namespace paged {
namespace {

template <int D, int NH>
int pass_cfg(Work& w, bool launch, cudaStream_t st) {
  using C = CfgF32<D, NH, kShares>;
  plan_work(w, C::Stages::kTile, NH, C::kCtas);
  if (!launch) return ATTN_OK;
  if (w.own.o) {
    if constexpr (D <= 128) return enqueue_own_f32<D, NH>(w, st);
    return ATTN_ERR_UNSUPPORTED;   // (no plan of attn_fwd_shared comes here)
  }
  return enqueue_f32<D, NH, false>(w, st);
}

template <int D>
int pass_heads(Work& w, bool launch, cudaStream_t st) {
  return w.p.qpg <= 4 ? pass_cfg<D, 4>(w, launch, st) : pass_cfg<D, 8>(w, launch, st);
}

}  // namespace

bool cores_f32(Work& w, bool launch, cudaStream_t st, int* rc) {
  if (w.p.kv_int8) return false;
  switch (w.p.D) {
    case 64: *rc = pass_heads<64>(w, launch, st); return true;
    case 128: *rc = pass_heads<128>(w, launch, st); return true;
    case 256: *rc = pass_heads<256>(w, launch, st); return true;
    default: return false;
  }
}

}  // namespace paged
}  // namespace attn
