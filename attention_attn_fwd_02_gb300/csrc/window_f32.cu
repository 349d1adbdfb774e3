// window_f32.cu -- float32 windows with first keys (window_f32.cuh).
#include "window_f32.cuh"

namespace attn {

int window_f32_try(const Problem& p, int first, const Split& sp, cudaStream_t st, int* used) {
  *used = 0;
  if (p.dtype != ATTN_F32 || p.kv_int8 || p.Sk < 1) return ATTN_OK;
  if (!tma_layout_ok_es(p.Q, p.q, p.Sq, p.H, p.B, 4) || !tma_layout_ok_es(p.K, p.k, p.Sk, p.G, p.B, 4) ||
      !tma_layout_ok_es(p.V, p.v, p.Sk, p.G, p.B, 4) || !tma_layout_ok_es(p.O, p.o, p.Sq, p.H, p.B, 4))
    return ATTN_OK;   // 16-byte loads and stores of rows
  const float sc = p.scale * S::kLog2;
  if (!(sc == sc) || isinf(sc)) return ATTN_OK;
  const int rc = launch_head_dim<kPlain>(p, make_ext(first, nullptr), sp, sp.n_splits, st);
  if (rc < 0) return ATTN_OK;
  *used = 1;
  return rc;
}

}  // namespace attn
