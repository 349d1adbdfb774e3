// shared_f32.cu -- float32 prompts over a shared prefix in a paged cache (window_f32.cuh).
#include "shared.h"
#include "window_f32.cuh"

namespace attn {

int shared_f32_try(const Problem& p, const Ext& x, const Split& sp, cudaStream_t st, int* used) {
  *used = 0;
  const int pages = (int)min(x.n_pages, 0x7fffffffu);
  if (p.dtype != ATTN_F32 || p.kv_int8 || p.Sk < 1 || pages < 1) return ATTN_OK;
  if (!tma_layout_ok_es(p.Q, p.q, p.Sq, p.H, p.B, 4) || !tma_layout_ok_es(p.K, p.k, x.page_size, p.G, pages, 4) ||
      !tma_layout_ok_es(p.V, p.v, x.page_size, p.G, pages, 4) || !tma_layout_ok_es(p.O, p.o, p.Sq, p.H, p.B, 4))
    return ATTN_OK;   // 16-byte loads and stores of rows
  const float sc = p.scale * S::kLog2;
  if (!(sc == sc) || isinf(sc)) return ATTN_OK;
  const int rc = launch_head_dim<true>(p, x, sp, st);
  if (rc < 0) return ATTN_OK;
  *used = 1;
  return rc;
}

}  // namespace attn
