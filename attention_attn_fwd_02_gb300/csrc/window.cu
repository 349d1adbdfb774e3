// window.cu -- which tensor-core kernel a windowed forward with first keys takes.
#include <math.h>

#include "tma.h"
#include "visible.cuh"

namespace attn {

int window_tc64(const Problem& p, int first, const Split& sp, cudaStream_t st);
int window_tc128(const Problem& p, int first, const Split& sp, cudaStream_t st);

int window_tc_try(const Problem& p, int first, const Split& sp, cudaStream_t st, int* used) {
  *used = 0;
  if (p.dtype != ATTN_BF16 && p.dtype != ATTN_F16) return ATTN_OK;
  if (p.kv_int8 || (p.D != 64 && p.D != 128) || p.Sk < 1 || p.Sq < 1) return ATTN_OK;
  const float sc = p.scale * 1.4426950408889634f;
  if (!(sc == sc) || isinf(sc)) return ATTN_OK;
  if (!tma_layout_ok(p.Q, p.q, p.Sq, p.H, p.B) || !tma_layout_ok(p.K, p.k, p.Sk, p.G, p.B) ||
      !tma_layout_ok(p.V, p.v, p.Sk, p.G, p.B) || !tma_layout_ok(p.O, p.o, p.Sq, p.H, p.B))
    return ATTN_OK;
  const int rc = p.D == 64 ? window_tc64(p, first, sp, st) : window_tc128(p, first, sp, st);
  if (rc < 0) return ATTN_OK;  // tensor map refused: another pass
  *used = 1;
  return rc;
}

}  // namespace attn
