// prefill_tc.cu -- which tensor-core prefill kernel a problem takes, and the
// head_dim 64/128 kernel's instances (prefill_tc_fwd.cuh).
#include "prefill_tc_fwd.cuh"

namespace attn {

int prefill_tc_first64(const Problem& p, const Split& sp, cudaStream_t st, int first);
int prefill_tc_first128(const Problem& p, const Split& sp, cudaStream_t st, int first);

namespace {
// Types, shapes and layouts the tensor-core kernels take.
bool takes(const Problem& p) {
  if (p.dtype != ATTN_BF16 && p.dtype != ATTN_F16) return false;
  if (p.kv_int8) return false;  // int8 caches: the CUDA-core path
  if (p.D != 64 && p.D != 128 && p.D != 256) return false;
  if (p.Sk < 1 || p.Sq < 1) return false;
  if (p.Sk > 0x3fffffff || p.Sq > 0x3fffffff) return false;
  const float sc = p.scale * tc::kLog2e;
  if (!(sc == sc) || isinf(sc)) return false;
  return tma_layout_ok(p.Q, p.q, p.Sq, p.H, p.B) && tma_layout_ok(p.K, p.k, p.Sk, p.G, p.B) &&
         tma_layout_ok(p.V, p.v, p.Sk, p.G, p.B) && tma_layout_ok(p.O, p.o, p.Sq, p.H, p.B);
}
}  // namespace

int prefill_tc_try(const Problem& p, const Split& sp, cudaStream_t st, int* used) {
  *used = 0;
  if (!takes(p)) return ATTN_OK;
  int rc = -1;
  if (p.D == 256) {
    rc = prefill_tc2_launch(p, sp, st);      // CTA pairs
    if (rc < 0) rc = prefill_tc1_launch(p, sp, st);
  } else {
    rc = p.D == 64 ? tc::launch_d<64, false>(p, sp, st, 0) : tc::launch_d<128, false>(p, sp, st, 0);
  }
  if (rc < 0) return ATTN_OK;  // tensor map refused: generic path
  *used = 1;
  return rc;
}

int prefill_tc_first_try(const Problem& p, int first, const Split& sp, cudaStream_t st, int* used) {
  *used = 0;
  if (!takes(p) || p.D == 256) return ATTN_OK;
  const int rc = p.D == 64 ? prefill_tc_first64(p, sp, st, first) : prefill_tc_first128(p, sp, st, first);
  if (rc < 0) return ATTN_OK;
  *used = 1;
  return rc;
}

}  // namespace attn
