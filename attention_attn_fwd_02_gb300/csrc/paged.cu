// paged.cu -- which paged decode pass a problem takes, its plan and workspace.
#include "paged.cuh"
#include "tma.h"

namespace attn {
namespace paged {

// The tensor-core pass's instances for one pair of types (paged_mma_*.cu): fill in the
// plan, and with `launch` enqueue the pass.  False when there is none for the problem.
bool mma_f16(Work& w, bool launch, cudaStream_t st, int* rc);
bool mma_bf16(Work& w, bool launch, cudaStream_t st, int* rc);
bool mma_f16_q8(Work& w, bool launch, cudaStream_t st, int* rc);
bool mma_bf16_q8(Work& w, bool launch, cudaStream_t st, int* rc);
// The CUDA-core pass over float32 caches (paged_f32.cu).
bool cores_f32(Work& w, bool launch, cudaStream_t st, int* rc);

namespace {

bool pass(Work& w, bool launch, cudaStream_t st, int* rc) {
  const Problem& p = w.p;
  if (p.dtype == ATTN_F16) return p.kv_int8 ? mma_f16_q8(w, launch, st, rc) : mma_f16(w, launch, st, rc);
  if (p.dtype == ATTN_BF16) return p.kv_int8 ? mma_bf16_q8(w, launch, st, rc) : mma_bf16(w, launch, st, rc);
  return cores_f32(w, launch, st, rc);
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }
size_t rows_of(const Work& w) { return (size_t)w.ctas * 2 * w.heads; }
size_t sums_bytes(const Work& w) { return round256(rows_of(w) * 2 * sizeof(float)); }   // part_m and part_l

size_t parts_bytes(const Work& w) { return round256(rows_of(w) * w.p.D * sizeof(float)) + sums_bytes(w); }

// Lays the fragments' arrays out in a workspace; returns what is behind them.
char* lay_out(Work& w, void* workspace) {
  w.part_o = static_cast<float*>(workspace);
  w.part_m = reinterpret_cast<float*>(static_cast<char*>(workspace) + round256(rows_of(w) * w.p.D * sizeof(float)));
  w.part_l = w.part_m + rows_of(w);
  return static_cast<char*>(workspace) + parts_bytes(w);
}

}  // namespace
}  // namespace paged

size_t paged_ws_bytes(const Problem& p, int first) {
  paged::Work w{};
  w.p = p;
  w.x.first = first;
  int rc = 0;
  if (p.B < 1 || !paged::pass(w, false, nullptr, &rc) || w.cluster || w.stride) return 0;
  return paged::parts_bytes(w) + paged::round256(w.ctas * sizeof(paged::CutUnit));
}

size_t paged_own_bytes(const Problem& p, int sms) {
  paged::Work w{};
  w.p = p;
  w.own.sms = sms;
  int rc = 0;
  if (p.B < 1 || !paged::pass(w, false, nullptr, &rc) || w.cluster || w.stride) return 0;
  return paged::parts_bytes(w) + paged::round256((size_t)p.B * p.G * w.n_hc * sizeof(int2));
}

bool paged_own(const Problem& p, const Ext& x, const paged::OwnPart& own, void* workspace, cudaStream_t st,
               paged::Work* done, int* rc) {
  paged::Work w{};
  w.p = p;
  w.x = x;
  w.own = own;
  if (!paged::pass(w, false, st, rc)) return false;
  if (!w.cluster && !w.stride) w.own.note = reinterpret_cast<int2*>(paged::lay_out(w, workspace));
  paged::pass(w, true, st, rc);
  *done = w;
  return true;
}

int paged_try(const Problem& p, const Ext& x, void* workspace, cudaStream_t st, int* used) {
  *used = 0;
  const int es = p.kv_int8 ? 1 : p.dtype == ATTN_F32 ? 4 : 2;
  const float sc = p.scale * paged::kLog2e;
  if (!(sc == sc) || isinf(sc)) return ATTN_OK;
  // 16-byte loads of cache rows.
  if (!tma_layout_ok_es(p.K, p.k, x.page_size, p.G, (int)min(x.n_pages, 0x7fffffffu), es) ||
      !tma_layout_ok_es(p.V, p.v, x.page_size, p.G, (int)min(x.n_pages, 0x7fffffffu), es))
    return ATTN_OK;
  paged::Work w{};
  w.p = p;
  w.x = x;
  int rc = 0;
  if (!paged::pass(w, false, st, &rc)) return ATTN_OK;
  if (!w.cluster && !w.stride)   // only shares have fragments
    w.cuts = reinterpret_cast<paged::CutUnit*>(paged::lay_out(w, workspace));
  *used = 1;
  paged::pass(w, true, st, &rc);
  return rc;
}

}  // namespace attn
