// shared_f32.cu -- float32 over a shared prefix in a paged cache: register tiles
// (window_f32.cuh) of each entry's rows, or of the packed rows of all entries
// against the prefix, whose partial results are merged with the own keys'.
#include "shared.h"
#include "window_f32.cuh"

namespace attn {
namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
size_t round256(size_t x) { return (x + 255) / 256 * 256; }

// 16-byte loads and stores of rows, and a scale that can be taken in base 2.
bool takes(const Problem& p, const Ext& x) {
  const int pages = (int)min(x.n_pages, 0x7fffffffu);
  const float sc = p.scale * S::kLog2;
  return p.dtype == ATTN_F32 && !p.kv_int8 && p.Sk > 0 && pages > 0 && sc == sc && !isinf(sc) &&
         tma_layout_ok_es(p.Q, p.q, p.Sq, p.H, p.B, 4) && tma_layout_ok_es(p.K, p.k, x.page_size, p.G, pages, 4) &&
         tma_layout_ok_es(p.V, p.v, x.page_size, p.G, pages, 4) && tma_layout_ok_es(p.O, p.o, p.Sq, p.H, p.B, 4);
}

}  // namespace

int shared_f32_try(const Problem& p, const Ext& x, const Split& sp, cudaStream_t st, int* used) {
  *used = 0;
  if (!takes(p, x)) return ATTN_OK;
  const int rc = launch_head_dim<kPaged>(p, x, sp, sp.n_splits, st);
  if (rc < 0) return ATTN_OK;
  *used = 1;
  if (rc || sp.n_splits == 1) return rc;
  cudaError_t e;
  if (p.D == 64 || p.D == 128) {   // (5 questions of 33 tokens behind 501 keys, 5 parts: 33.5 us with the other merge)
    shr::Work w{};
    w.own_slot = w.splits = sp.n_splits;
    w.part_o = sp.part_o;
    w.part_m = sp.part_lse;
    w.part_l = sp.part_l;
    e = launch_shared_merge(p, w, nullptr, st);
  } else {
    e = launch_combine(p, sp, p.dtype, st);
  }
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

// Rows against keys on register tiles run at some 20 TFLOP/s where their CTAs fill the SMs.  Each entry by itself, rows
// that are not there are computed too (tiles of 32 rows); one query an entry, the decode pass over pages reads the
// prefix out of L2 at some 7.5 TB/s once an entry.  Packed, a pass, the merge and the partial results come on top.
// (157 entries of 8/8 heads, head_dim 64, behind 39706 keys: 2698 us by the decode pass, 638 packed; 33 entries of 12/4
// heads, head_dim 128, behind 24940: 471 and 380.)
bool shared_f32_plan(const Problem& p, shr::Work& w) {
  if (p.dtype != ATTN_F32 || p.kv_int8 || (p.D != 64 && p.D != 128) || p.prefix < 1 || p.B < 2) return false;
  const int64_t rows = (int64_t)p.Sq * p.qpg, all = rows * p.B, own = p.Sk - p.prefix;
  if (all > (1 << 30) || all * p.G > (1ll << 31)) return false;
  auto product = [&](int64_t r, int64_t keys) { return 4.0 * (double)(r * p.G) * keys * p.D / 20.0e6; };
  const double part_us = (double)(all * p.G) * p.D * 8 / 6.0e6;
  const int64_t blocks = ceil_div(all, 64) * p.G;
  int64_t n = clamp64(ceil_div(608, blocks), 1, 32);
  n = clamp64(n, 1, ceil_div(p.prefix, 128));
  const double us_packed = 12.0 + product(ceil_div(all, 64) * 64, p.prefix) + (n + 1) * part_us;
  const double us_each = p.Sq == 1 ? (double)p.B * p.G * ceil_div(p.qpg, 8) * p.prefix * p.D * 8 / 7.5e6
                                   : product(ceil_div(rows, 32) * 32 * p.B, p.prefix);
  if (us_each < us_packed) return false;
  w = shr::Work{};
  w.own_slot = (int)n;
  w.parts_b = own > 0;
  w.splits = (int)n + w.parts_b;
  return true;
}

size_t shared_f32_bytes(const Problem& p, const shr::Work& w) {
  const size_t rows = (size_t)p.B * p.H * p.Sq * w.splits;
  return round256(rows * p.D * sizeof(float)) + 2 * round256(rows * sizeof(float));
}

int shared_f32_packed(const Problem& p, const Ext& x, shr::Work& w, const Problem& own, const Ext& x_own, void* workspace,
                      cudaStream_t st, int* used) {
  *used = 0;
  if (!takes(p, x)) return ATTN_OK;
  const size_t rows = (size_t)p.B * p.H * p.Sq * w.splits;
  w.part_o = static_cast<float*>(workspace);
  w.part_m = reinterpret_cast<float*>(static_cast<char*>(workspace) + round256(rows * p.D * sizeof(float)));
  w.part_l = w.part_m + round256(rows * sizeof(float)) / sizeof(float);
  Split s{w.own_slot, 1, w.part_o, w.part_m, w.part_l};
  int rc = launch_head_dim<kPacked>(p, x, s, w.splits, st);
  if (rc < 0) return ATTN_OK;
  *used = 1;
  if (rc) return rc;
  paged::Work decode{};
  const bool decoded = p.Sq == 1 && own.Sk > 0;
  if (decoded) {
    const paged::OwnPart part{w.part_o + (int64_t)w.own_slot * p.D, w.part_m + w.own_slot, w.part_l + w.own_slot,
                              w.splits, 0, nullptr};
    if (!paged_own(own, x_own, part, static_cast<char*>(workspace) + shared_f32_bytes(p, w), st, &decode, &rc))
      return ATTN_ERR_UNSUPPORTED;
  } else if (own.Sk > 0) {
    s = Split{1, 1, w.part_o + (int64_t)w.own_slot * p.D, w.part_m + w.own_slot, w.part_l + w.own_slot};
    rc = launch_head_dim<kPaged>(own, x_own, s, w.splits, st);
    if (rc < 0) return ATTN_ERR_CUDA;   // (no more than 2^30 CTAs: two rows an entry and kv head or more)
  }
  if (rc) return rc;
  return launch_shared_merge(p, w, decoded ? &decode : nullptr, st) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace attn
