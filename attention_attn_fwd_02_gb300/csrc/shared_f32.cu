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

// Rows against keys on register tiles run at some 25 TFLOP/s where their CTAs fill the SMs.  Each entry by itself, rows
// that are not there are computed too (tiles of 32 rows); one query an entry, the decode pass over pages reads the
// prefix out of L2 at some 7.5 TB/s once an entry.  Packed, a pass, the merge and the partial results come on top.
// (157 entries of 8/8 heads, head_dim 64, behind 39706 keys: 2698 us by the decode pass, 638 packed; 7 of 16/8 heads,
// head_dim 64, behind 36567: 170 and 114; 3 of 8/4 heads, head_dim 128, behind 46887: 117 and 183.)  A CTA takes 3 us or
// more a tile of 32 keys, so both lists are cut until their CTAs fill the SMs (9 entries of 2 tokens, 4/2 heads, head_dim
// 64, behind 11635 keys with up to 1611 own ones: 172 us with 32 parts of the prefix and whole own lists, 51 now).
bool shared_f32_plan(const Problem& p, shr::Work& w) {
  if (p.dtype != ATTN_F32 || p.kv_int8 || (p.D != 64 && p.D != 128) || p.prefix < 1 || p.B < 2) return false;
  const int64_t rows = (int64_t)p.Sq * p.qpg, all = rows * p.B, own = p.Sk - p.prefix;
  if (all > (1 << 30) || all * p.G > (1ll << 31)) return false;
  auto product = [&](int64_t r, int64_t keys) { return 4.0 * (double)(r * p.G) * keys * p.D / 25.0e6; };
  const double part_us = (double)(all * p.G) * p.D * 8 / 6.0e6;
  const int64_t blocks = ceil_div(all, 64) * p.G;
  const int64_t n = clamp64(ceil_div(608, blocks), 1, ceil_div(p.prefix, 128));
  const int tile = all > 32 && blocks * n >= 2 * shr::kSms ? 64 : 32;   // (as launch_d takes them)
  const double us_packed = 32.0 + product(ceil_div(all, tile) * tile, p.prefix) + (n + 1) * part_us;
  const double us_each =
      18.0 + (p.Sq == 1 ? shr::decode_us(p, 8, 4, 7.5e6, 4096) : product(ceil_div(rows, 32) * 32 * p.B, p.prefix));
  if (us_each < us_packed) return false;
  w = shr::Work{};
  w.own_slot = (int)n;
  w.parts_b = own > 0;
  if (own > 0 && p.Sq > 1)   // (as many CTAs for the own keys)
    w.parts_b = (int)clamp64(608 / (ceil_div(rows, 64) * p.B * p.G), 1, ceil_div(own, 128));
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
    s = Split{w.parts_b, 1, w.part_o + (int64_t)w.own_slot * p.D, w.part_m + w.own_slot, w.part_l + w.own_slot};
    rc = launch_head_dim<kPaged>(own, x_own, s, w.splits, st);
    if (rc < 0) return ATTN_ERR_CUDA;   // (no more than 2^30 CTAs: two rows an entry and kv head or more)
  }
  if (rc) return rc;
  return launch_shared_merge(p, w, decoded ? &decode : nullptr, st) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace attn
