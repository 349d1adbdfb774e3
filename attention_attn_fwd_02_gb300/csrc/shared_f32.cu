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

// Parts of each row block's list of `keys` keys (groups: lists by kv head, of `rows` rows each) that take the least time,
// in *us.  An SM takes its CTAs in rounds of as many as it holds; in each a tile of 32 keys takes what one CTA needs by
// itself (head_dim 128: 4.1 us with 32 rows, 6.3 with 64) or what all need of the SM's shared memory and FMAs (2.8 and 4.2 a
// CTA).  Rows of partial results are written and read.  (128 rows of 8 kv heads, head_dim 64, against 16384 keys: 377 us
// in 19 parts, one and a third round, 266 in 14.)
int best_parts(int64_t groups, int64_t rows, int64_t keys, int D, double* us) {
  const int64_t tiles = ceil_div(keys, 32);
  const double part_us = (double)(groups * rows) * D * 8 / 6.0e6;
  int best = 1;
  *us = 0;
  for (int64_t n = 1, list = tiles; n <= 256 && n <= tiles; n = ceil_div(tiles, list - 1)) {   // (the fewest parts of a length)
    list = ceil_div(tiles, n);
    const int tm = row_tiles(D, groups * n, rows);   // rows a thread, as launch_d takes them
    const int64_t sm = ceil_div(groups * ceil_div(rows, 16 * tm) * n, shr::kSms), held = D > 128 || (D > 64 && tm == 4) ? 2 : 3;
    const double alone = D * (tm == 4 ? 0.050 : 0.034), shared = D * (tm == 4 ? 0.0325 : 0.021);
    const double last = (double)(sm % held) * shared;
    double t = (double)(sm / held) * (4.0 + (double)list * (held * shared > alone ? held * shared : alone));
    if (sm % held) t += 4.0 + (double)list * (last > alone ? last : alone);
    if (n > 1) t += 4.0 + (n + 1) * part_us + 0.04 * n;
    if (n == 1 || t < *us) {
      *us = t;
      best = (int)n;
    }
    if (sm > 8 * held || list == 1) break;
  }
  return best;
}

}  // namespace

int shared_f32_parts(const Problem& p) {
  double us;
  return best_parts((int64_t)p.B * p.G, (int64_t)p.Sq * p.qpg, p.Sk, p.D, &us);
}

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

// Each entry by itself, rows that are not there are computed too (tiles of 32 rows); one query an entry, the decode pass over
// pages reads the prefix out of L2 at some 7.5 TB/s once an entry, at some 22 TFLOP/s.  Packed, a pass, the merge and the
// partial results come on top.  (157 entries of 8/8 heads, head_dim 64, behind 39706 keys: 2698 us by the decode pass, 638
// packed; 7 of 16/8 heads, head_dim 64, behind 36567: 170 and 114; 3 of 8/4 heads, head_dim 128, behind 46887: 117 and
// 183.  9 of 2 tokens, 4/2 heads, head_dim 64, behind 11635 keys with up to 1611 own ones: 172 us with 32 parts of the
// prefix and whole own lists, 51 with the parts above.)
bool shared_f32_plan(const Problem& p, shr::Work& w) {
  if (p.dtype != ATTN_F32 || p.kv_int8 || (p.D != 64 && p.D != 128) || p.prefix < 1 || p.B < 2) return false;
  const int64_t rows = (int64_t)p.Sq * p.qpg, all = rows * p.B, own = p.Sk - p.prefix;
  if (all > (1 << 30) || all * p.G > (1ll << 31)) return false;
  const int64_t some = own < 2048 ? own : 2048;   // (how many own keys there are is not known here)
  double us_prefix, us_own = 10.0, us_list;
  const int n = best_parts(p.G, all, p.prefix, p.D, &us_prefix);
  const int n_own = own > 0 && p.Sq > 1 ? best_parts((int64_t)p.B * p.G, rows, some, p.D, &us_own) : own > 0;
  best_parts((int64_t)p.B * p.G, rows, p.prefix + some, p.D, &us_list);
  const double us_packed = 12.0 + us_prefix + us_own;
  const double us_copies = shr::decode_us(p, 8, 4, 7.5e6, 4096), us_fmas = 4.0 * p.B * p.H * p.prefix * p.D / 22.0e6;
  const double us_each = p.Sq == 1 ? 18.0 + (us_copies > us_fmas ? us_copies : us_fmas) : 6.0 + us_list;
  if (us_each < us_packed) return false;
  w = shr::Work{};
  w.own_slot = n;
  w.parts_b = n_own;
  w.splits = n + n_own;
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
