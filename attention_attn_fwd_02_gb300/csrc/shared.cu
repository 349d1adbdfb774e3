// shared.cu -- the tensor-core pass over a shared prefix: which problems it
// takes and how they are divided into items (shared.h).
#include <math.h>

#include "shared.h"
#include "tma.h"

namespace attn {

int shared_tc64(const Problem& p, const Ext& x, const shr::Work& w, const Split& sp, cudaStream_t st);
int shared_tc128(const Problem& p, const Ext& x, const shr::Work& w, const Split& sp, cudaStream_t st);

namespace shr {
namespace {

constexpr int kMaxParts = 32;   // of a list

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// us: a key tile of both row tiles (of one, in turn), an item's fixed cost, and the merge of n parts of all rows.
struct Cost {
  double tile, tile_alt, item;
  double rows_us;   // a part of every row, written and read
  explicit Cost(const Problem& p)
      : tile(p.D == 64 ? 1.0 : 1.4), tile_alt(p.D == 64 ? 0.45 : 0.6), item(3.0),
        rows_us((double)p.B * p.H * p.Sq * p.D * 8 / 6.0e6) {}
  double merge(int n) const { return n > 1 ? 4.0 + n * rows_us : 0.0; }
  double pass(int64_t items, int64_t tiles, bool alt) const {
    return (double)ceil_div(items, kSms) * ((double)tiles * (alt ? tile_alt : tile) + item);
  }
};

// The number of parts of `tiles` key tiles, for `blocks` row blocks, that takes the least time.
int best_parts(const Cost& c, int64_t blocks, int64_t tiles, bool alt, bool merged, double* us) {
  int best = 1;
  *us = 0;
  for (int n = 1; n <= kMaxParts && n <= tiles; ++n) {
    const double t = c.pass(blocks * n, ceil_div(tiles, n), alt) +
                     (merged ? (n << alt) * c.rows_us : c.merge(n << alt));
    if (n == 1 || t < *us) {
      *us = t;
      best = n;
    }
  }
  return best;
}

}  // namespace
}  // namespace shr

bool shared_tc_plan(const Problem& p, int page_size, shr::Work& w) {
  using namespace shr;
  if (p.dtype != ATTN_BF16 && p.dtype != ATTN_F16) return false;
  if (p.kv_int8 || (p.D != 64 && p.D != 128) || p.Sk < 1 || page_size % 8) return false;
  const float sc = p.scale * 1.4426950408889634f;
  if (!(sc == sc) || isinf(sc)) return false;
  const int64_t rows = (int64_t)p.Sq * p.qpg, all = rows * p.B;
  if (all > (1 << 30) || (int64_t)p.B * p.H * p.Sq > (1ll << 31)) return false;
  w = Work{};
  w.piece = kKeys;
  while (page_size % w.piece) w.piece /= 2;
  const int64_t pre = ceil_div(p.prefix, kKeys), own = ceil_div(p.Sk - p.prefix, kKeys);
  w.blocks_b = (int)ceil_div(rows, 2 * kRows);
  const int64_t blocks_b = w.blocks_b * (int64_t)p.G * p.B;
  const Cost c(p);
  // Each entry by itself: its rows walk the prefix and their own keys.
  double us_joined = 0;
  const int parts_joined = best_parts(c, blocks_b, pre + own, false, false, &us_joined);
  // Or the prefix once for the packed rows of all entries.
  w.blocks_a = (int)ceil_div(all, 2 * kRows);
  w.alt_a = all <= kRows;
  w.alt_b = rows <= kRows;
  double us_a = 0, us_b = 0;
  w.parts_a = best_parts(c, (int64_t)w.blocks_a * p.G, pre, w.alt_a, true, &us_a);
  w.parts_b = best_parts(c, blocks_b, own, w.alt_b, true, &us_b);
  if (pre > 0 && p.B > 1 && us_a + us_b + 4.0 < us_joined) {
    if (own == 0) w.parts_b = 0;
    w.n_a = w.blocks_a * p.G * w.parts_a;
    w.splits = (w.parts_a << w.alt_a) + (w.parts_b << w.alt_b);
  } else {
    w.blocks_a = w.parts_a = w.alt_a = w.alt_b = 0;
    w.joined = 1;
    w.parts_b = w.splits = parts_joined;
  }
  const int64_t n = w.n_a + blocks_b * w.parts_b;
  if (n > 0x3fffffff) return false;
  w.n_items = (int)n;
  return true;
}

int shared_tc_try(const Problem& p, const Ext& x, const shr::Work& w, const Split& s, cudaStream_t st, int* used) {
  *used = 0;
  const int pages = (int)min(x.n_pages, 0x7fffffffu);
  if (pages < 1 || pages == 0x7fffffff) return ATTN_OK;
  if (!tma_layout_ok(p.Q, p.q, p.Sq, p.H, p.B) || !tma_layout_ok(p.K, p.k, x.page_size, p.G, pages) ||
      !tma_layout_ok(p.V, p.v, x.page_size, p.G, pages) || !tma_layout_ok(p.O, p.o, p.Sq, p.H, p.B))
    return ATTN_OK;
  const int rc = p.D == 64 ? shared_tc64(p, x, w, s, st) : shared_tc128(p, x, w, s, st);
  if (rc < 0) return ATTN_OK;  // tensor map refused: another pass
  *used = 1;
  return rc;
}

}  // namespace attn
