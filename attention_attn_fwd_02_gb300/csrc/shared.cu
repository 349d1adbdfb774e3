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
constexpr double kUnit = 0.2;   // us of a cost unit of Shares

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// us: `items` items of `tiles` key tiles, dealt to the SMs in turn.
double pass_us(int64_t items, int64_t tiles, bool alt) {
  return (double)ceil_div(items, kSms) * ((double)tiles * (alt ? Shares::kTileAlt : Shares::kTile) + Shares::kEnd) * kUnit;
}

// The number of parts of `tiles` key tiles, for `blocks` row blocks, that takes the least time; part_us: what a partial
// result of every row costs, merge_us: the merge, where more than one part asks for it.
int best_parts(int64_t blocks, int64_t tiles, bool alt, double part_us, double merge_us, double* us) {
  int best = 1;
  *us = 0;
  for (int n = 1; n <= kMaxParts && n <= tiles; ++n) {
    const double t = pass_us(blocks * n, ceil_div(tiles, n), alt) + ((n > 1) * merge_us) + (n << alt) * part_us;
    if (n == 1 || t < *us) {
      *us = t;
      best = n;
    }
  }
  return best;
}

}  // namespace

int Shares::cut(int heads) {
  const int64_t full = (int64_t)tiles * kTile + kEnd, less = alt ? (int64_t)tiles * (kTile - kTileAlt) : 0;
  const int64_t total = heads * (blocks * full - less);
  int64_t begin = 0;   // of unit u, whose place in its kv head is k
  int u = 0, k = 0, most = 1;
  for (int c = 0; c <= ctas; ++c) {
    const int64_t t = total * c / ctas;
    const int units = heads * blocks;
    auto cost = [&]() { return k == blocks - 1 ? full - less : full; };
    while (u < units && t - begin >= cost()) {
      begin += cost();
      ++u;
      k = k + 1 < blocks ? k + 1 : 0;
    }
    const int64_t at = (t - begin) / (alt && k == blocks - 1 ? kTileAlt : kTile);
    const bool behind = u < units && at >= tiles;   // in a unit's end
    unit[c] = u + behind;
    tile[c] = u < units && !behind ? (int)at : 0;
    if (c == ctas) break;
    // The number of this share's first fragment: one more than the last share's, where that has tiles of the unit.
    frag[c] = 0;
    if (tile[c] > 0) {
      const bool same = unit[c - 1] == unit[c];
      frag[c] = (int16_t)(same ? frag[c - 1] + 1 : 1);
      most = frag[c] + 1 > most ? frag[c] + 1 : most;
    }
  }
  return most;
}

}  // namespace shr

bool shared_tc_plan(const Problem& p, int page_size, shr::Work& w) {
  using namespace shr;
  if (p.dtype != ATTN_BF16 && p.dtype != ATTN_F16) return false;
  if (p.kv_int8 || (p.D != 64 && p.D != 128) || p.Sk < 1 || page_size % 8) return false;
  const float sc = p.scale * 1.4426950408889634f;
  if (!(sc == sc) || isinf(sc)) return false;
  const int64_t rows = (int64_t)p.Sq * p.qpg, all = rows * p.B;
  if (all > (1 << 30) || all * p.G > (1ll << 31)) return false;
  w = Work{};
  w.piece = kKeys;
  while (page_size % w.piece) w.piece /= 2;
  const int64_t pre = ceil_div(p.prefix, kKeys), own = ceil_div(p.Sk - p.prefix, kKeys);
  const double part_us = (double)(all * p.G) * p.D * 8 / 6.0e6;   // a partial result of every row, written and read
  constexpr double kMerge = 4.0, kPass = 5.0;                      // a merge's and a pass's fixed cost
  // The prefix once for the packed rows of all entries.
  Shares& s = w.pre;
  s.tiles = (int)pre;
  s.blocks = (int)ceil_div(all, 2 * kRows);
  s.alt = (all - 1) % (2 * kRows) < kRows;
  const int64_t total =
      p.G * (s.blocks * (pre * Shares::kTile + Shares::kEnd) - s.alt * pre * (Shares::kTile - Shares::kTileAlt));
  int ctas = kSms;
  if (p.Sq == 1 && own > 0) {
    // The decode pass over pages takes the own keys, side by side with the prefix's: each gets SMs by its cost, own
    // lists being half as long as they can be.
    const double us_own = (double)p.B * p.G * (p.Sk - p.prefix) * p.D * 2 / 6.0e6, us_all = (double)total * kUnit / kSms;
    ctas = (int)(kSms * (us_all + kPass) / (us_all + us_own + 2 * kPass));
    w.own_sms = kSms - ctas;
  }
  s.ctas = (int)clamp64(total / (2 * Shares::kTile), 1, ctas);
  const int frags = s.cut(p.G);
  w.own_slot = frags << s.alt;
  const double us_pre = kPass + (double)total / s.ctas * kUnit;
  if (p.Sq == 1) {
    // The decode pass can take the prefix's keys too, once an entry, out of L2.
    const int per = p.qpg > 8 ? 16 : 8;
    const double us_each = (double)p.B * p.G * ceil_div(p.qpg, per) * p.prefix * p.D * 4 / 12.0e6;
    if (us_pre + kMerge + frags * part_us + kPass > us_each) return false;
    w.own_sms = kSms - s.ctas;
    w.one_tile = all <= kRows;
    w.parts_b = own > 0;
    w.splits = w.own_slot + w.parts_b;
    return true;
  }
  w.blocks_b = (int)ceil_div(rows, 2 * kRows);
  const int64_t blocks_b = w.blocks_b * (int64_t)p.G * p.B;
  if (blocks_b > 0x3fffffff / kMaxParts) return false;
  // Each entry by itself: its rows walk the prefix and their own keys.
  double us_joined = 0, us_own = 0;
  const int parts_joined = best_parts(blocks_b, pre + own, false, part_us, kMerge, &us_joined);
  if (parts_joined == 1) us_joined -= part_us;
  w.alt_b = rows <= kRows;
  w.parts_b = own > 0 ? best_parts(blocks_b, own, w.alt_b, part_us, 0.0, &us_own) : 0;
  if (pre > 0 && p.B > 1 && us_pre + frags * part_us + us_own + kMerge < us_joined) {
    w.splits = w.own_slot + (w.parts_b << w.alt_b);
    w.one_tile = all <= kRows;
  } else {
    s = Shares{};
    w.own_slot = w.alt_b = 0;
    w.joined = 1;
    w.parts_b = w.splits = parts_joined;
  }
  w.n_b = (int)(blocks_b * w.parts_b);
  return true;
}

int shared_tc_try(const Problem& p, const Ext& x, const shr::Work& w, const Split& s, const Problem& own, const Ext& x_own,
                  void* ws_own, cudaStream_t st, int* used) {
  *used = 0;
  const int pages = (int)min(x.n_pages, 0x7fffffffu);
  if (pages < 1 || pages == 0x7fffffff) return ATTN_OK;
  if (!tma_layout_ok(p.Q, p.q, p.Sq, p.H, p.B) || !tma_layout_ok(p.K, p.k, x.page_size, p.G, pages) ||
      !tma_layout_ok(p.V, p.v, x.page_size, p.G, pages) || !tma_layout_ok(p.O, p.o, p.Sq, p.H, p.B))
    return ATTN_OK;
  int rc = p.D == 64 ? shared_tc64(p, x, w, s, st) : shared_tc128(p, x, w, s, st);
  if (rc < 0) return ATTN_OK;  // tensor map refused: another pass
  *used = 1;
  if (rc) return rc;
  paged::Work decode{};
  const bool decoded = p.Sq == 1 && own.Sk > 0;
  if (decoded) {   // (its types and layouts are among the ones checked above)
    const paged::OwnPart part{s.part_o + (int64_t)w.own_slot * p.D, s.part_lse + w.own_slot, s.part_l + w.own_slot,
                              w.splits, w.own_sms, nullptr};
    if (!paged_own(own, x_own, part, ws_own, st, &decode, &rc)) return ATTN_ERR_UNSUPPORTED;
    if (rc) return rc;
  }
  if (w.splits == 1) return ATTN_OK;
  return launch_shared_merge(p, w, s, decoded ? &decode : nullptr, st) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace attn
