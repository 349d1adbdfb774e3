// shared.cu -- the tensor-core pass over a shared prefix: which problems it
// takes and how they are divided (shared.h).
#include <math.h>

#include "shared.h"
#include "tma.h"

namespace attn {

int shared_tc64(const Problem& p, const Ext& x, const shr::Work& w, cudaStream_t st);
int shared_tc128(const Problem& p, const Ext& x, const shr::Work& w, cudaStream_t st);

namespace shr {
namespace {

constexpr int kMaxParts = 32;   // of an entry item's list
constexpr double kUnit = 0.2;   // us of a cost unit of Shares
constexpr double kPass = 5.0;   // us, a pass's fixed cost
constexpr double kMerge = 4.0;  // us, a merge's

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// `count` units side by side of `tiles` key tiles, each of `tile` cost units.
struct Run {
  int64_t count, tiles;
  int tile;
  int64_t cost() const { return tiles * tile + Shares::kEnd; }
};

// The runs of a plan's list, in its order; joined: the first `units` units (the others are dealt whole).
struct Runs {
  const Problem& p;
  const Work& w;
  int64_t pre, units = 0;
  int64_t size() const { return w.joined ? w.blocks : 2 * (int64_t)p.G; }
  Run at(int64_t i) const {
    if (!w.joined) {   // a kv head's blocks of two row tiles, then the one that may have one
      const bool last = i & 1;
      return {last ? w.alt : w.blocks - w.alt, pre, last ? Shares::kTileAlt : Shares::kTile};
    }
    const int blk = w.blocks - 1 - (int)i;
    const int64_t per = (int64_t)p.B * p.G;
    return {clamp64(units - i * per, 0, per), most_tiles(p, blk, (int)pre),
            w.is_alt(blk) ? Shares::kTileAlt : Shares::kTile};
  }
  int64_t total() const {
    int64_t t = 0;
    for (int64_t i = 0; i < size(); ++i) t += at(i).count * at(i).cost();
    return t;
  }
};

// Cuts the list into s.ctas shares (each is to have a tile's cost at least).  Returns the most fragments of a unit.
int cut(const Runs& runs, int64_t total, Shares& s) {
  int64_t i = 0, first = 0, begin = 0;   // run, its first unit, and where that begins
  Run run = runs.at(0);
  int most = 1;
  for (int c = 0; c <= s.ctas; ++c) {
    const int64_t t = total / s.ctas * c + total % s.ctas * c / s.ctas;
    while (i + 1 < runs.size() && t - begin >= run.count * run.cost()) {
      begin += run.count * run.cost();
      first += run.count;
      run = runs.at(++i);
    }
    const int64_t k = clamp64((t - begin) / run.cost(), 0, run.count);   // the units in front, of this run
    const int64_t at = (t - begin - k * run.cost()) / run.tile;
    const bool next = k < run.count && at >= run.tiles;   // in a unit's end
    s.unit[c] = (int)(first + k + next);
    s.tile[c] = next || k == run.count ? 0 : (int)at;
    if (c > 0 && s.tile[c - 1] > 0 && s.unit[c] > s.unit[c - 1]) s.cut[s.n_cut++] = (int16_t)(c - 1);
    if (c == s.ctas) break;
    s.frag[c] = 0;
    if (s.tile[c] > 0) {   // one more than the last share's, where that began in the unit too
      s.frag[c] = (int16_t)(s.unit[c - 1] == s.unit[c] ? s.frag[c - 1] + 1 : 1);
      most = s.frag[c] + 1 > most ? s.frag[c] + 1 : most;
    }
  }
  return most;
}

// The number of parts of entry items' lists of `tiles` key tiles that takes the least time, at most four items a CTA (the
// lists may turn out short); part_us: a partial result of every row, written and read.
int best_parts(int64_t items, int64_t tiles, bool alt, double part_us, double* us) {
  int best = 1;
  *us = 0;
  for (int n = 1; n <= kMaxParts && n <= tiles && (n == 1 || items * n <= 4 * kSms); ++n) {
    const double list = (double)(ceil_div(tiles, n) * (alt ? Shares::kTileAlt : Shares::kTile) + Shares::kEnd) * kUnit;
    const double t = (double)ceil_div(items * n, kSms) * list + n * part_us;
    if (n == 1 || t < *us) {
      *us = t;
      best = n;
    }
  }
  return best;
}

size_t round256(size_t x) { return (x + 255) / 256 * 256; }

int64_t kept_rows(const Problem& p, const Work& w) {
  return w.joined ? (int64_t)w.list.ctas * 2 * 2 * kRows : (int64_t)p.B * p.H * p.Sq * w.splits;
}

}  // namespace
}  // namespace shr

bool shared_tc_plan(const Problem& p, int page_size, shr::Work& w) {
  using namespace shr;
  if (p.dtype != ATTN_BF16 && p.dtype != ATTN_F16) return false;
  if (p.kv_int8 || (p.D != 64 && p.D != 128) || p.Sk < 1 || page_size % 8) return false;
  const int64_t rows = (int64_t)p.Sq * p.qpg, all = rows * p.B;
  if (all > (1 << 30) || all * p.G > (1ll << 31)) return false;
  w = Work{};
  w.piece = kKeys;
  while (page_size % w.piece) w.piece /= 2;
  const int64_t pre = ceil_div(p.prefix, kKeys), own = ceil_div(p.Sk - p.prefix, kKeys);
  const double part_us = (double)(all * p.G) * p.D * 8 / 6.0e6;   // a partial result of every row, written and read
  auto has_half = [](int64_t n) { return (int)((n - 1) % (2 * kRows) < kRows); };   // the last block has one row tile
  // One query an entry, the decode pass can take the prefix's keys too; it starts some 7 us faster than the two passes side
  // by side and their merge (of 163 shapes the one that this says takes 0.35 % longer than the better one on average).
  const double us_each = shr::decode_us(p, p.qpg > 8 ? 16 : 8, 2, 10.9e6, 8192) - 2.0;
  // The prefix once for the packed rows of all entries.
  double us_packed = INFINITY;
  if (pre > 0) {
    w.blocks = (int)ceil_div(all, 2 * kRows);
    w.alt = has_half(all);
    const Runs runs{p, w, pre};
    const int64_t total = runs.total();
    int ctas = kSms;
    bool own_all = false;
    if (p.Sq == 1 && own > 0) {
      // The decode pass over pages takes the own keys, side by side with the prefix's: each gets SMs by its cost, own
      // lists being half as long as they can be (a unit's end costs the decode pass 2 us, three CTAs an SM; beside it
      // the prefix's tiles take half as long again).  As many CTAs for each unit, where they are alike, so that no CTA
      // has parts of two.  64 entries of 32/8 heads behind 8192 keys with up to 1024 own ones, by CTAs of the prefix's:
      // 32 59.5 us, 40 54.0, 48 49.8, 56 48.8, 64 47.7, 72 58.3, and between these 41 57.3, 50 54.8; 32 entries behind
      // 131072 with up to 512: 104 104.1, 120 104.2, 136 106.1.
      const int64_t units = (int64_t)p.B * p.G * ceil_div(p.qpg, p.qpg > 8 ? 16 : 8);
      const double us_own = (double)p.B * p.G * (p.Sk - p.prefix) * p.D * 2 / 6.0e6 + (double)units * 2.0 / (3 * kSms);
      const double us_all = 1.5 * (double)total * kUnit / kSms;
      ctas = (int)(kSms * (us_all + kPass) / (us_all + us_own + 2 * kPass));
      // No fewer than a third of the SMs: how many own keys there are is not known here, but that they may be many.
      // Then the decode pass is planned for all SMs: its last CTAs follow the prefix's.
      const int alike = w.blocks * p.G;
      if (ctas < kSms / 3) ctas = kSms / 3;
      if ((w.blocks == 1 || !w.alt) && alike < kSms && 2 * ctas > alike) {
        ctas = (ctas + alike / 2) / alike * alike;
        if (ctas >= kSms) ctas -= alike;
      }
      const double us_first = kPass + us_all * kSms / ctas, us_beside = us_own * kSms / (kSms - ctas);
      own_all = us_first + us_own < (us_first > us_beside ? us_first : us_beside);
    }
    w.list.ctas = (int)clamp64(total / (2 * Shares::kTile), 1, ctas);
    us_packed = kPass + kMerge + (double)total / w.list.ctas * kUnit + part_us;
    if (p.Sq == 1 && us_packed > us_each) return false;
    w.own_slot = cut(runs, total, w.list);
    us_packed += (w.own_slot - 1) * part_us;
    w.one_tile = all <= kRows;
    w.own_sms = own_all ? kSms : kSms - w.list.ctas;
  }
  if (p.Sq == 1) {
    w.parts_b = own > 0;
    w.splits = w.own_slot + w.parts_b;
    return us_packed <= us_each;
  }
  w.blocks_b = (int)ceil_div(rows, 2 * kRows);
  w.alt_b = has_half(rows);
  const int64_t items = w.blocks_b * (int64_t)p.G * p.B;
  if (items > 0x3fffffff / kMaxParts) return false;
  // What is compared below is with own lists of some 2048 keys at most: how many there are is not known here, and where they
  // are many, both divide them alike (16 entries of 5 tokens behind 20480 keys with 320 own ones: 46.7 us, or 129.5 each
  // by itself, as room for 131072 own keys had it decided).
  Problem e = p;
  e.Sk = p.prefix + (int)clamp64(p.Sk - p.prefix, 0, p.Sq + 1024 < 2048 ? 2048 : (int64_t)p.Sq + 1024);
  double us_own = 0;
  if (own > 0) best_parts(items, ceil_div(e.Sk - e.prefix, kKeys), rows <= kRows, part_us, &us_own);
  us_packed += us_own;
  w.parts_b = own > 0 ? best_parts(items, own, rows <= kRows, part_us, &us_own) : 0;
  w.n_b = (int)items * w.parts_b;
  w.splits = w.own_slot + w.parts_b;
  // Or each entry by itself: its rows walk the prefix and their own keys.
  Work v{};
  v.joined = 1;
  v.piece = w.piece;
  v.blocks = v.blocks_b = w.blocks_b;
  v.alt = v.alt_b = w.alt_b;
  v.parts_b = 1;
  v.one_tile = rows <= kRows;
  const double us_all = (double)Runs{e, v, pre, items}.total() * kUnit;
  const Runs left{e, v, pre, items % kSms};
  const int64_t total = left.total();
  const int ctas = (int)clamp64(total / (2 * Shares::kTile), 1, kSms);
  // Cut units cost the write and the read of about a fragment and a half a share, and the merge; uncut ones leave SMs
  // without work for most of a unit's time.
  const double us_cut = kMerge + (double)ctas * 3 * kRows * p.D * 8 / 6.0e6;
  int64_t longest = 0;
  for (int64_t i = 0; i < left.size(); ++i) {
    const Run run = left.at(i);
    if (run.count > 0 && run.cost() > longest) longest = run.cost();
  }
  const double us_left = (double)(longest * kSms - total) / kSms * kUnit;
  double us_joined = kPass + us_all / kSms + us_left;
  v.n_b = (int)items;
  if (us_cut < us_left) {
    us_joined = kPass + us_all / kSms + us_cut;
    v.list.ctas = ctas;
    v.first_b = (int)(items % kSms);
    v.n_b = (int)(items - v.first_b);
    const Runs runs{p, v, pre, items % kSms};
    v.splits = cut(runs, runs.total(), v.list) > 1;
  }
  if (!(us_packed < us_joined)) w = v;
  return true;
}

size_t shared_tc_bytes(const Problem& p, const shr::Work& w) {
  using namespace shr;
  if (w.splits == 0) return 0;
  const size_t rows = (size_t)kept_rows(p, w);
  return round256(rows * p.D * sizeof(float)) + 2 * round256(rows * sizeof(float)) +
         round256(w.joined ? 0 : (size_t)w.blocks * p.G * sizeof(int));
}

int shared_tc_try(const Problem& p, const Ext& x, shr::Work& w, const Problem& own, const Ext& x_own, void* workspace,
                  cudaStream_t st, int* used) {
  using namespace shr;
  *used = 0;
  const int pages = (int)min(x.n_pages, 0x7fffffffu);
  const float sc = p.scale * 1.4426950408889634f;
  if (pages < 1 || pages == 0x7fffffff || !(sc == sc) || isinf(sc)) return ATTN_OK;
  if (!tma_layout_ok(p.Q, p.q, p.Sq, p.H, p.B) || !tma_layout_ok(p.K, p.k, x.page_size, p.G, pages) ||
      !tma_layout_ok(p.V, p.v, x.page_size, p.G, pages) || !tma_layout_ok(p.O, p.o, p.Sq, p.H, p.B))
    return ATTN_OK;
  if (w.splits > 0) {
    const int64_t rows = kept_rows(p, w);
    char* at = static_cast<char*>(workspace);
    w.part_o = reinterpret_cast<float*>(at);
    at += round256(rows * p.D * sizeof(float));
    w.part_m = reinterpret_cast<float*>(at);
    at += round256(rows * sizeof(float));
    w.part_l = reinterpret_cast<float*>(at);
    w.note = reinterpret_cast<int*>(at + round256(rows * sizeof(float)));
  }
  int rc = p.D == 64 ? shared_tc64(p, x, w, st) : shared_tc128(p, x, w, st);
  if (rc < 0) return ATTN_OK;  // tensor map refused: another pass
  *used = 1;
  if (rc) return rc;
  paged::Work decode{};
  const bool decoded = p.Sq == 1 && own.Sk > 0;
  if (decoded) {   // (its types and layouts are among the ones checked above)
    const paged::OwnPart part{w.part_o + (int64_t)w.own_slot * p.D, w.part_m + w.own_slot, w.part_l + w.own_slot,
                              w.splits, w.own_sms, nullptr};
    void* ws = static_cast<char*>(workspace) + shared_tc_bytes(p, w);
    if (!paged_own(own, x_own, part, ws, st, &decode, &rc)) return ATTN_ERR_UNSUPPORTED;
    if (rc) return rc;
  }
  if (w.splits == 0) return ATTN_OK;
  return launch_shared_merge(p, w, decoded ? &decode : nullptr, st) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace attn
