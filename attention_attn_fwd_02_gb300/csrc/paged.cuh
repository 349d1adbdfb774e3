// paged.cuh -- how the decode passes over a paged cache share their work.
//
// The visible keys of a batch entry are a list of key tiles (visible.cuh).
// Every (batch entry, kv head, chunk of its query heads) -- a unit -- walks its
// entry's list, and the lists of all units, laid end to end, are cut into
// shares of equal cost, one a CTA (a unit's end costs about what a tile does):
// every SM streams as long as the others whatever the entries' lengths, one
// launch fits short and long caches, and a CTA's fixed cost is paid once.  A share's piece of a unit is a fragment.  A
// fragment that holds its unit's whole list writes the unit's rows of O; a CTA
// has at most two others (its first and its last), whose partial results go
// to two slots of the workspace, and the join kernel merges the fragments of a
// unit in list order.  The cut depends on the lengths alone, so results are
// deterministic.
//
// Short lists have no fragments and no join.  Few units: a unit is a thread-block
// cluster's of 2 to 8 CTAs, each with a part of its list, which merges the
// parts through distributed shared memory.  Many: a CTA takes whole units, one
// after the other.
#pragma once

#include "visible.cuh"

namespace attn {
namespace paged {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kSms = 152;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kSlack = 8.0f;   // log2 units: how far a score may rise above a reference that is a maximum
constexpr unsigned kAll = 0xffffffffu;

// How a pass's CTAs divide the units: equal shares of all tiles, a cluster a
// unit, or whole units in turn.
enum { kShares = 0, kCluster = 1, kWhole = 2 };

// A unit cut by shares, noted by the share that ends it: its fragments are the
// last one of share c0 (slot 1 when that share began in front of the unit),
// all of the shares between, and the first one of the noting share.
struct CutUnit {
  int b, u;   // b < 0: the share ends no cut unit
  int c0, late;
};

struct Work {
  Problem p;
  Ext x;
  int unit;        // keys of a tile
  int heads;       // query heads of a unit (at most)
  int n_hc;        // chunks of a kv head's query heads
  int ctas;        // shares
  float* part_o;   // [ctas][2][heads][D]
  float* part_m;   // [ctas][2][heads]  natural maxima (-inf: no visible key)
  float* part_l;   // [ctas][2][heads]  sums (maxima apart: Split::part_l says why)
  CutUnit* cuts;   // [ctas]
  int cluster;     // > 0: CTAs of the cluster that holds one unit (no shares)
  int stride;      // > 0: CTA c takes the units c, c + stride, ... (no shares)
};

__device__ __forceinline__ int entry_tiles(const Work& w, int b) {
  return tile_list(row_vis(w.p, w.x.first, b, 0), w.unit).n;
}

// What a unit with n tiles costs, in tiles: its end (merge, output, the next unit's queries) counts as kEnd more.
// (3 against 1: 256 entries of up to 1000 rows, cut into shares, 106 -> 98 us, the batch of 64 181.0 -> 180.5.)
constexpr int kEnd = 3;
__device__ __forceinline__ int unit_cost(int n) { return n > 0 ? n + kEnd : 0; }

// Shares: CTA c of n takes what lies in [c * total / n, (c + 1) * total / n) of the costs.
__device__ __forceinline__ int64_t share_begin(int64_t total, int n, int c) { return total * c / n; }
__device__ __forceinline__ int share_of(int64_t total, int n, int64_t at) {
  return (int)(((at + 1) * n - 1) / total);
}

// A place in the list of all units: unit u of entry b, tile `tile` of its n.
struct Cursor {
  int b, u, tile, n;
  Vis v;
  TileList tl;

  __device__ __forceinline__ void load(const Work& w) {
    v = row_vis(w.p, w.x.first, b, 0);
    tl = tile_list(v, w.unit);
    n = tl.n;
  }
  // To the first tile of unit `id`, or of the next one w.stride behind it that has tiles.  False: there is none.
  __device__ __forceinline__ bool at_unit(const Work& w, int units, int64_t id) {
    tile = 0;
    for (; id < (int64_t)w.p.B * units; id += w.stride) {
      b = (int)(id / units);
      u = (int)(id - (int64_t)b * units);
      load(w);
      if (n > 0) return true;
    }
    return false;
  }
  // To the next tile; the caller stays inside the total.
  template <int MODE>
  __device__ __forceinline__ void next(const Work& w, int units) {
    if (++tile < n) return;
    tile = 0;
    if constexpr (MODE == kCluster) return;   // (a cluster has one unit)
    if constexpr (MODE == kWhole) {
      at_unit(w, units, (int64_t)b * units + u + w.stride);
      return;
    }
    if (++u < units) return;
    u = 0;
    do ++b;
    while (b + 1 < w.p.B && entry_tiles(w, b) == 0);
    if (b < w.p.B) load(w);
  }
};

// A share: the total of the costs, the number of shares and where this one begins.
struct Share {
  int64_t total, t0;
  int shares;
};
// The sum over a warp's lanes of x >= 0, in 64 bits.
__device__ __forceinline__ int64_t warp_sum(int x) {
  return __reduce_add_sync(kAll, x & 0xffff) + ((int64_t)__reduce_add_sync(kAll, x >> 16) << 16);
}
// CTA cta's share, its first tile and how many it has.  Warp-wide: the lanes hold 32 entries at a time.
__device__ __forceinline__ int find_share(const Work& w, int units, int cta, int lane, Share& s, Cursor& out) {
  const int n0 = lane < w.p.B ? entry_tiles(w, lane) : 0;
  int64_t all = warp_sum(unit_cost(n0));
  for (int base = 32; base < w.p.B; base += 32)
    all += warp_sum(base + lane < w.p.B ? unit_cost(entry_tiles(w, base + lane)) : 0);
  s.total = all * units;
  s.shares = (int)min((int64_t)w.ctas, s.total);
  if (cta >= s.shares) return 0;
  s.t0 = share_begin(s.total, s.shares, cta);
  const int64_t t1 = share_begin(s.total, s.shares, cta + 1);
  int64_t before = 0, filled = 0;    // costs and entries with tiles of the chunks so far
  int64_t from = -1, to = -1;        // tiles in front of t0 and t1
  for (int base = 0; to < 0 && base < w.p.B; base += 32) {
    const int n = base == 0 ? n0 : base + lane < w.p.B ? entry_tiles(w, base + lane) : 0;
    const unsigned some = __ballot_sync(kAll, n > 0);
    int64_t cost = unit_cost(n);   // inclusive sum
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(kAll, cost, o);
      if (lane >= o) cost += y;
    }
    // The entry of this chunk that holds place t: its lane; u and tile there.
    auto place = [&](int64_t t, int l, int& u, int& tile) {
      const int own = __shfl_sync(kAll, n, l), c = unit_cost(own);
      const int64_t front = before + __shfl_sync(kAll, cost, l) - c, rem = t - front * units;
      u = (int)(rem / c);
      tile = (int)(rem - (int64_t)u * c);
      return (front - kEnd * (filled + __popc(some & ((1u << l) - 1u)))) * units + (int64_t)u * own + min(tile, own);
    };
    int u, tile;
    const unsigned h0 = __ballot_sync(kAll, (before + cost) * units > s.t0);
    if (from < 0 && h0) {
      out.b = base + __ffs(h0) - 1;
      from = place(s.t0, __ffs(h0) - 1, out.u, out.tile);
    }
    const unsigned h1 = __ballot_sync(kAll, (before + cost) * units > t1 - 1);
    if (h1) {   // tiles up to and with place t1 - 1
      to = place(t1 - 1, __ffs(h1) - 1, u, tile);
      to += tile < __shfl_sync(kAll, n, __ffs(h1) - 1);
    }
    before += __shfl_sync(kAll, cost, 31);
    filled += __popc(some);
  }
  if (to <= from) return 0;
  out.load(w);
  if (out.tile >= out.n) {   // t0 is at a unit's end
    out.tile = out.n - 1;
    out.template next<kShares>(w, units);
  }
  return (int)(to - from);
}

// Copies 16 bytes to shared memory without waiting; sz = 0 writes zeros and reads nothing.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int sz) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(sz) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// The 16-byte unit u of row r of a stage, in bytes: swizzled so that the same
// unit of 8 neighbouring rows lies in different banks.
template <int UNITS>
__device__ __forceinline__ uint32_t swz(int r, int u) {
  return (uint32_t)(r * UNITS * 16 + ((u ^ (UNITS >= 8 ? r & 7 : (r >> 1) & 3)) << 4));
}

// A warp's ring of stages.  Each holds KEYS keys of a tile, rows of ROW bytes
// (elements of ES): K rows, then V rows.  Rows are copied with cp.async from wherever the page
// list puts them; rows that are hidden or have no page arrive as zeros, and
// nothing is read for them.
template <int ROW, int ES, int KEYS, int STAGES, int MODE>
struct Ring {
  static constexpr int kUnits = ROW / 16;
  static constexpr int kStage = 2 * KEYS * ROW;
  static constexpr int kBytes = kWarps * STAGES * kStage;
  static constexpr int kTile = kWarps * KEYS;
  static constexpr uint32_t kAllKeys = KEYS == 32 ? 0xffffffffu : (1u << (KEYS & 31)) - 1u;
  const Work& w;
  Cursor in;               // the next tile to copy
  const uint8_t *kbase, *vbase;
  uint32_t ring;           // shared-memory address of this warp's stages
  int* key;                // [STAGES] first key of a stage
  uint32_t* vis;           // [STAGES] its visible keys, bit r = row r
  int units, warp, lane, page;
  bool one_page, same;

  __device__ __forceinline__ Ring(const Work& work, const Cursor& at, int n_units, uint8_t* smem, int* keys,
                                  uint32_t* masks)
      : w(work), in(at), units(n_units), warp(threadIdx.x / 32), lane(threadIdx.x % 32) {
    const Problem& p = w.p;
    kbase = static_cast<const uint8_t*>(p.K) + p.k.off * ES;
    vbase = static_cast<const uint8_t*>(p.V) + p.v.off * ES;
    ring = smem_u32(smem) + warp * STAGES * kStage;
    key = keys + warp * STAGES;
    vis = masks + warp * STAGES;
    one_page = w.x.page_size % KEYS == 0;   // a stage's keys share a page
    same = p.k.bs == p.v.bs && p.k.hs == p.v.hs && p.k.rs == p.v.rs;
    look_up();
  }
  // The page of row lane % KEYS of the next tile.
  __device__ __forceinline__ void look_up() {
    const int k = in.tl.tile(in.tile) * kTile + warp * KEYS + lane % KEYS;
    page = visible(in.v, k) ? page_of(w.x, in.b, k) : -1;
  }
  // Copies the next tile into stage s; with `more` moves on and looks up the pages of the tile behind it.
  __device__ __forceinline__ void issue(int s, bool more) {
    const Problem& p = w.p;
    const int k0 = in.tl.tile(in.tile) * kTile + warp * KEYS, kr = lane % KEYS;
    const uint32_t mask = __ballot_sync(kAll, page >= 0);
    const int g = in.u / w.n_hc, r = k0 + kr - page_index(w.x, k0 + kr) * w.x.page_size, pg = max(page, 0);
    const int64_t ko = ((int64_t)pg * p.k.bs + (int64_t)g * p.k.hs + (int64_t)r * p.k.rs) * ES;
    const int64_t vo = same ? ko : ((int64_t)pg * p.v.bs + (int64_t)g * p.v.hs + (int64_t)r * p.v.rs) * ES;
    if (lane == 0) {
      key[s] = k0;
      vis[s] = mask;
    }
    const uint32_t dst = ring + s * kStage;
    constexpr int kPasses = KEYS * kUnits / 32;
    if constexpr (kUnits <= 32) {
      // One pass of the lanes copies kRowsPer rows; its swizzle differs from the first pass's by a constant.
      constexpr int kRowsPer = 32 / kUnits;
      const int u = lane % kUnits, ru = lane / kUnits;
      const uint32_t sw = swz<kUnits>(ru, u);
      auto place = [&](int j) { return dst + (sw ^ (kUnits >= 8 ? ((j * kRowsPer) & 7) << 4 : 0)) + j * kRowsPer * ROW; };
      if (one_page && (mask & kAllKeys) == kAllKeys) {
        // Every row of one page: the addresses advance by the row stride.
        const uint8_t* ks = kbase + __shfl_sync(kAll, ko, 0) + (int64_t)ru * p.k.rs * ES + u * 16;
        const uint8_t* vs = vbase + __shfl_sync(kAll, vo, 0) + (int64_t)ru * p.v.rs * ES + u * 16;
        const int64_t kst = (int64_t)kRowsPer * p.k.rs * ES, vst = (int64_t)kRowsPer * p.v.rs * ES;
#pragma unroll
        for (int j = 0; j < kPasses; ++j, ks += kst) copy16(place(j), ks, 16);
#pragma unroll
        for (int j = 0; j < kPasses; ++j, vs += vst) copy16(place(j) + KEYS * ROW, vs, 16);
      } else {
#pragma unroll
        for (int j = 0; j < kPasses; ++j) {
          const int row = j * kRowsPer + ru;
          const int64_t a = __shfl_sync(kAll, ko, row), c = same ? a : __shfl_sync(kAll, vo, row);
          const int sz = (mask >> row) & 1u ? 16 : 0;
          copy16(place(j), kbase + a + u * 16, sz);
          copy16(place(j) + KEYS * ROW, vbase + c + u * 16, sz);
        }
      }
    } else {   // rows of 64 units: two passes a row
#pragma unroll
      for (int j = 0; j < kPasses; ++j) {
        const int row = j / (kUnits / 32), u = j % (kUnits / 32) * 32 + lane;
        const int64_t a = __shfl_sync(kAll, ko, row), c = same ? a : __shfl_sync(kAll, vo, row);
        const int sz = (mask >> row) & 1u ? 16 : 0;
        copy16(dst + swz<kUnits>(row, u), kbase + a + u * 16, sz);
        copy16(dst + KEYS * ROW + swz<kUnits>(row, u), vbase + c + u * 16, sz);
      }
    }
    if (more) {
      in.template next<MODE>(w, units);
      look_up();
    }
  }
};

// Where a row's finished fragment goes.  M: reference maximum in the units of
// Scores<NAT> (-inf: no visible key), L: sum relative to it, a: numerator of element d.
template <typename T, bool NAT>
__device__ __forceinline__ void put_row(const Work& w, bool whole, int cta, int slot, int b, int h, int hh, int d,
                                        float M, float L, float a) {
  const Problem& p = w.p;
  M = Scores<NAT>::natural(M);
  if (!whole) {
    const int64_t at = ((int64_t)cta * 2 + slot) * w.heads + hh;
    const bool none = L == 0.f;
    w.part_o[at * p.D + d] = none ? 0.f : a / L;
    if (d == 0) {
      w.part_m[at] = none ? -INFINITY : M;
      w.part_l[at] = L;
    }
    return;
  }
  if (p.sink_on) a *= fold_sink<false>(M, L, sink_logit(p, h));
  const bool none = L == 0.f;
  static_cast<T*>(p.O)[p.o.off + (int64_t)b * p.o.bs + (int64_t)h * p.o.hs + d] =
      from_f32<T>(none ? (p.masked_zero ? 0.f : NAN) : a / L);
  if (p.lse && d == 0)
    p.lse[(int64_t)b * p.lse_bs + (int64_t)h * p.lse_hs] = none ? -INFINITY : Scores<NAT>::lse(M, log2f(L));
}

// What a row without a visible key returns, for all heads of entry b.  The
// CTA's threads share it.
template <typename T>
__device__ __forceinline__ void fill_entry(const Work& w, int b) {
  const Problem& p = w.p;
  for (int x = threadIdx.x; x < p.H * p.D; x += kThreads) {
    const int h = x / p.D, d = x - h * p.D;
    float M = -INFINITY, L = 0.f;
    if (p.sink_on) fold_sink<false>(M, L, sink_logit(p, h));
    const bool none = L == 0.f;
    static_cast<T*>(p.O)[p.o.off + (int64_t)b * p.o.bs + (int64_t)h * p.o.hs + d] =
        from_f32<T>(none ? (p.masked_zero ? 0.f : NAN) : 0.f / L);
    if (p.lse && d == 0)
      p.lse[(int64_t)b * p.lse_bs + (int64_t)h * p.lse_hs] = none ? -INFINITY : M + logf(L);
  }
}

// What every CTA of a pass without clusters does beside its units: its entries
// without a visible key.
template <typename T>
__device__ __forceinline__ void fill_entries(const Work& w, int cta) {
  for (int b = cta; b < w.p.B; b += w.ctas)
    if (entry_tiles(w, b) == 0) fill_entry<T>(w, b);
}

// Notes a cut unit that ends in share `cta` (whose first fragment it is), `first` tiles into its list.
__device__ __forceinline__ void note_cut(const Work& w, const Share& s, int cta, const Cursor& c, int first) {
  const int64_t at = s.t0 - first;
  const int c0 = share_of(s.total, s.shares, at);
  // (Share c0 has a fragment in front of it if it begins in front of the last unit's end.)
  w.cuts[cta] = {c.b, c.u, c0, share_begin(s.total, s.shares, c0) < at - kEnd ? 1 : 0};
}

// ---- units held by a cluster ----

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The float at the same place of CTA `rank`'s shared memory.
__device__ __forceinline__ float peer(const float* p, uint32_t rank) {
  uint32_t a = (uint32_t)__cvta_generic_to_shared(p), r;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(r) : "memory");
  return v;
}

// A CTA's part of a unit in shared memory: numerators [heads][D], then
// reference maxima [heads] and sums [heads].
struct Part {
  float *a, *m, *l;
  __device__ __forceinline__ Part(void* base, int heads, int D)
      : a(static_cast<float*>(base)), m(a + heads * D), l(m + heads) {}
  __device__ __forceinline__ void put(int D, int hh, int d, float M, float L, float x) const {
    a[hh * D + d] = x;
    if (d == 0) {
      m[hh] = M;
      l[hh] = L;
    }
  }
};

// Lets the kernel behind this one in the stream start its prologue, and waits
// in that kernel until everything in front of it is done and visible.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// Merges the parts of the unit (b, heads h0 ..) that the cluster's CTAs hold; each CTA writes its share of the rows.
template <typename T, bool NAT>
__device__ __forceinline__ void cluster_join(const Work& w, const Part& part, int b, int h0, int nh) {
  const int D = w.p.D, n = w.cluster;
  cluster_sync();
  for (int x = cluster_rank() * kThreads + threadIdx.x; x < nh * D; x += n * kThreads) {
    const int hh = x / D, d = x - hh * D;
    float m[8], l[8], a[8], M = -INFINITY, L = 0.f, A = 0.f;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      m[q] = q < n ? peer(part.m + hh, q) : -INFINITY;
      l[q] = q < n ? peer(part.l + hh, q) : 0.f;
      a[q] = q < n ? peer(part.a + x, q) : 0.f;
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) M = fmaxf(M, m[q]);
    const float mu = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float f = Scores<NAT>::weight(m[q], mu);
      L = fmaf(f, l[q], L);
      A = fmaf(f, a[q], A);
    }
    put_row<T, NAT>(w, true, 0, 0, b, h0 + hh, hh, d, M, L, A);
  }
  cluster_sync();   // no CTA leaves while its part is being read
}

// Host: merges the fragments of cut units.  Enqueued right behind the pass.
cudaError_t launch_join(const Work& w, cudaStream_t st);

// Host: the work of a pass with `ctas` CTAs an SM.  A cluster a unit, of the most
// CTAs (8 to 2) with which all units run at once, if a CTA has at most 16 tiles,
// or 24 when the units fill half of the machine or are no more than four (whose
// many fragments a join would read in turn); else whole units, if a unit has at
// most 24 tiles and the rounds of units are no more than 12 tiles longer than
// equal shares; else shares, never more than there can be tiles.  Shares cost about 10
// us more (finding the place, fragments, the join), the others' CTAs wait for the
// longest list.  Device time, bf16, 32/8 heads, head_dim 128, shares against
// these: one sequence of 700 rows 10.9 -> 6.4 us, 25 of up to 1500 rows 26.9 ->
// 21.0, 12 of up to 6000 rows 41.8 -> 32.7 (clusters); 57 of 900 to 1000 rows
// 48.9 -> 38.6, 90 of up to 100 rows 19.9 -> 12.6 (whole units); the other way
// round, 8/8 heads: one sequence of 12000 rows 16.1 against 21.0 in clusters.
// (float32 passes take the same limits, which were measured in bf16 alone.)
inline void plan_work(Work& w, int tile, int heads, int ctas) {
  w.unit = tile;
  w.heads = heads;
  w.n_hc = (w.p.qpg + heads - 1) / heads;
  const int64_t units = (int64_t)w.p.B * w.p.G * w.n_hc, n = (int64_t)kSms * ctas;
  int64_t span = w.p.Sk;
  if (w.p.causal && w.p.window >= 0) {
    const int64_t seen = (int64_t)w.p.window + 1 + w.x.first + 2 * tile;   // both parts may end inside tiles
    span = seen < span ? seen : span;
  }
  const int64_t list = (span + tile - 1) / tile, most = units * list, rounds = (units + n - 1) / n;
  w.cluster = w.stride = 0;
  for (int c = 8; c > 1 && !w.cluster; --c)
    if (units * c <= n && list >= c && list <= (2 * units * c >= n || units <= 4 ? 24 : 16) * c) w.cluster = c;
  w.ctas = (int)(w.cluster ? units * w.cluster : most < 1 ? 1 : most < n ? most : n);
  if (!w.cluster && list <= 24 && (rounds < 2 || rounds * n * list <= most + 12 * n))
    w.stride = w.ctas = (int)(units < 1 ? 1 : units < n ? units : n);
}

// Host: enqueues a pass, and the join behind shares.
template <typename Kernel>
int launch_pass(Kernel kern, const Work& w, int smem, cudaStream_t st) {
  if (ensure_smem((const void*)kern, smem) != cudaSuccess) return ATTN_ERR_CUDA;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)w.cluster;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)w.ctas);
  c.blockDim = dim3(kThreads);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  c.attrs = &at;
  c.numAttrs = w.cluster ? 1 : 0;
  if (cudaLaunchKernelEx(&c, kern, w) != cudaSuccess) return ATTN_ERR_CUDA;
  return w.cluster || w.stride || launch_join(w, st) == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace paged

// Fast passes: *used = 1 when one took the problem.  bytes: workspace they need.
size_t paged_ws_bytes(const Problem& p, int first);
int paged_try(const Problem& p, const Ext& x, void* workspace, cudaStream_t st, int* used);

}  // namespace attn
