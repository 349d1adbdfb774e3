// visible.cuh -- key visibility of windows with first keys, and paged caches.
//
// A row's visible keys are [lo, fe) and [wl, hi): the first keys of its span
// and the keys from its window's left end to its diagonal.  A kernel takes the
// union over its rows, which has the same form, as a list of key tiles without
// the tiles in the gap, and a split pass takes an equal part of that list.
#pragma once

#include "common.cuh"

namespace attn {

// First keys and page lists, passed by value next to a Problem.
struct Ext {
  int first;             // first keys visible behind the window
  int page_size;         // 0: K and V are not paged
  uint32_t n_pages;
  const int32_t* table;
  int64_t table_stride;
  uint32_t div_mul;      // k / page_size = umulhi(k, div_mul) >> div_shift for 0 <= k < 2^31 (page_size > 1)
  int div_shift;
};

inline Ext make_ext(int first, const attn_pages* pages) {
  Ext x{first, 0, 0u, nullptr, 0, 0u, 0};
  if (!pages) return x;
  x.page_size = pages->page_size;
  x.n_pages = (uint32_t)pages->n_pages;
  x.table = pages->table;
  x.table_stride = pages->table_stride;
  // With 2^s < d <= 2^(s+1) and m = ceil(2^(32+s) / d) < 2^32: m d - 2^(32+s) < d <= 2^(s+1), so
  // floor(k m / 2^(32+s)) is exact while k < 2^31.
  const uint64_t d = (uint64_t)x.page_size;
  while ((uint64_t)2 << x.div_shift < d) ++x.div_shift;
  if (d > 1) x.div_mul = (uint32_t)((((uint64_t)1 << (32 + x.div_shift)) + d - 1) / d);
  return x;
}

__device__ __forceinline__ int page_index(const Ext& x, int k) {
  return x.page_size == 1 ? k : (int)(__umulhi((uint32_t)k, x.div_mul) >> x.div_shift);
}

// Visible keys [lo, fe) and [wl, hi).  When the two meet, fe = lo and [wl, hi)
// holds them all; a row whose window is behind every key has wl = hi = fe.
struct Vis {
  int lo, fe, wl, hi;
};

__device__ __forceinline__ Vis row_vis(const Problem& p, int first, int b, int i) {
  int64_t kl = p.Sk;
  if (p.klens) kl = clamp64((int64_t)p.klens[b] + p.klens_plus, 0, p.Sk);
  int64_t hi = kl, lo = 0, wl = 0;
  if (p.seg) lo = clamp64((int64_t)p.seg[(int64_t)b * p.seg_bs + i], 0, p.Sk);
  if (p.causal) {
    const int64_t diag = (int64_t)i + (p.align_klens ? kl - p.Sq : p.coff);
    hi = min(hi, max(diag + 1, (int64_t)0));
    if (p.window >= 0) wl = diag - p.window;
  }
  lo = min(lo, hi);
  wl = clamp64(wl, lo, hi);
  const int64_t fe = min(lo + first, hi);
  if (fe > lo && wl >= hi) return {(int)lo, (int)fe, (int)fe, (int)fe};   // the window is empty
  const bool gap = fe < wl && fe > lo;
  return {(int)lo, (int)(gap ? fe : lo), (int)(fe >= wl ? lo : wl), (int)hi};
}

__device__ __forceinline__ bool visible(const Vis& v, int k) {
  return (k >= v.wl && k < v.hi) || (k >= v.lo && k < v.fe);
}

// Whether every key of [a, z) is visible.
__device__ __forceinline__ bool within(const Vis& v, int a, int z) {
  return (a >= v.wl && z <= v.hi) || (a >= v.lo && z <= v.fe);
}

// The union of rows, from the ends over the rows that have one of first parts
// [f_lo, f_hi) and window parts [w_lo, w_hi) (low ends at INT_MAX, high ends
// negative where no row has one).
__device__ __forceinline__ Vis vis_union(int f_lo, int f_hi, int w_lo, int w_hi) {
  if (w_hi <= w_lo) return f_hi <= f_lo ? Vis{0, 0, 0, 0} : Vis{f_lo, f_hi, f_hi, f_hi};
  if (f_hi <= f_lo) return {w_lo, w_lo, w_lo, w_hi};
  const int lo = min(f_lo, w_lo);
  return f_hi < w_lo ? Vis{lo, f_hi, w_lo, w_hi} : Vis{lo, lo, lo, w_hi};
}

// The union's tiles of `unit` keys, in key order, without those of the gap.
struct TileList {
  int ta, na, tb, n;   // na tiles from tile ta, then n - na tiles from tile tb
  __device__ __forceinline__ int tile(int i) const { return i < na ? ta + i : tb + (i - na); }
};

__device__ __forceinline__ TileList tile_list(const Vis& u, int unit) {
  TileList t;
  t.ta = u.lo / unit;
  const int ea = u.fe > u.lo ? (u.fe + unit - 1) / unit : t.ta;   // end of the first part's tiles
  t.na = ea - t.ta;
  t.tb = max(u.wl / unit, ea);
  const int eb = (u.hi + unit - 1) / unit;
  t.n = t.na + (u.hi > u.wl ? max(eb - t.tb, 0) : 0);
  return t;
}

// Part `part` of `parts` of a list of n tiles: [begin, end).
__device__ __forceinline__ void list_part(int n, int part, int parts, int& begin, int& end) {
  begin = (int)((int64_t)n * part / parts);
  end = (int)((int64_t)n * (part + 1) / parts);
}

// Page of key k of entry b, or -1 when the entry's list names no page of the pool there.
__device__ __forceinline__ int page_of(const Ext& x, int b, int k) {
  const int32_t pg = __ldg(x.table + (int64_t)b * x.table_stride + page_index(x, k));
  return (uint32_t)pg < x.n_pages ? pg : -1;
}

// The CUDA-core forward with first keys and paged caches.
cudaError_t launch_simt_ext(const Problem& p, const Ext& x, const Split& s, cudaStream_t st);

// The tensor-core and float32 forwards with first keys: as prefill_tc_try.
int window_tc_try(const Problem& p, int first, const Split& sp, cudaStream_t st, int* used);
int window_f32_try(const Problem& p, int first, const Split& s, cudaStream_t st, int* used);

}  // namespace attn
