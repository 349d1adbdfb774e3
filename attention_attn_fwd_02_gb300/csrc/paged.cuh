// paged.cuh -- how the decode passes over a paged cache share their work.
//
// The visible keys of a batch entry are a list of key tiles (visible.cuh).
// Every (batch entry, kv head, chunk of its query heads) -- a unit -- walks its
// entry's list, and the lists of all units, laid end to end, are cut into
// equal shares, one a CTA: every SM streams the same number of cache bytes
// whatever the entries' lengths, one launch fits short and long caches, and a
// CTA's fixed cost is paid once.  A share's piece of a unit is a fragment.  A
// fragment that holds its unit's whole list writes the unit's rows of O; a CTA
// has at most two others (its first and its last), whose partial results go
// to two slots of the workspace, and the join kernel merges the fragments of a
// unit in list order.  The cut depends on the lengths alone, so results are
// deterministic.
#pragma once

#include "visible.cuh"

namespace attn {
namespace paged {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kSms = 152;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kSlack = 8.0f;   // log2 units: how far a score may rise above the reference maximum
constexpr unsigned kAll = 0xffffffffu;

struct Work {
  Problem p;
  Ext x;
  int unit;        // keys of a tile
  int heads;       // query heads of a unit (at most)
  int n_hc;        // chunks of a kv head's query heads
  int ctas;        // shares
  float* part_o;   // [ctas][2][heads][D]
  float* part_lse; // [ctas][2][heads]
};

__device__ __forceinline__ int entry_tiles(const Work& w, int b) {
  return tile_list(row_vis(w.p, w.x.first, b, 0), w.unit).n;
}

// Tiles of one unit of every entry in front of entry b (b = B: of all).  Warp-wide.
__device__ __forceinline__ int64_t tiles_before(const Work& w, int b, int lane) {
  int64_t n = 0;
  for (int i = lane; i < b; i += 32) n += entry_tiles(w, i);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(kAll, n, o);
  return n;
}

// Shares: CTA c of n takes tiles [c * total / n, (c + 1) * total / n).
__device__ __forceinline__ int64_t share_begin(int64_t total, int n, int c) { return total * c / n; }
__device__ __forceinline__ int share_of(int64_t total, int n, int64_t tile) {
  return (int)(((tile + 1) * n - 1) / total);
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
  // To the next tile; the caller stays inside the total.
  __device__ __forceinline__ void next(const Work& w, int units) {
    if (++tile < n) return;
    tile = 0;
    if (++u < units) return;
    u = 0;
    do ++b;
    while (b + 1 < w.p.B && entry_tiles(w, b) == 0);
    if (b < w.p.B) load(w);
  }
};

// The cursor at tile `at` of the whole list (at < total).  Warp-wide.
__device__ __forceinline__ Cursor seek(const Work& w, int64_t at, int units, int lane) {
  Cursor c;
  int64_t before = 0;
  c.b = 0;
  for (int base = 0; base < w.p.B; base += 32) {
    const int n = base + lane < w.p.B ? entry_tiles(w, base + lane) : 0;
    int64_t incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(kAll, incl, o);
      if (lane >= o) incl += y;
    }
    const unsigned hit = __ballot_sync(kAll, (before + incl) * units > at);
    if (hit) {
      const int l = __ffs(hit) - 1;
      c.b = base + l;
      before += __shfl_sync(kAll, incl - n, l);
      break;
    }
    before += __shfl_sync(kAll, incl, 31);
  }
  c.load(w);
  const int64_t rem = at - before * units;
  c.u = (int)(rem / c.n);
  c.tile = (int)(rem % c.n);
  return c;
}

// Copies 16 bytes to shared memory without waiting; sz = 0 writes zeros and reads nothing.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int sz) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(sz) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t smem_u32(const void* p) { return (uint32_t)__cvta_generic_to_shared(p); }

// Where a row's finished fragment goes.  M: reference maximum in log2 units
// (-inf: no visible key), L: sum relative to it, a: numerator of element d.
template <typename T>
__device__ __forceinline__ void put_row(const Work& w, bool whole, int cta, int slot, int b, int h, int hh, int d,
                                        float M, float L, float a) {
  const Problem& p = w.p;
  if (!whole) {
    const int64_t at = ((int64_t)cta * 2 + slot) * w.heads + hh;
    const bool none = L == 0.f;
    w.part_o[at * p.D + d] = none ? 0.f : a / L;
    if (d == 0) w.part_lse[at] = none ? -INFINITY : (M + log2f(L)) * kLn2;
    return;
  }
  if (p.sink_on) a *= fold_sink<true>(M, L, sink_logit(p, h) * kLog2e);
  const bool none = L == 0.f;
  static_cast<T*>(p.O)[p.o.off + (int64_t)b * p.o.bs + (int64_t)h * p.o.hs + d] =
      from_f32<T>(none ? (p.masked_zero ? 0.f : NAN) : a / L);
  if (p.lse && d == 0)
    p.lse[(int64_t)b * p.lse_bs + (int64_t)h * p.lse_hs] = none ? -INFINITY : (M + log2f(L)) * kLn2;
}

// Host: merges the fragments of the units that no single share holds, and
// fills the rows of entries without a visible key.
cudaError_t launch_join(const Work& w, cudaStream_t st);

}  // namespace paged

// Fast passes: *used = 1 when one took the problem.  bytes: workspace they need.
size_t paged_ws_bytes(const Problem& p);
int paged_try(const Problem& p, const Ext& x, void* workspace, cudaStream_t st, int* used);

}  // namespace attn
