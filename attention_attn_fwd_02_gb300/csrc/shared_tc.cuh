// shared_tc.cuh -- f16/bf16 attention of a batch over a shared prefix and each
// entry's own keys in a paged cache, head_dim 64 or 128, on the tensor cores.
//
// What it computes: O = softmax(scale Q K^T + mask) V and the LSE over the
// prefix's keys and the entry's own ones, or partial results of both that are
// merged by their maxima and sums.
//
// What bounds it: HBM for one token an entry, as a key tile of 128 x head_dim
// is read once for up to 256 rows of all entries (64 entries of 4 heads a kv
// head fill both row tiles); the tensor cores and the exponentials, as in the
// prefill kernel, once the rows are prompts.
//
// The tile step is the windowed kernel's (window_tc.cuh): a persistent CTA an
// SM, two 128-row tiles that ping-pong, S = Q K^T and O += P V as tcgen05 MMAs
// with TMEM accumulators, a thread to a row of S, P over S as packed pairs, a
// reference maximum that moves with a slack.  What is its own:
//   - a block of one row tile deals its key tiles to both row tiles of the
//     kernel in turn, so that one's softmax overlaps the other's products;
//   - K and V tiles are put together from a page list: a warp for K and one for
//     V, whose lanes look up a page each, a tile ahead, and issue a TMA box of
//     `piece` rows and 64 columns each (some 40 cycles a box).  A piece without a page is copied from a page
//     behind the pool: it arrives as zeros and counts its bytes;
//   - K and V tiles alternate in one ring of as many slots as the shared memory
//     holds: what is on its way bounds the rate that an SM reads at;
//   - Q rows come from wherever (entry, query, head) puts them, with cp.async
//     by the warp that finds the items, as soon as the item in front has taken
//     its last S: rows pack without gaps whatever the strides.  A CTA's first
//     queries are loaded by the softmax threads, a row each, which have nothing
//     else to do then (one warp takes 5 us for the rows, 256 threads 1).
// P enters the product as one value of the element type, as in attn_fwd and by
// choice: in two halves, as the decode pass takes it, a key tile would be three
// products instead of two, 2.0 us instead of 1.33 of an SM's tensor time with two row
// tiles, against 1.45 for its copy from HBM.  It costs 0.0023 instead of 0.0017
// relative error in bf16, 0.00029 instead of 0.00021 in f16 (the output's rounding alone).
//
// Measured (32 query heads over 8, head_dim 128, bf16): a key tile takes an SM
// 1.45 us from HBM, whether one row tile reads it or two (6.9 TB/s on all SMs),
// and 1.55 us for two row tiles out of L2 (1.65 PFLOP/s; one row tile 0.65 to
// 1.0).  A launch costs 12 to 15 us besides, most of it instruction fetch: a
// CTA's first S is there after 7 us, its first P 5 us later (0.9 from the second
// tile on), and the epilogue takes 3.  Four slots of the ring instead of five or six:
// 115 -> 107 us behind 131072 keys.  Prefetches of later tiles into L2 read
// half of HBM twice (537 -> 818 MB) and cost a third of the speed; a step of the
// softmax warps on nothing, to fetch their instructions early, gained nothing.
#pragma once

#include <type_traits>

#include "prefill_tc.h"
#include "shared.h"
#include "tc_ptx.cuh"
#include "tma.h"

namespace attn {
namespace shr {

using namespace tc;

constexpr int BM = kRows;
constexpr int BN = kKeys;
constexpr int kThreads = 384;
// Registers after the split, as in the prefill kernel: 8 warps x 216 and 4
// warps x 56 fit the 168 a thread that the block is launched with.
constexpr int kSoftmaxRegs = 216;
constexpr int kProducerRegs = 56;
constexpr int kSplitRegs = 8 * 32 * kSoftmaxRegs + 4 * 32 * kProducerRegs;
static_assert(kSplitRegs <= kThreads * ((65536 / kThreads) & ~7), "register split exceeds the block's registers");
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kSlack = 8.0f;     // log2 units
constexpr int kMaxSlots = 13;      // tiles of the ring
constexpr int kNotes = 16;         // key tiles whose pages are noted (see the copy of K)

// A row block's part of its tile list, as the roles read it.
struct Item {
  int b, g;              // b < 0: a prefix item
  int row0, rows;        // first row, and the rows there are
  int t0, np, o0, n;     // np prefix tiles from t0, then n - np own tiles from o0
  int turn;              // the list is walked from tile `turn` of it on, and round
  int n0;                // the tiles of row tile 0: the first n0 (not alt)
  int own_end;           // own keys that some row of the block sees
  int alt, some1, slot;  // key tiles in turn; row tile 1 has rows; the partial result (-1: O is written)
  // The i-th tile of the walk: whether it is the prefix's, and its first key there.
  __device__ __forceinline__ int key(int i, bool& pre) const {
    i += i < n - turn ? turn : turn - n;
    pre = i < np;
    return (pre ? t0 + i : o0 + i - np) * kKeys;
  }
  __device__ __forceinline__ bool has(int t, int i) const {
    return alt ? (i & 1) == t : t ? some1 != 0 : i < n0;
  }
};

struct Bars {
  uint64_t q_first, q_full, q_empty;
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  uint64_t s_full[2], p_full[2], o_done[2];
  uint64_t item_full[2], item_empty[2];
  uint64_t pair_have, pair_done;
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
};

template <int D>
struct Cfg {
  static constexpr int kChunks = D / 64;                  // 64-column (128-byte) chunks
  static constexpr int kTile = 128 * D * 2;               // bytes of a tile of Q, K or V
  static constexpr int kTiles = D <= 64 ? 14 : 7;         // of shared memory: one or two of Q, the ring
  static constexpr int kSmem = kTiles * kTile;
  static constexpr int kS0 = 0, kS1 = BN, kO0 = 2 * BN, kO1 = 2 * BN + D;
  static_assert(2 * BN + 2 * D <= 512, "TMEM budget");
  static_assert(kTiles - 1 <= kMaxSlots && kNotes >= (kTiles - 1) / 2 + 4, "slots and notes");
};

// A place in the ring of n slots and its phase.
struct Slot {
  int s;
  uint32_t ph;
  __device__ __forceinline__ void next_tile(int n) {   // K's (or V's) slot of the next key tile
    s += 2;
    if (s >= n) {
      s -= n;
      ph ^= 1u;
    }
  }
};

// The lowest n bits (n may lie outside [0, 32]).
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }

// 32 bytes to global memory in one store (32-byte aligned).
__device__ __forceinline__ void store32(void* dst, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Own keys that row i of entry b sees: the first ones, up to its diagonal.
__device__ __forceinline__ int own_seen(const Problem& p, int b, int i) { return row_vis(p, 0, b, i).hi - p.prefix; }

// XF: scores under a mask, a softcap or a scale that is not positive.
template <int D, bool BF16, bool XF>
__global__ void __launch_bounds__(kThreads, 1)
    shared_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const Problem p, const Ext x, const __grid_constant__ Work w, const int wide_rows,
                     const int drop_first_copy) {
  using C = Cfg<D>;
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* q_s = smem_raw;   // (on a 1024-byte boundary: launch() has looked)
  const int n_slots = C::kTiles - (w.one_tile ? 1 : 2);
  uint8_t* ring = q_s + (C::kTiles - n_slots) * C::kTile;
  __shared__ Bars sb;
  __shared__ Item items[2];
  __shared__ uint2 notes[kNotes];        // of a key tile: which of its pieces have no page; its first key, + 1: the prefix's
  __shared__ float2 pair_ml[2][BM];      // items of one row tile: reference maxima and sums of both halves of the keys

  using S = Scores<XF>;   // (masks come with XF)
  constexpr float kRise = XF ? kSlack * kLn2 : kSlack;   // in the units of the scores
  // A row's reference is a maximum, less a lead where P is f16: p is 2^5 at that maximum, and what f16 cannot hold
  // (2^-25) is 2^-30 of the row's largest probability (window_tc.cuh).
  constexpr float kLead = (BF16 ? 0.f : 5.f) * (XF ? kLn2 : 1.f);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  __shared__ int items_a, my_items;   // this CTA's items of the list (in front), and all of its items

  paged::let_next_start();
  if (threadIdx.x == 32) {
    int n = 0;
    if (const int c = blockIdx.x; c < w.list.ctas) {
      const int u0 = w.list.unit[c], u1 = w.list.unit[c + 1], t0 = w.list.tile[c], t1 = w.list.tile[c + 1];
      n = u1 > u0 ? u1 - u0 + (t1 > 0) : t1 > t0;
    }
    items_a = n;
    my_items = n + max(0, (w.n_b - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x);
  }
  if (threadIdx.x == 0) {
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
    sb.abort = 0;
    for (int s = 0; s < kMaxSlots; ++s) {
      mbar_init(&sb.full[s], 1);
      mbar_init(&sb.empty[s], 1);
    }
    mbar_init(&sb.q_first, 2 * BM);
    mbar_init(&sb.q_full, 32);
    mbar_init(&sb.q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sb.s_full[i], 1);
      mbar_init(&sb.p_full[i], BM);
      mbar_init(&sb.o_done[i], 1);
      mbar_init(&sb.item_full[i], 32);
      mbar_init(&sb.item_empty[i], 3 + 2 * BM);   // the copy and MMA warps and every softmax thread
    }
    mbar_init(&sb.pair_have, 2 * BM);
    mbar_init(&sb.pair_done, 2 * BM);
    mbar_init(&sb.mma_done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 9) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(su32(&sb.tmem_base))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = sb.tmem_base;

  if (warp == 10) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
    // ---------------- items, and their queries ----------------
    constexpr int kUnits = D / 8, kRowsAt = 32 / kUnits;   // 16-byte units of a row; rows that a copy of all lanes takes
    const int c = min((int)blockIdx.x, kSms - 1);
    const int pre = p.prefix / BN + (p.prefix % BN > 0);   // the prefix's tiles
    int u = w.list.unit[c], tile = w.list.tile[c], walked = 0;
    for (int k = 0; k < my_items; ++k) {
      const int buf = k & 1;
      if (k >= 2 && !wait_warp(&sb.item_empty[buf], (uint32_t)((k >> 1) - 1) & 1u, &sb.abort, p.status)) break;
      Item it;
      it.turn = 0;
      if (!w.joined && k < items_a) {
        // The share's last unit first: it may walk its tiles from the first on, as all CTAs then do side by side, and the
        // others go on from where it ends (`walked`).  CTAs that read the same tiles at the same time read them out of
        // their die's L2.
        u = k == 0 ? w.list.unit[c] + items_a - 1 : w.list.unit[c] + k - 1;
        tile = u == w.list.unit[c] ? w.list.tile[c] : 0;
      }
      const bool ends = k < items_a && u == w.list.unit[c + 1];   // the share ends in the middle of the unit
      if (k < items_a && !w.joined) {
        const int blk = u % w.blocks;
        it.b = -1;
        it.g = u / w.blocks;
        it.row0 = blk * 2 * BM;
        it.rows = p.B * p.Sq * p.qpg;
        it.own_end = 0;
        it.alt = w.is_alt(blk);
        it.slot = tile > 0 ? w.list.frag[c] : 0;   // (a unit that begins here has its first fragment here)
        it.t0 = tile;
        it.np = it.n = it.n0 = (ends ? w.list.tile[c + 1] : pre) - tile;
        it.o0 = 0;
        const int at = walked % pre - tile;
        it.turn = at > 0 && at < it.n ? at : 0;
        walked += it.n;
        if (!ends && lane == 0) w.note[u] = it.slot + 1;
      } else {
        // The rows of one entry: a unit's part of its list, or an item's.
        int blk, np = 0, part = 0;
        int rest = u;
        if (k >= items_a) {   // items in turn, to and fro: the ones in front are longer
          const int round = k - items_a, grid = (int)gridDim.x;
          rest = w.first_b + round * grid + (round % 2 && (round + 1) * grid <= w.n_b ? grid - 1 - (int)blockIdx.x
                                                                                       : (int)blockIdx.x);
          part = rest % w.parts_b;
          rest /= w.parts_b;
        }
        it.g = rest % p.G;
        rest /= p.G;
        it.b = rest % p.B;
        blk = w.blocks_b - 1 - rest / p.B;
        it.alt = w.alt_b && blk == w.blocks_b - 1;
        if (w.joined) {
          it.slot = k >= items_a ? -1 : tile > 0 ? 0 : ends ? 1 : -1;
          np = pre;
        } else {
          it.slot = w.own_slot + part;
        }
        it.row0 = blk * 2 * BM;
        it.rows = p.Sq * p.qpg;
        it.own_end = own_seen(p, it.b, (min(it.row0 + 2 * BM, it.rows) - 1) / p.qpg);
        const int end0 = own_seen(p, it.b, (min(it.row0 + BM, it.rows) - 1) / p.qpg);
        int i0, i1;
        const int all = np + (it.own_end + BN - 1) / BN;
        if (k < items_a) {   // (the shares on both sides of a cut find the same place for it)
          const float part = (float)all / (float)most_tiles(p, blk, pre);
          i0 = min((int)(tile * part), all);
          i1 = ends ? min((int)(w.list.tile[c + 1] * part), all) : all;
        } else {
          list_part(all, part, w.parts_b, i0, i1);
        }
        it.t0 = min(i0, np);
        it.np = min(i1, np) - it.t0;
        it.o0 = max(i0 - np, 0);
        it.n = i1 - i0;
        it.n0 = min(max(np + (end0 + BN - 1) / BN - i0, 0), it.n);
      }
      ++u;
      tile = 0;
      it.some1 = it.row0 + BM < it.rows;
      if (lane == 0) items[buf] = it;
      __syncwarp();
      mbar_arrive(&sb.item_full[buf]);
      if (k == 0) continue;   // (the softmax threads load the first queries)
      // Where this lane's rows lane, lane + 32, ... of the block are (-1: there is no such row).
      int64_t at[2 * BM / 32];
#pragma unroll
      for (int j = 0; j < 2 * BM / 32; ++j) {
        const int row = it.row0 + 32 * j + lane;
        at[j] = -1;
        if (row < it.rows) {
          int q = row / p.qpg, b = it.b;
          const int h = it.g * p.qpg + row - q * p.qpg;
          if (b < 0) {
            b = q / p.Sq;
            q -= b * p.Sq;
          }
          at[j] = (int64_t)b * p.q.bs + (int64_t)h * p.q.hs + (int64_t)q * p.q.rs;
        }
      }
      if (!wait_warp(&sb.q_empty, (uint32_t)(k - 1) & 1u, &sb.abort, p.status)) break;
      const T* Q = static_cast<const T*>(p.Q) + p.q.off + lane % kUnits * 8;
      const int rl = lane / kUnits, un = lane % kUnits;
#pragma unroll
      for (int j = 0; j < 2 * BM / 32; ++j) {
        // (Behind the last row no warp takes a step; row tiles that hold the same rows share the first tile.)
        if (it.row0 + 32 * j >= it.rows) break;
#pragma unroll 4
        for (int r0 = 0; r0 < 32; r0 += kRowsAt) {
          const int64_t from = __shfl_sync(0xffffffffu, at[j], r0 + rl);
          const int row = 32 * j + r0 + rl;   // (128-byte swizzle)
          paged::copy16(su32(q_s + row / BM * C::kTile + (un / 8) * BM * 128 + row % BM * 128 + (((un % 8) ^ (row & 7)) << 4)),
                        Q + (from < 0 ? 0 : from), from < 0 ? 0 : 16);
        }
      }
      paged::copy_commit();
      paged::copy_wait<0>();
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_arrive(&sb.q_full);
    }
  } else if (warp == 8 || warp == 11) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
    // ---------------- copies of K (warp 8) and V: every lane a piece of a tile ----------------
    const bool is_k = warp == 8;
    const CUtensorMap* map = is_k ? &tm_k : &tm_v;
    const int pieces = BN / w.piece;   // 1 .. 16
    const int piece = lane % pieces, chunk = lane / pieces;
    const bool copies = chunk < C::kChunks;
    const int at = chunk * BN * 128 + piece * w.piece * 128;
    // This lane's piece of tile i of an item: its page (n_pages behind the last key, -1: there is none) and row in it.
    auto look_up = [&](const Item& it, int i, int& row) {
      bool pre;
      const int r = it.key(i, pre) + piece * w.piece;
      row = 0;
      if (r >= (pre ? p.prefix : it.own_end)) return (int)x.n_pages;
      const int pi = page_index(x, r);
      row = r - pi * x.page_size;
      const int32_t pg = __ldg((pre ? x.prefix_table : x.table + (int64_t)it.b * x.table_stride) + pi);
      return (uint32_t)pg < x.n_pages ? (int)pg : -1;
    };
    Slot sl{is_k ? 0 : 1, 0u};
    int gt = 0;   // tiles copied
    bool ok = true;
    for (int k = 0; ok && k < my_items; ++k) {
      const int buf = k & 1;
      if (!(ok = wait_warp(&sb.item_full[buf], (uint32_t)(k >> 1) & 1u, &sb.abort, p.status))) break;
      const Item& it = items[buf];
      const int n = it.n, g = it.g;
      int row = 0, page = 0;
      if (n > 0) page = look_up(it, 0, row);
      for (int i = 0; i < n; ++i) {
        const uint32_t missing = __ballot_sync(0xffffffffu, page < 0 && chunk == 0);
        const int pg = page < 0 ? (int)x.n_pages : page, prow = row;
        bool pre;
        const uint32_t first_key = (uint32_t)it.key(i, pre) + (pre ? 1u : 0u);
        if (i + 1 < n) page = look_up(it, i + 1, row);   // arrives while this tile waits for its slot
        if (!(ok = wait_warp(&sb.empty[sl.s], sl.ph ^ 1u, &sb.abort, p.status))) break;
        if (lane == 0) {
          // Note gt % kNotes was read for tile gt - kNotes.  The slot was free: the product that used it is done, of tile
          // gt - n_slots / 2 - 1 or a later one, whose S followed the row tiles' reading of notes two tiles further back.
          if (is_k) notes[gt % kNotes] = make_uint2(missing, first_key);
          mbar_expect_tx(&sb.full[sl.s], C::kTile);
        }
        __syncwarp();
        // Test hook (attn_test_inject): the first CTA's first K copy is
        // announced but never issued, so the MMA warp's wait runs out.
        const bool dropped = drop_first_copy && is_k && gt == 0 && blockIdx.x == 0;
        if (copies && !dropped) tma_load_4d(ring + sl.s * C::kTile + at, map, &sb.full[sl.s], chunk * 64, prow, g, pg);
        sl.next_tile(n_slots);
        ++gt;
      }
      if (ok && lane == 0) mbar_arrive(&sb.item_empty[buf]);
    }
    // Copies still in flight land before the CTA can exit: the last ones, whose slots were not refilled (the others
    // completed before theirs were).
    if (lane == 0) {
      Slot last{is_k ? 0 : 1, 0u};
      for (int i = 0; i < gt; ++i) {
        if (i >= gt - n_slots / 2) drain_bar(&sb.full[last.s], last.ph, p.status);
        last.next_tile(n_slots);
      }
    }
    __syncwarp();
  } else if (warp == 9) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
    // ---------------- MMA issuer (warp-wide; one elected lane issues) ----------------
    constexpr uint32_t kIdQK = idesc_f16(BF16, false, BM, BN);
    constexpr uint32_t kIdPV = idesc_f16(BF16, true, BM, D);
    const uint32_t q_addr = su32(q_s), ring_addr = su32(ring);
    const uint64_t qd0 = sdesc(q_addr, 16, 1024), kd0 = sdesc(ring_addr, 16, 1024);
    const uint64_t vd0 = sdesc(ring_addr, BN * 128, 1024);
    // S of row tile tt from the queries of tile `qt`.
    auto issue_qk = [&](int tt, int qt, int s) {
      fence_after();
      const uint64_t ad = sdesc_add(qd0, (uint32_t)(qt * C::kTile));
      const uint64_t bd0 = sdesc_add(kd0, (uint32_t)(s * C::kTile));
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint64_t a = sdesc_add(ad, (uint32_t)((kk / 4) * BM * 128 + (kk % 4) * 32));
        const uint64_t bd = sdesc_add(bd0, (uint32_t)((kk / 4) * BN * 128 + (kk % 4) * 32));
        mma_ss_w(tmem + (tt ? C::kS1 : C::kS0), a, bd, kIdQK, kk > 0);
      }
      mma_commit_w(&sb.s_full[tt]);
    };
    auto issue_pv = [&](int tt, int s, bool start) {
      fence_after();
      const uint64_t bd0 = sdesc_add(vd0, (uint32_t)(s * C::kTile));
#pragma unroll
      for (int kk = 0; kk < BN / 16; ++kk) {
        const uint64_t bd = sdesc_add(bd0, (uint32_t)(kk * 16 * 128));
        mma_ts_w(tmem + (tt ? C::kO1 : C::kO0), tmem + (tt ? C::kS1 : C::kS0) + kk * 8, bd, kIdPV,
                 (!start || kk > 0) ? 1u : 0u);
      }
      mma_commit_w(&sb.o_done[tt]);
    };
    // Zeroes the V rows of a tile's keys that no row of the item sees (they may hold anything).
    auto clear_tail = [&](const Item& it, int i, int s) {
      bool pre;
      const int k0 = it.key(i, pre), seen = (pre ? p.prefix : it.own_end) - k0;
      if (seen >= BN) return;
      for (int u = seen * (C::kChunks * 8) + lane; u < BN * (C::kChunks * 8); u += 32) {
        const int row = u / (C::kChunks * 8), rest = u % (C::kChunks * 8);
        *reinterpret_cast<uint4*>(ring + s * C::kTile + (rest / 8) * BN * 128 + row * 128 + (rest % 8) * 16) =
            make_uint4(0, 0, 0, 0);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
    };
    int c0 = 0, c1 = 0;                // P V steps of each row tile so far
    Slot ks{0, 0u}, vs{1, 0u};         // the next key tile to take S of, and the next to take P V of
    bool ok = true, issued = false;
    auto k_ready = [&]() { return wait_warp(&sb.full[ks.s], ks.ph, &sb.abort, p.status); };
    for (int k = 0; ok && k < my_items; ++k) {
      const int buf = k & 1;
      if (!(ok = wait_warp(&sb.item_full[buf], (uint32_t)(k >> 1) & 1u, &sb.abort, p.status))) break;
      const Item& it = items[buf];
      const int n = it.n;
      if (!(ok = wait_warp(k ? &sb.q_full : &sb.q_first, (uint32_t)(k ? k - 1 : 0) & 1u, &sb.abort, p.status))) break;
      bool start0 = true, start1 = true;
      if (n == 0) {
        if (lane == 0) mbar_arrive(&sb.q_empty);
      } else if (it.alt) {
        issued = true;
        // Tile i belongs to row tile i % 2: P V of tile i, then S of tile i + 2.
        auto next_s = [&](int i) {
          if (!k_ready()) return false;
          issue_qk(i & 1, 0, ks.s);
          mma_commit_w(&sb.empty[ks.s]);
          if (i + 1 == n) mma_commit_w(&sb.q_empty);   // that was the item's last S
          ks.next_tile(n_slots);
          return true;
        };
        for (int i = 0; ok && i < 2 && i < n; ++i) ok = next_s(i);
        for (int i = 0; ok && i < n; ++i) {
          const int t = i & 1;
          if (!(ok = wait_warp(&sb.full[vs.s], vs.ph, &sb.abort, p.status))) break;
          clear_tail(it, i, vs.s);
          if (!(ok = wait_warp(&sb.p_full[t], (uint32_t)(t ? c1 : c0) & 1u, &sb.abort, p.status))) break;
          issue_pv(t, vs.s, t ? start1 : start0);
          mma_commit_w(&sb.empty[vs.s]);
          vs.next_tile(n_slots);
          if (t) {
            start1 = false;
            ++c1;
          } else {
            start0 = false;
            ++c0;
          }
          if (i + 2 < n) ok = next_s(i + 2);
        }
      } else {
        issued = true;
        const int n0 = it.n0;
        const bool some1 = it.some1 != 0;
        if (!(ok = k_ready())) break;
        if (n0 > 0) issue_qk(0, 0, ks.s);
        if (some1) issue_qk(1, 1, ks.s);
        mma_commit_w(&sb.empty[ks.s]);
        if (n == 1) mma_commit_w(&sb.q_empty);
        ks.next_tile(n_slots);
        bool rv = mbar_test(&sb.full[vs.s], vs.ph);   // the next V landed?
        for (int i = 0; i < n; ++i) {
          const bool more = i + 1 < n, has0 = i < n0;
          const bool rp0 = !has0 || mbar_test(&sb.p_full[0], (uint32_t)c0 & 1u);
          if (!(ok = wait_ready(rv, &sb.full[vs.s], vs.ph, &sb.abort, p.status))) break;
          clear_tail(it, i, vs.s);
          const bool rk = !more || mbar_test(&sb.full[ks.s], ks.ph);
          // Row tile 0: P0 V, then the next S0.  (P of an item's first tile
          // follows the threads' reading of the previous item's O, so O may be
          // overwritten.)
          if (has0) {
            if (!(ok = wait_ready(rp0, &sb.p_full[0], (uint32_t)c0 & 1u, &sb.abort, p.status))) break;
            issue_pv(0, vs.s, start0);
            start0 = false;
            ++c0;
          }
          const bool rp1 = !some1 || mbar_test(&sb.p_full[1], (uint32_t)c1 & 1u);
          if (more) {
            if (!(ok = wait_ready(rk, &sb.full[ks.s], ks.ph, &sb.abort, p.status))) break;
            if (i + 1 < n0) issue_qk(0, 0, ks.s);
          }
          const int v_done = vs.s;
          vs.next_tile(n_slots);
          rv = more && mbar_test(&sb.full[vs.s], vs.ph);
          // Row tile 1: P1 V, then the next S1.
          if (some1) {
            if (!(ok = wait_ready(rp1, &sb.p_full[1], (uint32_t)c1 & 1u, &sb.abort, p.status))) break;
            issue_pv(1, v_done, start1);
            start1 = false;
            ++c1;
          }
          mma_commit_w(&sb.empty[v_done]);
          if (more) {
            if (some1) issue_qk(1, 1, ks.s);
            mma_commit_w(&sb.empty[ks.s]);
            if (i + 2 == n) mma_commit_w(&sb.q_empty);
            ks.next_tile(n_slots);
          }
        }
      }
      if (ok && lane == 0) mbar_arrive(&sb.item_empty[buf]);
      __syncwarp();
    }
    // Every MMA issued above has completed before TMEM is freed.
    if (issued) {
      mma_commit_w(&sb.mma_done);
      if (lane == 0) drain_bar(&sb.mma_done, 0, p.status);
    }
    __syncwarp();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ---------------- softmax: one thread per query row ----------------
    const int t = warp / 4, r = (warp % 4) * 32 + lane;   // row tile, row in it = TMEM lane
    const uint32_t lane_off = (uint32_t)((warp % 4) * 32) << 16;
    const uint32_t s_tm = tmem + lane_off + (t ? C::kS1 : C::kS0);
    const uint32_t o_tm = tmem + lane_off + (t ? C::kO1 : C::kO0);
    const float sc = p.scale * kLog2e;
    const bool capped = XF && p.softcap > 0.f;
    const float kinv = capped ? p.scale / p.softcap : 0.f;
    const float c_eff = XF ? 1.f : sc;   // of a value in x, to the units of m_ref
    uint32_t xs[BN];
    // This thread's row of an item: entry, query and head (false: there is none).
    auto row_of = [&](const Item& it, int& b, int& i, int& h) {
      const int row = it.row0 + (it.alt ? r : t * BM + r);
      if (row >= it.rows) {
        b = i = h = 0;
        return false;
      }
      const int q = row / p.qpg;
      h = it.g * p.qpg + row - q * p.qpg;
      b = it.b;
      i = q;
      if (it.b < 0) {
        b = q / p.Sq;
        i = q - b * p.Sq;
      }
      return true;
    };
    int j = 0;    // key tiles so far
    int gt = 0;   // key tiles of the items so far
    uint32_t pair_phase = 0u;
    bool ok = true;
    for (int k = 0; ok && k < my_items; ++k) {
      const int buf = k & 1;
      if (!(ok = wait_warp(&sb.item_full[buf], (uint32_t)(k >> 1) & 1u, &sb.abort, p.status))) break;
      const Item& it = items[buf];
      const int n = it.n;
      int b, qi, h;
      const bool valid = row_of(it, b, qi, h);
      if (k == 0) {
        if (t == 0 || it.some1) {   // (row tiles that hold the same rows share the first tile)
          const uint4* src = reinterpret_cast<const uint4*>(static_cast<const T*>(p.Q) + p.q.off + (int64_t)b * p.q.bs +
                                                            (int64_t)h * p.q.hs + (int64_t)qi * p.q.rs);
          uint4* dst = reinterpret_cast<uint4*>(q_s + t * C::kTile + r * 128);
          uint4 v[D / 8];
#pragma unroll
          for (int u = 0; u < D / 8; ++u) v[u] = valid ? __ldg(src + u) : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int u = 0; u < D / 8; ++u) dst[(u / 8) * BM * 8 + ((u % 8) ^ (r & 7))] = v[u];
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        mbar_arrive(&sb.q_first);
      }
      const bool idle = !__any_sync(0xffffffffu, valid);   // no row of this warp exists: its P is not used
      // Own keys that the row sees (the prefix's are all seen); a row that does not exist hides nothing.
      const int seen_own = !valid ? 0x7fffffff : it.b < 0 ? 0 : own_seen(p, b, qi);
      const float* mrow = nullptr;
      if (XF && p.M && valid)
        mrow = p.M + p.m.off + (int64_t)b * p.m.bs + (int64_t)h * p.m.hs + (int64_t)qi * p.m.rs;
      float m_ref = -INFINITY, l = 0.f;
      int done = 0;
      for (int i = 0; i < n; ++i) {
        if (!it.has(t, i)) continue;
        if (!(ok = wait_warp(&sb.s_full[t], (uint32_t)j & 1u, &sb.abort, p.status))) break;
        fence_after();
        const uint2 note = notes[(gt + i) % kNotes];
        const uint32_t missing = note.x;
        const bool pre = note.y & 1u;
        const int k0 = (int)(note.y & ~1u);
        const int seen_n = (pre && valid ? p.prefix : seen_own) - k0;   // the row sees the tile's first seen_n keys
        // Which of columns 32 c .. of the tile the row sees.
        auto seen_bits = [&](int c) {
          uint32_t bits = low_bits(seen_n - 32 * c);
          if (missing)
            for (int q = 0; q < 32; q += min(w.piece, 32))
              if ((missing >> ((32 * c + q) / w.piece)) & 1u) bits &= ~(low_bits(w.piece) << q);
          return bits;
        };
        bool rescale = false;
        float corr = 1.f;
        // With a finite reference maximum P is computed against it without
        // scanning for the tile's maximum; a row whose tile sum reaches kLagMax
        // makes the warp redo the tile with the scan.
        constexpr float kLagMax = BF16 ? 0x1p64f : 65504.f;   // (no p of f16 overflows below)
        if (!idle) {
          bool scan = __any_sync(0xffffffffu, !(m_ref > -INFINITY));
#pragma unroll 1
          for (int pass = 0; pass < 2; ++pass) {
            if constexpr (XF) {
              const float* mk = mrow ? mrow + (pre ? 0 : p.prefix) + k0 : nullptr;
#pragma unroll
              for (int c = 0; c < BN / 32; ++c) {
                const uint32_t seen = seen_bits(c);
                tmem_ld32(s_tm + c * 32, xs + c * 32);
                tmem_ld_wait_regs<1>(xs + c * 32);
#pragma unroll
                for (int e = c * 32; e < c * 32 + 32; ++e) {
                  float v = -INFINITY;
                  if ((seen >> (e % 32)) & 1u) {
                    const float s = __uint_as_float(xs[e]);
                    v = capped ? p.softcap * tanh_exp2(s * kinv) : s * p.scale;
                    if (mk) v += mk[e];
                  }
                  xs[e] = __float_as_uint(v);
                  if ((e & 7) == 7) asm volatile("" ::: "memory");  // at most 8 mask loads in flight
                }
              }
            } else {
#pragma unroll
              for (int c = 0; c < BN / 32; ++c) tmem_ld32(s_tm + c * 32, xs + c * 32);
              tmem_ld_wait_regs<BN / 32>(xs);
              if (seen_n < BN || missing) {   // hide by bits, one select a column
#pragma unroll
                for (int c = 0; c < BN / 32; ++c) {
                  const uint32_t seen = seen_bits(c);
#pragma unroll
                  for (int e = 0; e < 32; ++e)
                    if (!(seen & (1u << e))) xs[c * 32 + e] = __float_as_uint(-INFINITY);
                }
              }
            }
            if (scan) {
              float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
              for (int e = 0; e < BN; e += 4) {
                mx0 = max3(mx0, __uint_as_float(xs[e]), __uint_as_float(xs[e + 1]));
                mx1 = max3(mx1, __uint_as_float(xs[e + 2]), __uint_as_float(xs[e + 3]));
              }
              float mt = fmaxf(mx0, mx1) * c_eff;
              const bool raise = mt - m_ref > kRise;      // also true for the first tile with a visible key
              mt -= kLead;
              if (raise) corr = S::weight(m_ref, mt);     // 0 when m_ref = -inf
              rescale = raise && m_ref > -INFINITY;       // O holds earlier tiles' sums
              if (raise) {
                l *= corr;
                m_ref = mt;
              }
            }
            const float neg = -(m_ref == -INFINITY ? 0.f : m_ref);
            const uint64_t c2 = f2u(c_eff, c_eff), n2 = f2u(neg, neg);
            float la0 = 0.f, la1 = 0.f, lb0 = 0.f, lb1 = 0.f;
#pragma unroll
            for (int e = 0; e < BN; e += 4) {
              float a0, a1, b0, b1;
              fma2(a0, a1, __uint_as_float(xs[e]), __uint_as_float(xs[e + 1]), c2, n2);
              fma2(b0, b1, __uint_as_float(xs[e + 2]), __uint_as_float(xs[e + 3]), c2, n2);
              if constexpr (XF) {   // natural differences
                fma2(a0, a1, a0, a1, f2u(kLog2e, kLog2e), 0);
                fma2(b0, b1, b0, b1, f2u(kLog2e, kLog2e), 0);
              }
              a0 = ex2(a0);
              a1 = ex2(a1);
              b0 = ex2(b0);
              b1 = ex2(b1);
              add2(la0, la1, a0, a1);
              add2(lb0, lb1, b0, b1);
              xs[e / 2] = pack2<BF16>(a0, a1);
              xs[e / 2 + 1] = pack2<BF16>(b0, b1);
            }
            const float lt = (la0 + la1) + (lb0 + lb1);
            if (scan || !__any_sync(0xffffffffu, lt >= kLagMax)) {   // NaN sums stay (a NaN row)
              l += lt;
              break;
            }
            scan = true;
          }
#pragma unroll
          for (int c = 0; c < 2; ++c) tmem_st32(s_tm + c * 32, xs + c * 32);
        }
        if (__any_sync(0xffffffffu, rescale)) {
          // P V of the previous tile must have landed in O before it is scaled.
          if (!(ok = wait_warp(&sb.o_done[t], (uint32_t)(j - 1) & 1u, &sb.abort, p.status))) break;
          fence_after();
          const float f = rescale ? corr : 1.f;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(o_tm + c * 32, o);
            tmem_ld_wait_regs<1>(o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st32(o_tm + c * 32, o);
          }
        }
        tmem_st_wait();
        fence_before();
        mbar_arrive(&sb.p_full[t]);
        ++j;
        ++done;
      }
      if (!ok) break;
      gt += n;
      // ---- epilogue: O / l, special rows, LSE ----
      if (done > 0 && !(ok = wait_warp(&sb.o_done[t], (uint32_t)(j - 1) & 1u, &sb.abort, p.status))) break;
      fence_after();
      // One row tile: each half of the keys has a result of every row, and each half of the threads takes half of the
      // columns of both.  f: what this thread's own and the other result are weighed with.
      const bool pair = it.alt && n > 1;
      float f_own = 1.f, f_other = 0.f;
      if (pair) {
        pair_ml[t][r] = make_float2(m_ref, l);
        fence_before();
        mbar_arrive(&sb.pair_have);
        if (!(ok = wait_warp(&sb.pair_have, pair_phase, &sb.abort, p.status))) break;
        fence_after();
        const float2 other = pair_ml[t ^ 1][r];
        const float top = fmaxf(m_ref, other.x), mu = top == -INFINITY ? 0.f : top;
        f_own = S::weight(m_ref, mu);
        f_other = S::weight(other.x, mu);
        l = t ? fmaf(f_other, other.y, f_own * l) : fmaf(f_own, l, f_other * other.y);   // (the same bits in both)
        m_ref = top;
      }
      const bool split = it.slot >= 0;
      const int c_begin = pair ? t * (D / 64) : 0, c_end = pair ? (t + 1) * (D / 64) : it.alt && t ? 0 : D / 32;
      // The sink logit joins the denominator (and rescales the accumulated O); with parts the merge adds it once.
      float M = S::natural(m_ref);
      const float o_mul = p.sink_on && !split && valid ? fold_sink<false>(M, l, sink_logit(p, h)) : 1.f;
      const bool hidden_row = (l == 0.f);         // no visible key; a NaN l stays a NaN row
      const float inv = o_mul / l, inv_own = inv * f_own, inv_other = inv * f_other;
      const float fill = p.masked_zero ? 0.f : NAN;
      T* orow = static_cast<T*>(p.O) + p.o.off + (int64_t)b * p.o.bs + (int64_t)h * p.o.hs + (int64_t)qi * p.o.rs;
      const int64_t prow = w.joined ? ((int64_t)blockIdx.x * 2 + it.slot) * (2 * BM) + (it.alt ? r : t * BM + r)
                                    : (((int64_t)b * p.H + h) * p.Sq + qi) * w.splits + it.slot;
      float* po = w.part_o + prow * D;   // (not used when O is written)
      const uint32_t other_tm = tmem + lane_off + (t ? C::kO0 : C::kO1);
#pragma unroll 1
      for (int c = c_begin; c < c_end; ++c) {
        uint32_t o[32];
        if (done > 0) {
          tmem_ld32(o_tm + c * 32, o);
          tmem_ld_wait_regs<1>(o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * inv_own);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
        if (pair) {
          uint32_t o2[32];
          tmem_ld32(other_tm + c * 32, o2);
          tmem_ld_wait_regs<1>(o2);
#pragma unroll
          for (int e = 0; e < 32; ++e)
            o[e] = __float_as_uint(fmaf(__uint_as_float(o2[e]), inv_other, __uint_as_float(o[e])));
        }
        if (split) {
          if (valid && !hidden_row) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) store32(po + c * 32 + e, o + e);
          }
        } else {
          uint32_t y[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            y[e / 2] = pack2<BF16>(hidden_row ? fill : __uint_as_float(o[e]), hidden_row ? fill : __uint_as_float(o[e + 1]));
          if (valid) {
            if (wide_rows) {
              store32(orow + c * 32, y);
              store32(orow + c * 32 + 16, y + 8);
            } else {
              uint4* dst = reinterpret_cast<uint4*>(orow + c * 32);
#pragma unroll
              for (int v4 = 0; v4 < 4; ++v4)
                dst[v4] = make_uint4(y[4 * v4], y[4 * v4 + 1], y[4 * v4 + 2], y[4 * v4 + 3]);
            }
          }
        }
      }
      if (valid && !(it.alt && t)) {
        if (split) {
          w.part_m[prow] = hidden_row ? -INFINITY : M;
          w.part_l[prow] = l;
        } else if (p.lse) {
          p.lse[(int64_t)b * p.lse_bs + (int64_t)h * p.lse_hs + qi] = hidden_row ? -INFINITY : S::lse(M, __log2f(l));
        }
      }
      if (pair) {   // both are done with both results, before either goes on to the next item's
        fence_before();
        mbar_arrive(&sb.pair_done);
        if (!(ok = wait_warp(&sb.pair_done, pair_phase, &sb.abort, p.status))) break;
        pair_phase ^= 1u;
      }
      fence_before();   // O's loads come before the next item's P, and so before its P V
      mbar_arrive(&sb.item_empty[buf]);
    }
  }

  fence_before();
  __syncthreads();
  if (warp == 9) {
    fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// ---- host side -----------------------------------------------------------------------

template <int D, bool BF16, bool XF>
int launch(const Problem& p, const Ext& x, const Work& w, cudaStream_t st) {
  CUtensorMap mk, mv;
  if (!tma_map_bhsd(&mk, p.K, p.dtype, D, x.page_size, p.G, (int)x.n_pages, p.k, w.piece) ||
      !tma_map_bhsd(&mv, p.V, p.dtype, D, x.page_size, p.G, (int)x.n_pages, p.v, w.piece))
    return -1;  // not describable: caller falls back
  const int smem = Cfg<D>::kSmem;
  auto kern = shared_tc_kernel<D, BF16, XF>;
  // setmaxnreg.inc waits until the block's register pool holds the larger
  // count, so the pool the kernel is launched with must cover the split.  The
  // tiles fill what the kernel's own variables leave of the shared memory, and
  // lie on the swizzle's 1024-byte boundaries: the compiler pads the variables
  // to the alignment of the array behind them.
  static const bool fits = [] {
    cudaFuncAttributes a;
    if (cudaFuncGetAttributes(&a, (const void*)shared_tc_kernel<D, BF16, XF>) != cudaSuccess) return false;
    return a.numRegs * kThreads >= kSplitRegs && a.sharedSizeBytes % 1024 == 0 &&
           a.sharedSizeBytes + Cfg<D>::kSmem <= 227 * 1024;
  }();
  if (!fits) return -1;
  if (ensure_smem((const void*)kern, smem) != cudaSuccess) return ATTN_ERR_CUDA;
  // Rows of O on 32-byte boundaries take 32-byte stores.
  auto even = [](int64_t stride, int64_t extent) { return extent <= 1 || stride % 16 == 0; };
  const int wide = ((uintptr_t)p.O + (uintptr_t)p.o.off * 2) % 32 == 0 && even(p.o.bs, p.B) && even(p.o.hs, p.H) &&
                           even(p.o.rs, p.Sq)
                       ? 1
                       : 0;
  const int drop = take_injection() == ATTN_INJECT_DROP_FIRST_COPY ? 1 : 0;
  const int ctas = w.list.ctas > w.n_b ? w.list.ctas : w.n_b;
  kern<<<(unsigned)(ctas < kSms ? ctas : kSms), kThreads, smem, st>>>(mk, mv, p, x, w, wide, drop);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

template <int D>
int launch_d(const Problem& p, const Ext& x, const Work& w, cudaStream_t st) {
  const bool xf = p.M != nullptr || p.softcap > 0.f || !(p.scale * kLog2e > 0.f);
  if (p.dtype == ATTN_BF16)
    return xf ? launch<D, true, true>(p, x, w, st) : launch<D, true, false>(p, x, w, st);
  return xf ? launch<D, false, true>(p, x, w, st) : launch<D, false, false>(p, x, w, st);
}

}  // namespace shr
}  // namespace attn
