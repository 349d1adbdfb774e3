// window_tc.cuh -- f16/bf16 attention under a sliding window with first keys,
// head_dim 64 or 128, on the tensor cores.
//
// What it computes: O = softmax(scale Q K^T + mask) V and the LSE over each
// row's visible keys (visible.cuh).  The tile step is the prefill kernel's
// (prefill_tc.cu): two 128-row query tiles ping-pong, S = Q K^T and O += P V
// are tcgen05 MMAs with TMEM accumulators, a thread holds a row of S, P goes
// back over S as packed pairs, the reference maximum moves with a slack of 8
// log2 units.
//
// What is its own: under a window a query block has few key tiles, so what a
// CTA pays once weighs most -- launch, barriers, tensor memory, the first Q and
// K, the last O (about four tiles' time of the prefill kernel's per block; with
// 1023 keys of window a block has eleven tiles).  The kernel is persistent, one CTA an
// SM, and its CTAs take (query block, part) items in turn:
//   warp 10    finds the next items' rows, tiles and first keys two items
//              ahead (a window, per-entry lengths, segment starts), into
//              shared memory;
//   warp 8     copies (TMA): the next item's first K and V tiles and, once its
//              last S is issued, its Q, while the current item finishes;
//   warp 9     issues the MMAs: the next item's first S follows the current
//              one's last P V at once;
//   warps 0-7  softmax and epilogue; one query tile's epilogue overlaps the
//              other tile's last step and the next item's first.
// P enters the product as one value of the element type, as in attn_fwd (the
// reading there: "the probabilities are rounded to the element type"), while
// the row sums take it in float32: the error against 64 bits is 1.4 times the
// output's own rounding (prompt of 8192 in bf16: 0.0022 against 0.0016).  P in
// two halves takes that away, but a second P V and the halving cost a third of
// the kernel's speed (128.6 -> 174 us, and spills).
//
// Key tiles in the gap between the first keys and the window are not in an
// item's list; query tile 0 stops at its own last tile and query tile 1 leaves
// out the window's first tile where only tile 0 sees it.
//
// Few query blocks: a cluster of 2, 4 or 8 CTAs takes one block, each CTA a part
// of its list; the parts' O and row sums meet in distributed shared memory,
// where every CTA merges and writes its share of the rows.
//
// Waits are bounded as in the prefill kernel (the cluster barriers at the end
// are passed by every thread, also after a wait ran out).
#pragma once

#include <string.h>

#include <type_traits>

#include "prefill_tc.h"
#include "tc_ptx.cuh"
#include "tma.h"
#include "visible.cuh"

namespace attn {
namespace win {

using namespace tc;

constexpr int BM = 128;            // query rows per tile
constexpr int BN = 128;            // keys per tile
constexpr int kShort = 32;         // columns computed of a tile with few first keys
constexpr int kThreads = 384;
// Registers after the split, as in the prefill kernel: 8 warps x 216 and 4
// warps x 56 fit the 168 a thread that the block is launched with.
constexpr int kSoftmaxRegs = 216;
constexpr int kProducerRegs = 56;
constexpr int kSplitRegs = 8 * 32 * kSoftmaxRegs + 4 * 32 * kProducerRegs;
static_assert(kSplitRegs <= kThreads * ((65536 / kThreads) & ~7), "register split exceeds the block's registers");
constexpr int kSms = 152;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kSlack = 8.0f;     // log2 units

// A query block's part, as the roles read it.
struct Item {
  Vis uv;                // the rows' union
  int h, b, g, q0, part;
  int ta, na, tb, n;     // its tiles, as in TileList, from the part's first
  int n0;                // the tiles of query tile 0: the first n0
  int skip1;             // a tile that query tile 1 leaves out (-1: none)
  int some1;             // query tile 1 has a row
  __device__ __forceinline__ int key(int i) const { return (i < na ? ta + i : tb + (i - na)) * BN; }
  // A tile of at most kShort first keys and nothing else: only its first kShort columns are computed.
  __device__ __forceinline__ bool is_short(int i) const {
    return i < na && uv.fe - (ta + i) * BN <= kShort && uv.wl >= (ta + i + 1) * BN;
  }
};

struct Bars {
  uint64_t q_full, q_empty;
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t s_full[2], p_full[2], o_done[2];
  uint64_t item_full[2], item_empty[2];
  uint64_t mma_done;
  uint32_t tmem_base;
  int abort;
};

template <int D>
struct Cfg {
  static constexpr int kChunks = D / 64;                  // 64-column (128-byte) chunks
  static constexpr int kStages = D <= 64 ? 4 : 2;
  static constexpr int kQTile = BM * D * 2;               // bytes
  static constexpr int kKTile = BN * D * 2;
  static constexpr int kSmem = 2 * kQTile + 2 * kStages * kKTile;
  static constexpr int kS0 = 0, kS1 = BN, kO0 = 2 * BN, kO1 = 2 * BN + D;
  static_assert(2 * BN + 2 * D <= 512, "TMEM budget");
};

// The lowest n bits (n may lie outside [0, 32]).
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }
// Which of keys k .. k + 31 are visible, bit by bit.
__device__ __forceinline__ uint32_t seen_bits(const Vis& v, int k) {
  return (low_bits(v.hi - k) & ~low_bits(v.wl - k)) | (low_bits(v.fe - k) & ~low_bits(v.lo - k));
}

// 32 bytes to global memory in one store (32-byte aligned).
__device__ __forceinline__ void store32(void* dst, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// A float of CTA `rank`'s shared memory, at the address of this CTA's p.
__device__ __forceinline__ float peer(const float* p, uint32_t rank) {
  uint32_t r;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(su32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(r) : "memory");
  return v;
}

__device__ __forceinline__ float4 peer4(const float4* p, uint32_t rank) {
  uint32_t r;
  float4 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(su32(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(r)
               : "memory");
  return v;
}

// XF: scores under a mask, a softcap or a scale that is not positive.
template <int D, bool BF16, bool XF>
__global__ void __launch_bounds__(kThreads, 1)
    window_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const Problem p, const int first,
                     const int pair_heads, const int n_items, const int wide_rows, const int clustered, const int drop_first_copy,
                     const Split sp) {
  using C = Cfg<D>;
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* q_s = smem;
  uint8_t* k_s = q_s + 2 * C::kQTile;
  uint8_t* v_s = k_s + C::kStages * C::kKTile;
  __shared__ Bars sb;
  __shared__ Item items[2];
  __shared__ Vis row_v[2][2 * BM];
  // clustered: each row's reference maximum and sum; its numerators lie over the stages, [D / 4][2 BM][4].
  __shared__ float part_m[2 * BM], part_l[2 * BM];
  float4* const part_a = reinterpret_cast<float4*>(k_s);

  using S = Scores<XF>;   // (masks come with XF)
  constexpr float kRise = XF ? kSlack * kLn2 : kSlack;   // in the units of the scores
  // A row's reference is a maximum, less a lead where P is f16: p is 2^5 at that maximum, and what f16 cannot hold
  // (2^-25) is 2^-30 of the row's largest probability, for all keys together n 2^-30: under a quarter of f16's half
  // step up to 2^17 keys of window.  More lead takes room from the lag (kLagMax): a first tile of four keys puts the
  // reference some units under the next tile's sums, and with a lead of 7 most warps scanned twice there (4096
  // tokens, 32/8 heads, head_dim 64: 65 -> 74 us).
  constexpr float kLead = (BF16 ? 0.f : 5.f) * (XF ? kLn2 : 1.f);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int my_items = (n_items - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
  // The two query tiles are rows [q0, q0 + 256) of one head, or with
  // pair_heads (q_len <= 128) rows [0, q_len) of two query heads of a kv head.
  const int ht_step = pair_heads ? 1 : 0, rt_step = pair_heads ? 0 : BM;

  if (threadIdx.x == 0) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
    sb.abort = 0;
    mbar_init(&sb.q_full, 1);
    mbar_init(&sb.q_empty, 1);
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&sb.k_full[s], 1);
      mbar_init(&sb.k_empty[s], 1);
      mbar_init(&sb.v_full[s], 1);
      mbar_init(&sb.v_empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sb.s_full[i], 1);
      mbar_init(&sb.p_full[i], BM);
      mbar_init(&sb.o_done[i], 1);
      mbar_init(&sb.item_full[i], 32);
      mbar_init(&sb.item_empty[i], 2 + 2 * BM);   // the copy and MMA warps and every softmax thread
    }
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

  // clustered: the three barriers of the merge, for the warps that take no part in it.
  auto meet = [&]() {
    if (clustered)
      for (int i = 0; i < 3; ++i) cluster_sync();
  };
  if (warp == 10) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
    // ---------------- items: rows, unions, tile lists ----------------
    for (int k = 0; k < my_items; ++k) {
      const int buf = k & 1;
      if (k >= 2 && !wait_warp(&sb.item_empty[buf], (uint32_t)((k >> 1) - 1) & 1u, &sb.abort, p.status)) break;
      const int id = (int)blockIdx.x + k * (int)gridDim.x;
      const int blk = id / sp.n_splits, part = id % sp.n_splits;
      int h, b, g, q0;
      if (pair_heads) {
        const int npg = (p.qpg + 1) / 2, gb = blk / npg;
        g = gb % p.G;
        b = gb / p.G;
        h = g * p.qpg + 2 * (blk % npg);
        q0 = 0;
      } else {
        // Last query blocks first (the first ones see fewer keys); the heads of a block side by side share K and V in L2.
        const int hb = blk % (p.H * p.B), qb = n_items / sp.n_splits / (p.H * p.B) - 1 - blk / (p.H * p.B);
        h = hb % p.H;
        b = hb / p.H;
        g = h / p.qpg;
        q0 = qb * 2 * BM;
      }
      int w_lo = 0x7fffffff, w_hi = -1, f_lo = 0x7fffffff, f_hi = -1;   // both query tiles
      int hi_0 = -1, w_lo1 = 0x7fffffff, f_hi1 = -1;                    // query tile 0's end; tile 1's starts
      for (int r = lane; r < 2 * BM; r += 32) {
        const int tt = r / BM, row = pair_heads ? r % BM : q0 + r;
        // A row that does not exist hides nothing (its zero queries cost it no
        // pass of its own; it is not written) and has no part in the union.
        if (row >= p.Sq || h + tt * ht_step >= (g + 1) * p.qpg) {
          row_v[buf][r] = {0, 0, 0, 0x7fffffff};
          continue;
        }
        const Vis v = row_vis(p, first, b, row);
        row_v[buf][r] = v;
        if (v.hi > v.wl) {
          w_lo = min(w_lo, v.wl);
          w_hi = max(w_hi, v.hi);
          if (tt) w_lo1 = min(w_lo1, v.wl);
          else hi_0 = max(hi_0, v.hi);
        }
        if (v.fe > v.lo) {
          f_lo = min(f_lo, v.lo);
          f_hi = max(f_hi, v.fe);
          if (tt) f_hi1 = max(f_hi1, v.fe);
          else hi_0 = max(hi_0, v.fe);
        }
      }
      w_lo = __reduce_min_sync(0xffffffffu, w_lo);
      w_hi = __reduce_max_sync(0xffffffffu, w_hi);
      f_lo = __reduce_min_sync(0xffffffffu, f_lo);
      f_hi = __reduce_max_sync(0xffffffffu, f_hi);
      hi_0 = __reduce_max_sync(0xffffffffu, hi_0);
      w_lo1 = __reduce_min_sync(0xffffffffu, w_lo1);
      f_hi1 = __reduce_max_sync(0xffffffffu, f_hi1);
      if (lane == 0) {
        Item& it = items[buf];
        const Vis uv = vis_union(f_lo, f_hi, w_lo, w_hi);
        const TileList tl = tile_list(uv, BN);
        int i0 = 0, i1 = tl.n;
        if (sp.n_splits > 1) list_part(tl.n, part, sp.n_splits, i0, i1);
        it.uv = uv;
        it.h = h;
        it.b = b;
        it.g = g;
        it.q0 = q0;
        it.part = part;
        it.ta = tl.ta + i0;
        it.na = tl.na - i0;
        it.tb = tl.tb;
        it.n = i1 - i0;
        // Query tile 0's keys end at hi_0: its tiles are a prefix of the list.
        const int lim = hi_0 > 0 ? (hi_0 + BN - 1) / BN : 0;
        const int n0 = min(max(lim - tl.ta, 0), tl.na) + min(max(lim - tl.tb, 0), tl.n - tl.na);
        it.n0 = min(max(n0 - i0, 0), it.n);
        // The window's first tile, when it ends in front of query tile 1's windows and holds none of its first keys.
        const bool skip = tl.na < tl.n && (tl.tb + 1) * BN <= w_lo1 && tl.tb * BN >= f_hi1;
        it.some1 = pair_heads ? h + 1 < (g + 1) * p.qpg : q0 + BM < p.Sq;
        it.skip1 = skip && tl.na >= i0 && tl.na < i1 ? tl.na - i0 : -1;
      }
      __syncwarp();
      mbar_arrive(&sb.item_full[buf]);
    }
    meet();
  } else if (warp == 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
    // ---------------- copies ----------------
    if (lane == 0) {
      int gt = 0;        // tiles whose K and V copies were issued
      int k_only = -1;   // a tile whose K copy was issued but not its V copy
      int nq = 0;        // Q copies issued
      bool ok = true;
      for (int k = 0; ok && k < my_items; ++k) {
        const int buf = k & 1;
        if (!(ok = wait_bar(&sb.item_full[buf], (uint32_t)(k >> 1) & 1u, &sb.abort, p.status))) break;
        const int n = items[buf].n, h = items[buf].h, b = items[buf].b, g = items[buf].g, q0 = items[buf].q0;
        for (int i = 0; i < n; ++i) {
          const int s = gt % C::kStages;
          const uint32_t ph = (uint32_t)(gt / C::kStages) & 1u;
          const int krow = items[buf].key(i);
          if (!(ok = wait_bar(&sb.k_empty[s], ph ^ 1u, &sb.abort, p.status))) break;
          mbar_expect_tx(&sb.k_full[s], C::kKTile);
          // Test hook (attn_test_inject): the first CTA's first K copy is
          // announced but never issued, so the MMA warp's wait runs out.
          const bool dropped = drop_first_copy && gt == 0 && blockIdx.x == 0;
          for (int c = 0; c < C::kChunks && !dropped; ++c)
            tma_load_4d(k_s + s * C::kKTile + c * BN * 128, &tm_k, &sb.k_full[s], c * 64, krow, g, b);
          if (i == 0) {   // Q, once the previous item's last S is done with its own
            if (nq > 0 && !(ok = wait_bar(&sb.q_empty, (uint32_t)(nq - 1) & 1u, &sb.abort, p.status))) {
              k_only = gt;
              break;
            }
            mbar_expect_tx(&sb.q_full, 2 * C::kQTile);
            for (int tt = 0; tt < 2; ++tt)
              for (int c = 0; c < C::kChunks; ++c)
                tma_load_4d(q_s + tt * C::kQTile + c * BM * 128, &tm_q, &sb.q_full, c * 64, q0 + tt * rt_step,
                            h + tt * ht_step, b);
            ++nq;
          }
          if (!(ok = wait_bar(&sb.v_empty[s], ph ^ 1u, &sb.abort, p.status))) {
            k_only = gt;
            break;
          }
          mbar_expect_tx(&sb.v_full[s], C::kKTile);
          for (int c = 0; c < C::kChunks; ++c)
            tma_load_4d(v_s + s * C::kKTile + c * BN * 128, &tm_v, &sb.v_full[s], c * 64, krow, g, b);
          ++gt;
        }
        if (ok) mbar_arrive(&sb.item_empty[buf]);
      }
      // Copies still in flight land before the CTA can exit.  Earlier copies
      // completed before their stage (or Q) was refilled.
      if (nq > 0) drain_bar(&sb.q_full, (uint32_t)(nq - 1) & 1u, p.status);
      for (int i = gt > C::kStages ? gt - C::kStages : 0; i < gt; ++i) {
        const int s = i % C::kStages;
        const uint32_t ph = (uint32_t)(i / C::kStages) & 1u;
        drain_bar(&sb.k_full[s], ph, p.status);
        drain_bar(&sb.v_full[s], ph, p.status);
      }
      if (k_only >= 0) drain_bar(&sb.k_full[k_only % C::kStages], (uint32_t)(k_only / C::kStages) & 1u, p.status);
    }
    __syncwarp();
    meet();
  } else if (warp == 9) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
    // ---------------- MMA issuer (warp-wide; one elected lane issues) ----------------
    constexpr uint32_t kIdQK = idesc_f16(BF16, false, BM, BN), kIdShort = idesc_f16(BF16, false, BM, kShort);
    constexpr uint32_t kIdPV = idesc_f16(BF16, true, BM, D);
    const uint32_t q_addr = su32(q_s), k_addr = su32(k_s), v_addr = su32(v_s);
    const uint64_t qd0 = sdesc(q_addr, 16, 1024), qd1 = sdesc(q_addr + C::kQTile, 16, 1024);
    const uint64_t kd0 = sdesc(k_addr, 16, 1024), vd0 = sdesc(v_addr, BN * 128, 1024);
    auto issue_qk = [&](int tt, int s, bool small) {
      fence_after();
      const uint64_t ad = tt ? qd1 : qd0;
      const uint64_t bd0 = sdesc_add(kd0, (uint32_t)(s * C::kKTile));
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint64_t a = sdesc_add(ad, (uint32_t)((kk / 4) * BM * 128 + (kk % 4) * 32));
        const uint64_t bd = sdesc_add(bd0, (uint32_t)((kk / 4) * BN * 128 + (kk % 4) * 32));
        mma_ss_w(tmem + (tt ? C::kS1 : C::kS0), a, bd, small ? kIdShort : kIdQK, kk > 0);
      }
      mma_commit_w(&sb.s_full[tt]);
    };
    auto issue_pv = [&](int tt, int s, bool start, bool small) {
      fence_after();
      const uint64_t bd0 = sdesc_add(vd0, (uint32_t)(s * C::kKTile));
#pragma unroll
      for (int kk = 0; kk < BN / 16; ++kk) {
        if (kk == kShort / 16 && small) break;
        const uint64_t bd = sdesc_add(bd0, (uint32_t)(kk * 16 * 128));
        mma_ts_w(tmem + (tt ? C::kO1 : C::kO0), tmem + (tt ? C::kS1 : C::kS0) + kk * 8, bd, kIdPV,
                 (!start || kk > 0) ? 1u : 0u);
      }
      mma_commit_w(&sb.o_done[tt]);
    };
    int gt = 0, nq = 0, c0 = 0, c1 = 0;   // tiles, Q copies, and P V steps of each query tile so far
    bool ok = true, issued = false;
    for (int k = 0; ok && k < my_items; ++k) {
      const int buf = k & 1;
      if (!(ok = wait_warp(&sb.item_full[buf], (uint32_t)(k >> 1) & 1u, &sb.abort, p.status))) break;
      const int n = items[buf].n, n0 = items[buf].n0, skip1 = items[buf].skip1;
      const bool some1 = items[buf].some1 != 0;
      if (n > 0) {
        if (!(ok = wait_warp(&sb.q_full, (uint32_t)nq & 1u, &sb.abort, p.status))) break;
        ++nq;
        if (!(ok = wait_warp(&sb.k_full[gt % C::kStages], (uint32_t)(gt / C::kStages) & 1u, &sb.abort, p.status)))
          break;
        issued = true;
        bool small = !XF && items[buf].is_short(0);
        if (n0 > 0) issue_qk(0, gt % C::kStages, small);
        if (some1 && skip1 != 0) issue_qk(1, gt % C::kStages, small);
        mma_commit_w(&sb.k_empty[gt % C::kStages]);
        if (n == 1) mma_commit_w(&sb.q_empty);
        bool start0 = true, start1 = true;
        bool rv = mbar_test(&sb.v_full[gt % C::kStages], (uint32_t)(gt / C::kStages) & 1u);   // the next V landed?
        for (int i = 0; i < n; ++i, ++gt) {
          const int s = gt % C::kStages, s1 = (gt + 1) % C::kStages;
          const uint32_t ph = (uint32_t)(gt / C::kStages) & 1u, ph1 = (uint32_t)((gt + 1) / C::kStages) & 1u;
          const bool more = i + 1 < n, has0 = i < n0, has1 = some1 && i != skip1;
          const bool rp0 = !has0 || mbar_test(&sb.p_full[0], (uint32_t)c0 & 1u);
          if (!(ok = wait_ready(rv, &sb.v_full[s], ph, &sb.abort, p.status))) break;
          // Zero the V rows of keys no row of this item sees (they may hold
          // anything): in front of, between and behind the union's parts.
          const int k0 = items[buf].key(i), rows = small ? kShort : BN;
          const Vis uv = items[buf].uv;
          if (!within(uv, k0, k0 + rows)) {
            auto clear = [&](int a, int z) {   // rows [a, z) of the tile
              a = max(a - k0, 0);
              z = min(z - k0, rows);
              for (int u = a * (C::kChunks * 8) + lane; u < z * (C::kChunks * 8); u += 32) {
                const int row = u / (C::kChunks * 8), rest = u % (C::kChunks * 8);
                *reinterpret_cast<uint4*>(v_s + s * C::kKTile + (rest / 8) * BN * 128 + row * 128 + (rest % 8) * 16) =
                    make_uint4(0, 0, 0, 0);
              }
            };
            clear(k0, uv.fe > uv.lo ? uv.lo : uv.wl);
            if (uv.fe > uv.lo) clear(uv.fe, uv.wl);
            clear(uv.hi, k0 + BN);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
          }
          const bool rk = !more || mbar_test(&sb.k_full[s1], ph1);
          const bool next_small = !XF && more && items[buf].is_short(i + 1);
          // Query tile 0: P0 V, then the next S0.  (P of an item's first tile
          // follows the threads' reading of the previous item's O, so O may be
          // overwritten.)
          if (has0) {
            if (!(ok = wait_ready(rp0, &sb.p_full[0], (uint32_t)c0 & 1u, &sb.abort, p.status))) break;
            issue_pv(0, s, start0, small);
            start0 = false;
            ++c0;
          }
          const bool rp1 = !has1 || mbar_test(&sb.p_full[1], (uint32_t)c1 & 1u);
          if (more) {
            if (!(ok = wait_ready(rk, &sb.k_full[s1], ph1, &sb.abort, p.status))) break;
            if (i + 1 < n0) issue_qk(0, s1, next_small);
          }
          rv = more && mbar_test(&sb.v_full[s1], ph1);
          // Query tile 1: P1 V, then the next S1.
          if (has1) {
            if (!(ok = wait_ready(rp1, &sb.p_full[1], (uint32_t)c1 & 1u, &sb.abort, p.status))) break;
            issue_pv(1, s, start1, small);
            start1 = false;
            ++c1;
          }
          mma_commit_w(&sb.v_empty[s]);
          if (more) {
            if (some1 && i + 1 != skip1) issue_qk(1, s1, next_small);
            mma_commit_w(&sb.k_empty[s1]);
            if (i + 2 == n) mma_commit_w(&sb.q_empty);   // that was the item's last S
          }
          small = next_small;
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
    meet();
  } else if (warp == 11) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kProducerRegs));
    meet();
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ---------------- softmax: one thread per query row ----------------
    const int t = warp / 4, r = (warp % 4) * 32 + lane;   // query tile, row in it = TMEM lane
    const uint32_t lane_off = (uint32_t)((warp % 4) * 32) << 16;
    const uint32_t s_tm = tmem + lane_off + (t ? C::kS1 : C::kS0);
    const uint32_t o_tm = tmem + lane_off + (t ? C::kO1 : C::kO0);
    const float sc = p.scale * kLog2e;
    const bool capped = XF && p.softcap > 0.f;
    const float kinv = capped ? p.scale / p.softcap : 0.f;
    const float c_eff = XF ? 1.f : sc;   // of a value in x, to the units of m_ref
    uint32_t x[BN];
    int j = 0;   // key tiles so far
    bool ok = true;
    float m_ref = -INFINITY, l = 0.f;
    int done = 0;   // of them, this item's
    for (int k = 0; ok && k < my_items; ++k) {
      const int buf = k & 1;
      if (!(ok = wait_warp(&sb.item_full[buf], (uint32_t)(k >> 1) & 1u, &sb.abort, p.status))) break;
      const int n = items[buf].n, n_my = t ? (items[buf].some1 ? n : 0) : items[buf].n0;
      const int skip = t ? items[buf].skip1 : -1;
      const int h = items[buf].h + t * ht_step, b = items[buf].b;
      const int qrow = items[buf].q0 + t * rt_step + r;
      const Vis* rv = &row_v[buf][t * BM + r];
      const bool valid = qrow < p.Sq && h < (items[buf].g + 1) * p.qpg;
      const bool idle = !__any_sync(0xffffffffu, valid);   // no row of this warp exists: its P is not used
      const float* mrow = nullptr;
      if (XF && p.M && qrow < p.Sq)
        mrow = p.M + p.m.off + (int64_t)b * p.m.bs + (int64_t)h * p.m.hs + (int64_t)qrow * p.m.rs;
      m_ref = -INFINITY;
      l = 0.f;
      done = 0;
      for (int i = 0; i < n_my; ++i) {
        if (i == skip) continue;
        if (!(ok = wait_warp(&sb.s_full[t], (uint32_t)j & 1u, &sb.abort, p.status))) break;
        fence_after();
        const int k0 = items[buf].key(i);
        bool rescale = false;
        float corr = 1.f;
        // The first N columns of the tile.  With a finite reference maximum P is
        // computed against it without scanning for the tile's maximum; a row
        // whose tile sum reaches kLagMax makes the warp redo the tile with the
        // scan.
        auto step = [&](auto cols) {
          constexpr int N = decltype(cols)::value;
          constexpr float kLagMax = BF16 ? 0x1p64f : 65504.f;   // (no p of f16 overflows below)
          bool scan = __any_sync(0xffffffffu, !(m_ref > -INFINITY));
#pragma unroll 1
          for (int pass = 0; pass < 2; ++pass) {
            if constexpr (XF) {
              // Scores, one 32-column chunk at a time.
#pragma unroll
              for (int c = 0; c < N / 32; ++c) {
                const uint32_t seen = seen_bits(*rv, k0 + c * 32);
                tmem_ld32(s_tm + c * 32, x + c * 32);
                tmem_ld_wait_regs<1>(x + c * 32);
#pragma unroll
                for (int e = c * 32; e < c * 32 + 32; ++e) {
                  float v = -INFINITY;
                  if ((seen >> (e % 32)) & 1u) {
                    const float s = __uint_as_float(x[e]);
                    v = capped ? p.softcap * tanh_exp2(s * kinv) : s * p.scale;
                    if (mrow) v += mrow[k0 + e];
                  }
                  x[e] = __float_as_uint(v);
                  if ((e & 7) == 7) asm volatile("" ::: "memory");  // at most 8 mask loads in flight
                }
              }
            } else {
#pragma unroll
              for (int c = 0; c < N / 32; ++c) tmem_ld32(s_tm + c * 32, x + c * 32);
              tmem_ld_wait_regs<N / 32>(x);
              const Vis v = *rv;
              if (!within(v, k0, k0 + N)) {   // hide by bits, one select a column
#pragma unroll
                for (int c = 0; c < N / 32; ++c) {
                  const uint32_t seen = seen_bits(v, k0 + c * 32);
#pragma unroll
                  for (int e = 0; e < 32; ++e)
                    if (!(seen & (1u << e))) x[c * 32 + e] = __float_as_uint(-INFINITY);
                }
              }
            }
            if (scan) {
              float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
              for (int e = 0; e < N; e += 4) {
                mx0 = max3(mx0, __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
                mx1 = max3(mx1, __uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]));
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
            for (int e = 0; e < N; e += 4) {
              float a0, a1, b0, b1;
              fma2(a0, a1, __uint_as_float(x[e]), __uint_as_float(x[e + 1]), c2, n2);
              fma2(b0, b1, __uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]), c2, n2);
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
              x[e / 2] = pack2<BF16>(a0, a1);
              x[e / 2 + 1] = pack2<BF16>(b0, b1);
            }
            const float lt = (la0 + la1) + (lb0 + lb1);
            if (scan || !__any_sync(0xffffffffu, lt >= kLagMax)) {   // NaN sums stay (a NaN row)
              l += lt;
              break;
            }
            scan = true;
          }
          // (a short tile's P is its first 16 words; its P V reads no others)
#pragma unroll
          for (int c = 0; c < (N + 63) / 64; ++c) tmem_st32(s_tm + c * 32, x + c * 32);
        };
        if (!idle) {
          if (!XF && items[buf].is_short(i)) step(std::integral_constant<int, kShort>());
          else step(std::integral_constant<int, BN>());
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
      // ---- epilogue: O / l, special rows, LSE ----
      if (done > 0 && !(ok = wait_warp(&sb.o_done[t], (uint32_t)(j - 1) & 1u, &sb.abort, p.status))) break;
      fence_after();
      if (clustered) break;   // (its only item)
      const bool split = sp.n_splits > 1;
      // The sink logit joins the denominator (and rescales the accumulated O); with parts the merge adds it once.
      float M = S::natural(m_ref);
      const float o_mul = p.sink_on && !split ? fold_sink<false>(M, l, sink_logit(p, h)) : 1.f;
      const bool hidden_row = (l == 0.f);         // no visible key; a NaN l stays a NaN row
      const float inv = o_mul / l;
      const float fill = p.masked_zero ? 0.f : NAN;
      T* orow = static_cast<T*>(p.O) + p.o.off + (int64_t)b * p.o.bs + (int64_t)h * p.o.hs + (int64_t)qrow * p.o.rs;
      const int64_t prow = ((int64_t)b * p.H + h) * p.Sq + qrow;
      float4* po = split ? reinterpret_cast<float4*>(sp.part_o + (prow * sp.n_splits + items[buf].part) * D) : nullptr;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (done > 0) {
          tmem_ld32(o_tm + c * 32, o);
          tmem_ld_wait_regs<1>(o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
        if (split) {
          if (valid && !hidden_row) {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * inv);
#pragma unroll
            for (int e = 0; e < 32; e += 8) store32(po + c * 8 + e / 4, o + e);
          }
        } else {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float a = hidden_row ? fill : __uint_as_float(o[e]) * inv;
            const float bb = hidden_row ? fill : __uint_as_float(o[e + 1]) * inv;
            w[e / 2] = pack2<BF16>(a, bb);
          }
          if (valid) {
            if (wide_rows) {
              store32(orow + c * 32, w);
              store32(orow + c * 32 + 16, w + 8);
            } else {
              uint4* dst = reinterpret_cast<uint4*>(orow + c * 32);
#pragma unroll
              for (int v4 = 0; v4 < 4; ++v4)
                dst[v4] = make_uint4(w[4 * v4], w[4 * v4 + 1], w[4 * v4 + 2], w[4 * v4 + 3]);
            }
          }
        }
      }
      if (valid) {
        const float lse = hidden_row ? -INFINITY : S::lse(M, __log2f(l));
        if (split) {
          const int64_t at = prow * sp.n_splits + items[buf].part;
          sp.part_lse[at] = XF && sp.part_l && !hidden_row ? M : lse;
          if (XF && sp.part_l) sp.part_l[at] = l;
        } else if (p.lse) {
          p.lse[(int64_t)b * p.lse_bs + (int64_t)h * p.lse_hs + qrow] = lse;
        }
      }
      fence_before();   // O's loads come before the next item's P, and so before its P V
      mbar_arrive(&sb.item_empty[buf]);
    }
    if (clustered) {
      cluster_sync();   // every P V is done with V's stages
      const int row = t * BM + r;
      part_m[row] = m_ref;
      part_l[row] = l;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (done > 0) {   // (warp-uniform)
          tmem_ld32(o_tm + c * 32, o);
          tmem_ld_wait_regs<1>(o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0u;
        }
#pragma unroll
        for (int e = 0; e < 32; e += 4)
          part_a[(c * 8 + e / 4) * 2 * BM + row] = make_float4(__uint_as_float(o[e]), __uint_as_float(o[e + 1]),
                                                               __uint_as_float(o[e + 2]), __uint_as_float(o[e + 3]));
      }
      cluster_sync();
      // This CTA's rows: a thread takes 16 columns of a row from every part.
      const int parts = sp.n_splits, rows = 2 * BM / parts;
      const Item& it = items[0];
      for (int u = threadIdx.x; u < rows * (D / 16); u += 2 * BM) {
        const int mine = (int)cluster_rank() * rows + u % rows, col = u / rows * 16, tt = mine / BM;
        const int i = it.q0 + (pair_heads ? mine % BM : mine), hh = it.h + tt * ht_step;
        if (i >= p.Sq || hh >= (it.g + 1) * p.qpg) continue;
        float M = -INFINITY, L = 0.f, a[16];
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (q < parts) M = fmaxf(M, peer(part_m + mine, q));
        const float mu = M == -INFINITY ? 0.f : M;
#pragma unroll
        for (int e = 0; e < 16; ++e) a[e] = 0.f;
#pragma unroll 1
        for (int q0 = 0; q0 < parts; q0 += 4) {   // the loads of up to four parts before their sums
          float f[4], lq[4];
          float4 y[4][4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (q0 + q >= parts) continue;
            f[q] = peer(part_m + mine, q0 + q);
            lq[q] = peer(part_l + mine, q0 + q);
#pragma unroll
            for (int e = 0; e < 4; ++e) y[q][e] = peer4(part_a + (col / 4 + e) * 2 * BM + mine, q0 + q);
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            if (q0 + q >= parts) continue;
            f[q] = S::weight(f[q], mu);
            L = fmaf(f[q], lq[q], L);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              a[4 * e] = fmaf(f[q], y[q][e].x, a[4 * e]);
              a[4 * e + 1] = fmaf(f[q], y[q][e].y, a[4 * e + 1]);
              a[4 * e + 2] = fmaf(f[q], y[q][e].z, a[4 * e + 2]);
              a[4 * e + 3] = fmaf(f[q], y[q][e].w, a[4 * e + 3]);
            }
          }
        }
        M = S::natural(M);
        const float o_mul = p.sink_on ? fold_sink<false>(M, L, sink_logit(p, hh)) : 1.f;
        const bool hidden = L == 0.f;
        const float inv = o_mul / L, fill = p.masked_zero ? 0.f : NAN;
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 16; e += 2) w[e / 2] = pack2<BF16>(hidden ? fill : a[e] * inv, hidden ? fill : a[e + 1] * inv);
        T* dst = static_cast<T*>(p.O) + p.o.off + (int64_t)it.b * p.o.bs + (int64_t)hh * p.o.hs + (int64_t)i * p.o.rs + col;
        if (wide_rows) {
          store32(dst, w);
        } else {
          reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
          reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
        if (col == 0 && p.lse)
          p.lse[(int64_t)it.b * p.lse_bs + (int64_t)hh * p.lse_hs + i] = hidden ? -INFINITY : S::lse(M, __log2f(L));
      }
      cluster_sync();   // no CTA leaves while its part is being read
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
int launch(const Problem& p, int first, const Split& sp, cudaStream_t st) {
  CUtensorMap mq, mk, mv;
  if (!tma_map_bhsd(&mq, p.Q, p.dtype, D, p.Sq, p.H, p.B, p.q, BM) ||
      !tma_map_bhsd(&mk, p.K, p.dtype, D, p.Sk, p.G, p.B, p.k, BN) ||
      !tma_map_bhsd(&mv, p.V, p.dtype, D, p.Sk, p.G, p.B, p.v, BN))
    return -1;  // not describable: caller falls back
  const int pair = (p.Sq <= BM && p.qpg >= 2) ? 1 : 0;
  const int64_t nqb = (p.Sq + 2 * BM - 1) / (2 * BM);
  const int64_t n = (pair ? (int64_t)p.B * p.G * ((p.qpg + 1) / 2) : nqb * p.H * p.B) * sp.n_splits;
  if (n > 0x3fffffff) return -1;
  const int smem = Cfg<D>::kSmem + 1024;
  auto kern = window_tc_kernel<D, BF16, XF>;
  // setmaxnreg.inc waits until the block's register pool holds the larger
  // count, so the pool the kernel is launched with must cover the split.
  static const bool regs_ok = [] {
    cudaFuncAttributes a;
    if (cudaFuncGetAttributes(&a, (const void*)window_tc_kernel<D, BF16, XF>) != cudaSuccess) return false;
    return a.numRegs * kThreads >= kSplitRegs;
  }();
  if (!regs_ok) return -1;
  if (ensure_smem((const void*)kern, smem) != cudaSuccess) return ATTN_ERR_CUDA;
  // Rows of O on 32-byte boundaries take 32-byte stores.
  auto even = [](int64_t stride, int64_t extent) { return extent <= 1 || stride % 16 == 0; };
  const int wide = ((uintptr_t)p.O + (uintptr_t)p.o.off * 2) % 32 == 0 && even(p.o.bs, p.B) && even(p.o.hs, p.H) &&
                           even(p.o.rs, p.Sq)
                       ? 1
                       : 0;
  const int drop = take_injection() == ATTN_INJECT_DROP_FIRST_COPY ? 1 : 0;
  // Parts without a workspace are a cluster's CTAs.
  const int clustered = sp.n_splits > 1 && !sp.part_o ? 1 : 0;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)sp.n_splits;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)(clustered || n < kSms ? n : kSms));
  c.blockDim = dim3(kThreads);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  c.attrs = &at;
  c.numAttrs = clustered;
  return cudaLaunchKernelEx(&c, kern, mq, mk, mv, p, first, pair, (int)n, wide, clustered, drop, sp) == cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_CUDA;
}

template <int D>
int launch_d(const Problem& p, int first, const Split& sp, cudaStream_t st) {
  const bool xf = p.M != nullptr || p.softcap > 0.f || !(p.scale * kLog2e > 0.f);
  if (p.dtype == ATTN_BF16) return xf ? launch<D, true, true>(p, first, sp, st) : launch<D, true, false>(p, first, sp, st);
  return xf ? launch<D, false, true>(p, first, sp, st) : launch<D, false, false>(p, first, sp, st);
}

}  // namespace win
}  // namespace attn
