// paged_mma.cuh -- decode over a paged cache at head_dim 64, 128 or 256 with
// f16/bf16 queries and an f16/bf16 or int8 cache.
//
// What it computes: for one query row per (batch entry, head),
// O = softmax(scale q K^T + mask) V and its LSE over the entry's visible rows,
// with the online normaliser of "Attention" (recursiveai.org OneGPU docs),
// opening paragraph; the work is shared out as paged.cuh describes.
//
// What bounds it: HBM.  A cache byte is read once (a unit holds up to 8 or 16
// query heads of its kv head), so everything here serves to keep reads in
// flight.  Each of a CTA's four warps streams its own quarter of every key
// tile through its own ring of stages with cp.async: a row's address comes from
// the page list, so any page size, pool order and stride goes the same way,
// hidden rows and rows without a page arrive as zeros without being read, and
// a warp waits for its own copies only -- no barrier in the loop.  The ring
// runs on across fragments, so a unit's merge and output overlap the next
// unit's loads.
//
// The contractions use mma.sync m16n8k16 with the keys on the 16 rows and the
// query heads on the 8 columns (few heads share a kv head): S^T = K Q^T with K
// from ldmatrix, O^T += V^T P^T with V from ldmatrix.trans and P^T from the
// S^T accumulator through movmatrix.  P enters as the sum of two rounded
// halves (p rounded, and the rest rounded), so that the result carries the
// output's rounding only; the extra MMAs are free under the HBM time.
//
// int8 caches enter the MMAs as exact f16 integers (0x6400 | (x ^ 0x80) is
// 1152 + x, minus 1152).  The scales leave the loop: Q is scaled by k_scale,
// and by a power of two for each head that puts its largest element next to
// 2^11, and enters as two f16 halves; v_scale multiplies the finished row.
#pragma once

#include <type_traits>

#include "paged.cuh"

namespace attn {
namespace paged {

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ uint32_t movtrans(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
template <bool BF16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (BF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two floats rounded to the MMA type, and what the rounding left of them.
template <bool BF16>
__device__ __forceinline__ uint32_t pack_split(float a, float b, uint32_t& rest) {
  if constexpr (BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    const __nv_bfloat162 r = __floats2bfloat162_rn(a - __low2float(h), b - __high2float(h));
    rest = *reinterpret_cast<const uint32_t*>(&r);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __half2 h = __floats2half2_rn(a, b);
    const __half2 r = __floats2half2_rn(a - __low2float(h), b - __high2float(h));
    rest = *reinterpret_cast<const uint32_t*>(&r);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}
// Bytes 0 and 2 (or 1 and 3) of a word of int8 values as an exact f16 pair.
__device__ __forceinline__ uint32_t half_pair(uint32_t w, bool high) {
  const uint32_t biased = ((high ? w >> 8 : w) & 0x00FF00FFu) ^ 0x64806480u;   // 1152 + x
  const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&biased), __half2half2(__ushort_as_half(0x6480)));
  return *reinterpret_cast<const uint32_t*>(&v);
}

// KV8: int8 cache (MMAs in f16).  NT: column tiles of 8 query heads.
template <bool BF16, bool KV8, int D, int NT>
struct Cfg {
  static constexpr int kRow = D * (KV8 ? 1 : 2);                  // bytes of a cache row
  static constexpr int kUnits = kRow / 16;                        // 16-byte units of a row
  static constexpr int kKeys = kRow <= 128 ? 32 : 16;             // keys of a warp's stage
  static constexpr int kStage = 2 * kKeys * kRow;                 // bytes: K rows, then V rows
  static constexpr int kStages = 3;
  static constexpr int kRing = kWarps * kStages * kStage;
  static constexpr int kHeads = 8 * NT;
  static constexpr int kRed = kWarps * kHeads * 64 * 4;           // merge buffer: 64 columns at a time
  static constexpr int kSmem = kRing + kRed;
  static constexpr int kCtas = kSmem <= 113 * 1024 ? 2 : 1;       // an SM
  static constexpr int kTile = kWarps * kKeys;
};

// The 16-byte unit u of row r in a stage: swizzled so that the 8 rows an
// ldmatrix phase reads lie in different banks.
template <int UNITS>
__device__ __forceinline__ uint32_t swz(int r, int u) {
  return (uint32_t)(r * UNITS * 16 + ((u ^ (UNITS >= 8 ? r & 7 : (r >> 1) & 3)) << 4));
}

// XF: scores under a softcap or an additive mask.
template <bool BF16, bool KV8, int D, int NT, bool XF>
__global__ void __launch_bounds__(kThreads, Cfg<BF16, KV8, D, NT>::kCtas) paged_mma_kernel(const Work w) {
  using C = Cfg<BF16, KV8, D, NT>;
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  constexpr bool MB = BF16 && !KV8;   // MMA type bf16
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int st_key[kWarps][C::kStages];         // first key of a warp's stage
  __shared__ uint32_t st_vis[kWarps][C::kStages];    // which of its keys are visible
  __shared__ float red_m[kWarps][C::kHeads], red_l[kWarps][C::kHeads];
  const Problem& p = w.p;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, gid = lane >> 2, tig = lane & 3;
  const int units = p.G * w.n_hc;

  const int64_t total = tiles_before(w, p.B, lane) * units;
  const int shares = (int)min((int64_t)w.ctas, total);
  const int cta = blockIdx.x;
  if (cta >= shares) return;
  const int64_t t0 = share_begin(total, shares, cta);
  const int my = (int)(share_begin(total, shares, cta + 1) - t0);   // tiles of this share
  Cursor in = seek(w, t0, units, lane), out = in;

  uint8_t* ring = smem + warp * C::kStages * C::kStage;
  const uint32_t ring_a = smem_u32(ring);
  constexpr int kEs = KV8 ? 1 : 2;
  const uint8_t* kbase = static_cast<const uint8_t*>(p.K) + p.k.off * kEs;
  const uint8_t* vbase = static_cast<const uint8_t*>(p.V) + p.v.off * kEs;
  const bool one_page = w.x.page_size % C::kKeys == 0;   // a stage's keys share a page
  const int kr = lane % C::kKeys;                        // the stage row whose page this lane looks up

  // Page of this lane's row of the input cursor's tile.
  auto look_up = [&]() {
    const int key = in.tl.tile(in.tile) * C::kTile + warp * C::kKeys + kr;
    return visible(in.v, key) ? page_of(w.x, in.b, key) : -1;
  };
  int page = look_up();
  // Issues the input cursor's tile into a stage and moves on; `more`: another tile follows.
  auto issue = [&](int s, bool more) {
    const int k0 = in.tl.tile(in.tile) * C::kTile + warp * C::kKeys;
    const uint32_t vis = __ballot_sync(kAll, page >= 0);   // (bit r = row r; 16-key stages repeat)
    const int g = in.u / w.n_hc;
    const int r = (k0 + kr) % w.x.page_size;
    const int64_t ko = ((int64_t)max(page, 0) * p.k.bs + (int64_t)g * p.k.hs + (int64_t)r * p.k.rs) * kEs;
    const int64_t vo = ((int64_t)max(page, 0) * p.v.bs + (int64_t)g * p.v.hs + (int64_t)r * p.v.rs) * kEs;
    if (lane == 0) {
      st_key[warp][s] = k0;
      st_vis[warp][s] = vis;
    }
    const uint32_t dst = ring_a + s * C::kStage;
    constexpr int kRowsPer = 32 / C::kUnits;   // rows of one pass over the lanes (C::kUnits <= 32)
    const int u = lane % C::kUnits, ru = lane / C::kUnits;
    if (one_page && (vis == kAll || (C::kKeys == 16 && (vis & 0xffffu) == 0xffffu))) {
      // Every row of one page: the addresses advance by the row stride.
      const uint8_t* ks = kbase + __shfl_sync(kAll, ko, 0) + (int64_t)ru * p.k.rs * kEs + u * 16;
      const uint8_t* vs = vbase + __shfl_sync(kAll, vo, 0) + (int64_t)ru * p.v.rs * kEs + u * 16;
      const int64_t kst = (int64_t)kRowsPer * p.k.rs * kEs, vst = (int64_t)kRowsPer * p.v.rs * kEs;
#pragma unroll
      for (int j = 0; j < C::kKeys / kRowsPer; ++j)
        copy16(dst + swz<C::kUnits>(j * kRowsPer + ru, u), ks + j * kst, 16);
#pragma unroll
      for (int j = 0; j < C::kKeys / kRowsPer; ++j)
        copy16(dst + C::kKeys * C::kRow + swz<C::kUnits>(j * kRowsPer + ru, u), vs + j * vst, 16);
    } else {
#pragma unroll
      for (int j = 0; j < C::kKeys / kRowsPer; ++j) {
        const int row = j * kRowsPer + ru;
        const int64_t a = __shfl_sync(kAll, ko, row), c = __shfl_sync(kAll, vo, row);
        const int sz = (vis >> row) & 1u ? 16 : 0;
        copy16(dst + swz<C::kUnits>(row, u), kbase + a + u * 16, sz);
        copy16(dst + C::kKeys * C::kRow + swz<C::kUnits>(row, u), vbase + c + u * 16, sz);
      }
    }
    if (more) {   // look the next tile's pages up a tile ahead of their use
      in.next(w, units);
      page = look_up();
    }
  };
#pragma unroll
  for (int s = 0; s < C::kStages - 1; ++s) {
    if (s < my) issue(s, s + 1 < my);
    copy_commit();
  }

  // Q as the B operand (n = head, k = channels).
  uint32_t qh[NT][D / 16][2], ql[KV8 ? NT : 1][D / 16][2];
  float cs[NT][2];   // what a raw product is multiplied by, for the accumulator's two head columns
  auto load_q = [&]() {
    const int g = out.u / w.n_hc, h0 = g * p.qpg + (out.u % w.n_hc) * C::kHeads;
    const int nh = min(C::kHeads, (g + 1) * p.qpg - h0);
    const T* Q = static_cast<const T*>(p.Q) + p.q.off + (int64_t)out.b * p.q.bs;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int hh = 8 * j + gid;
      const T* row = Q + (int64_t)(h0 + hh) * p.q.hs;
      if constexpr (!KV8) {
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int d = 16 * c + 8 * e + 2 * tig;
            const uint16_t* src = reinterpret_cast<const uint16_t*>(row + d);
            qh[j][c][e] = hh < nh ? (uint32_t)src[0] | ((uint32_t)src[1] << 16) : 0u;
          }
        cs[j][0] = cs[j][1] = p.scale * kLog2e;
      } else {
        // Channels 4t, 4t + 2 (then 4t + 1, 4t + 3) of a 16-channel block: the order in which the bytes arrive.
        float top = 0.f;
#pragma unroll
        for (int c = 0; c < D / 4; c += 4)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int d = 4 * c + 4 * tig + e;
            if (hh < nh) top = fmaxf(top, fabsf(to_f32(row[d]) * p.k_scale[p.kv_per_channel ? g * D + d : 0]));
          }
        top = fmaxf(top, __shfl_xor_sync(kAll, top, 1));
        top = fmaxf(top, __shfl_xor_sync(kAll, top, 2));
        int ex = 0;
        if (top > 0.f && top < INFINITY) {
          frexpf(top, &ex);
          ex = max(-110, min(11 - ex, 110));   // 2^ex puts the largest element in [2^10, 2^11)
        }
        const float up = ldexpf(1.f, ex);
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int d = 16 * c + 4 * tig + e;
            v[e] = hh < nh ? to_f32(row[d]) * p.k_scale[p.kv_per_channel ? g * D + d : 0] * up : 0.f;
          }
          qh[j][c][0] = pack_split<false>(v[0], v[2], ql[j][c][0]);
          qh[j][c][1] = pack_split<false>(v[1], v[3], ql[j][c][1]);
        }
        const float down = p.scale * kLog2e * ldexpf(1.f, -ex);
        cs[j][0] = __shfl_sync(kAll, down, 8 * tig);       // heads 2 tig and 2 tig + 1 of the column tile
        cs[j][1] = __shfl_sync(kAll, down, 8 * tig + 4);
      }
    }
  };
  load_q();

  // O^T: rows 16 c + gid (and + 8) of the channels (int8: channels 16 c + 2 gid
  // and + 1), columns heads 8 j + 2 tig and + 1.
  float o[D / 16][NT][4], m_ref[NT][2], l[NT][2];
  auto reset = [&]() {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[c][j][e] = 0.f;
      m_ref[j][0] = m_ref[j][1] = -INFINITY;
      l[j][0] = l[j][1] = 0.f;
    }
  };
  reset();
  const bool capped = XF && p.softcap > 0.f;
  const float cap2 = p.softcap * kLog2e, cap_inv = capped ? 1.f / cap2 : 0.f;
  // ldmatrix source rows and unit offsets of this lane (K: keys x channels; V transposed).
  const int lk_row = (lane & 7) + ((lane >> 3) & 1) * 8, lk_u = lane >> 4;
  const int lv_row = KV8 ? lk_row : (lane & 7) + (lane >> 4) * 8, lv_u = KV8 ? lane >> 4 : (lane >> 3) & 1;

  int first_tile = out.tile, frag = 0;   // where the current fragment began in its unit; its number in this share
  for (int i = 0; i < my; ++i) {
    const int s = i % C::kStages;
    if (i + C::kStages - 1 < my) issue((i + C::kStages - 1) % C::kStages, i + C::kStages < my);
    copy_commit();
    copy_wait<C::kStages - 1>();
    __syncwarp();
    const uint32_t ks = ring_a + s * C::kStage, vs = ks + C::kKeys * C::kRow;
    const uint32_t vis = st_vis[warp][s];
#pragma unroll
    for (int mb = 0; mb < C::kKeys / 16; ++mb) {
      const uint32_t vb = (vis >> (16 * mb)) & 0xffffu;
      if (vb == 0) continue;
      float sc[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[j][e] = 0.f;
      if constexpr (!KV8) {
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          uint32_t a[4];
          ldsm4(ks + swz<C::kUnits>(16 * mb + lk_row, 2 * c + lk_u), a);
#pragma unroll
          for (int j = 0; j < NT; ++j) mma<MB>(sc[j], a, qh[j][c][0], qh[j][c][1]);
        }
      } else {
#pragma unroll
        for (int c = 0; c < D / 16; c += 2) {   // two 16-channel blocks: keys 0-7 and 8-15 of each
          uint32_t kw[4];
          ldsm4(ks + swz<C::kUnits>(16 * mb + lk_row, c + lk_u), kw);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint32_t a[4] = {half_pair(kw[2 * q], false), half_pair(kw[2 * q + 1], false),
                                   half_pair(kw[2 * q], true), half_pair(kw[2 * q + 1], true)};
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              mma<false>(sc[j], a, qh[j][c + q][0], qh[j][c + q][1]);
              mma<false>(sc[j], a, ql[j][c + q][0], ql[j][c + q][1]);
            }
          }
        }
      }
      // Scores in log2 units; hidden keys (rows gid and gid + 8 of the block) become -inf.
      bool rise = false;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = sc[j][e] * cs[j][e & 1];
          const int r = gid + 8 * (e >> 1);
          if (XF) {
            if (capped) x = cap2 * tanh_exp2(x * cap_inv);
            const int hh = 8 * j + 2 * tig + (e & 1);
            const int in_kv = (out.u % w.n_hc) * C::kHeads + hh;
            if (p.M && in_kv < p.qpg && ((vb >> r) & 1u))
              x = fmaf(p.M[p.m.off + (int64_t)out.b * p.m.bs +
                           (int64_t)(out.u / w.n_hc * p.qpg + in_kv) * p.m.hs + st_key[warp][s] + 16 * mb + r],
                       kLog2e, x);
          }
          sc[j][e] = (vb >> r) & 1u ? x : -INFINITY;
          rise |= sc[j][e] > m_ref[j][e & 1] + kSlack;
        }
      if (__any_sync(kAll, rise)) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int q = 0; q < 2; ++q) {   // a column's keys are spread over the lanes of a tig
            float mx = fmaxf(sc[j][q], sc[j][q + 2]);
            mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 4));
            mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 8));
            mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 16));
            if (mx > m_ref[j][q] + kSlack) {
              const float f = ex2_approx(m_ref[j][q] - mx);
              l[j][q] *= f;
#pragma unroll
              for (int c = 0; c < D / 16; ++c) {
                o[c][j][q] *= f;
                o[c][j][q + 2] *= f;
              }
              m_ref[j][q] = mx;
            }
          }
      }
      uint32_t ph[NT][2], pl[NT][2];   // P^T: keys 2 tig, + 1 (then + 8) x head gid
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const float mu0 = m_ref[j][0] == -INFINITY ? 0.f : m_ref[j][0];
        const float mu1 = m_ref[j][1] == -INFINITY ? 0.f : m_ref[j][1];
        float e[4];
        e[0] = ex2_approx(sc[j][0] - mu0);
        e[1] = ex2_approx(sc[j][1] - mu1);
        e[2] = ex2_approx(sc[j][2] - mu0);
        e[3] = ex2_approx(sc[j][3] - mu1);
        l[j][0] += e[0] + e[2];
        l[j][1] += e[1] + e[3];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t rest;
          ph[j][q] = movtrans(pack_split<MB>(e[2 * q], e[2 * q + 1], rest));
          pl[j][q] = movtrans(rest);
        }
      }
      if constexpr (!KV8) {
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          uint32_t a[4];
          ldsm4t(vs + swz<C::kUnits>(16 * mb + lv_row, 2 * c + lv_u), a);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            mma<MB>(o[c][j], a, ph[j][0], ph[j][1]);
            mma<MB>(o[c][j], a, pl[j][0], pl[j][1]);
          }
        }
      } else {
#pragma unroll
        for (int c = 0; c < D / 16; c += 2) {
          uint32_t vw[4];   // (block c, keys 0-7), (c, 8-15), (c + 1, 0-7), (c + 1, 8-15)
          ldsm4t(vs + swz<C::kUnits>(16 * mb + lv_row, c + lv_u), vw);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint32_t a[4] = {half_pair(vw[2 * q], false), half_pair(vw[2 * q], true),
                                   half_pair(vw[2 * q + 1], false), half_pair(vw[2 * q + 1], true)};
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              mma<false>(o[c + q][j], a, ph[j][0], ph[j][1]);
              mma<false>(o[c + q][j], a, pl[j][0], pl[j][1]);
            }
          }
        }
      }
    }
    __syncwarp();   // the stage is free

    const bool unit_ends = out.tile + 1 == out.n;
    if (unit_ends || i + 1 == my) {
      // The fragment ends: the four warps' results, merged in warp order, 64 columns at a time.
      const bool whole = unit_ends && first_tile == 0;
      const int slot = frag == 0 ? 0 : 1;
      const int g = out.u / w.n_hc, h0 = g * p.qpg + (out.u % w.n_hc) * C::kHeads;
      const int nh = min(C::kHeads, (g + 1) * p.qpg - h0);
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float x = l[j][q];
          x += __shfl_xor_sync(kAll, x, 4);
          x += __shfl_xor_sync(kAll, x, 8);
          x += __shfl_xor_sync(kAll, x, 16);
          if (gid == 0) {
            red_m[warp][8 * j + 2 * tig + q] = m_ref[j][q];
            red_l[warp][8 * j + 2 * tig + q] = x;
          }
        }
      float* red = reinterpret_cast<float*>(smem + C::kRing);   // [kWarps][kHeads][64]
#pragma unroll
      for (int part = 0; part < D / 64; ++part) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int d = 16 * c + (KV8 ? 2 * gid + (e >> 1) : gid + 8 * (e >> 1));
              red[(warp * C::kHeads + 8 * j + 2 * tig + (e & 1)) * 64 + d] = o[4 * part + c][j][e];
            }
        __syncthreads();
        for (int x = threadIdx.x; x < nh * 64; x += kThreads) {
          const int hh = x / 64, d = x % 64;
          float M = -INFINITY;
#pragma unroll
          for (int v = 0; v < kWarps; ++v) M = fmaxf(M, red_m[v][hh]);
          const float mu = M == -INFINITY ? 0.f : M;
          float L = 0.f, a = 0.f;
#pragma unroll
          for (int v = 0; v < kWarps; ++v) {
            const float f = ex2_approx(red_m[v][hh] - mu);
            L = fmaf(f, red_l[v][hh], L);
            a = fmaf(f, red[(v * C::kHeads + hh) * 64 + d], a);
          }
          const int dd = 64 * part + d;
          if (KV8) a *= p.v_scale[p.kv_per_channel ? g * D + dd : 0];
          put_row<T>(w, whole, cta, slot, out.b, h0 + hh, hh, dd, M, L, a);
        }
        __syncthreads();
      }
      ++frag;
    }
    if (i + 1 < my) {
      out.next(w, units);
      if (unit_ends) {
        first_tile = 0;
        load_q();
        reset();
      }
    }
  }
  copy_wait<0>();
}

template <bool BF16, bool KV8, int D, int NT, bool XF>
int launch_cfg(Work& w, cudaStream_t st) {
  using C = Cfg<BF16, KV8, D, NT>;
  auto kern = paged_mma_kernel<BF16, KV8, D, NT, XF>;
  if (ensure_smem((const void*)kern, C::kSmem) != cudaSuccess) return ATTN_ERR_CUDA;
  kern<<<w.ctas, kThreads, C::kSmem, st>>>(w);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

// Fills in the tile, the head chunks and the shares: two CTAs an SM (their
// rings fill its shared memory), never more than there can be tiles.
template <bool BF16, bool KV8, int D, int NT>
int plan_cfg(Work& w, bool launch, cudaStream_t st) {
  using C = Cfg<BF16, KV8, D, NT>;
  w.unit = C::kTile;
  w.heads = C::kHeads;
  w.n_hc = (w.p.qpg + C::kHeads - 1) / C::kHeads;
  const int64_t most = (int64_t)w.p.B * w.p.G * w.n_hc * ((w.p.Sk + (int64_t)C::kTile - 1) / C::kTile);
  w.ctas = (int)max((int64_t)1, min((int64_t)kSms * C::kCtas, most));
  if (!launch) return ATTN_OK;
  const bool xf = w.p.softcap > 0.f || w.p.M != nullptr;
  return xf ? launch_cfg<BF16, KV8, D, NT, true>(w, st) : launch_cfg<BF16, KV8, D, NT, false>(w, st);
}

// Two column tiles of heads a unit for more than eight heads a kv head (at
// head_dim 256 they would not fit the registers: the units then take eight
// heads each and read the cache rows again from L2).
template <bool BF16, bool KV8>
bool pick(Work& w, bool launch, cudaStream_t st, int* rc) {
  const bool two = w.p.qpg > 8;
  switch (w.p.D) {
    case 64: *rc = two ? plan_cfg<BF16, KV8, 64, 2>(w, launch, st) : plan_cfg<BF16, KV8, 64, 1>(w, launch, st); return true;
    case 128: *rc = two ? plan_cfg<BF16, KV8, 128, 2>(w, launch, st) : plan_cfg<BF16, KV8, 128, 1>(w, launch, st); return true;
    case 256: *rc = plan_cfg<BF16, KV8, 256, 1>(w, launch, st); return true;
    default: return false;
  }
}

}  // namespace paged
}  // namespace attn
