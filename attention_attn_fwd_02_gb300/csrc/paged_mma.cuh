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
// S^T accumulator through movmatrix.  P enters as the sum of two halves (p
// cut, and the rest rounded), so that the result carries the output's rounding
// only; the extra MMAs are free under the HBM time.  Over float caches both
// halves of a p > 0 are above zero, so that an infinite V gives an infinite
// result, as in the formula, and not the NaN of infinity times zero or less.
//
// int8 caches enter the MMAs as exact f16 integers (0x6400 | (x ^ 0x80) is
// 1152 + x, minus 1152).  The scales leave the loop: Q is scaled by k_scale,
// and by a power of two for each head that puts its largest element next to
// 2^11, and enters as two f16 halves (22 bits: a score of 200 keeps an error of
// 2^-14, where one f16 value would leave 0.05); v_scale multiplies the finished
// row.  With Q and P as one f16 value each the batch of 64 takes 110 us, with P
// as one 114, with both in halves 119 (and the result carries the output's rounding only).
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
// Two probabilities (>= 0) as sums of two values of the MMA type, both above zero where the probability is.  The
// first is cut a little below its value: p is off by 2^-15.6 of itself in bf16 (2^-9 of a rest that is at most 2^-7
// + 2^-9 of p), in f16 by 2^-21, or by 2^-23 in all where it is small and the halves are lifted to f16's least value.
template <bool BF16>
__device__ __forceinline__ uint32_t pack_above_zero(float a, float b, uint32_t& rest) {
  if constexpr (BF16) {
    const uint32_t ah = __float_as_uint(a * (1.f - 0x1p-9f)) & 0xffff0000u;
    const uint32_t bh = __float_as_uint(b * (1.f - 0x1p-9f)) & 0xffff0000u;
    const __nv_bfloat162 r = __floats2bfloat162_rn(a - __uint_as_float(ah), b - __uint_as_float(bh));
    rest = *reinterpret_cast<const uint32_t*>(&r);
    return __byte_perm(ah, bh, 0x7632);
  } else {
    uint32_t h;
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(b * (1.f - 0x1p-10f)), "f"(a * (1.f - 0x1p-10f)));
    const __half2 hh = *reinterpret_cast<const __half2*>(&h);
    const __half2 r = __floats2half2_rn(a - __low2float(hh), b - __high2float(hh));
    const uint32_t least = (a > 0.f ? 1u : 0u) | (b > 0.f ? 0x10000u : 0u);
    asm("max.u16x2 %0, %1, %2;" : "=r"(rest) : "r"(*reinterpret_cast<const uint32_t*>(&r)), "r"(least));
    asm("max.u16x2 %0, %1, %2;" : "=r"(h) : "r"(h), "r"(least));
    return h;
  }
}
// Bytes 0 and 2 (or 1 and 3) of a word of int8 values as an exact f16 pair.
__device__ __forceinline__ uint32_t half_pair(uint32_t w, bool high) {
  const uint32_t biased = ((high ? w >> 8 : w) & 0x00FF00FFu) ^ 0x64806480u;   // 1152 + x
  const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&biased), __half2half2(__ushort_as_half(0x6480)));
  return *reinterpret_cast<const uint32_t*>(&v);
}

// KV8: int8 cache (MMAs in f16).  NT: column tiles of 8 query heads.
template <bool BF16, bool KV8, int D, int NT, int MODE>
struct Cfg {
  static constexpr int kRow = D * (KV8 ? 1 : 2);                  // bytes of a cache row
  static constexpr int kKeys = kRow <= 128 ? 32 : 16;             // keys of a warp's stage
  static constexpr int kStages = 2 * kKeys * kRow > 8192 ? 3 : 2;
  using Stages = Ring<kRow, KV8 ? 1 : 2, kKeys, kStages, MODE>;
  static constexpr int kHeads = 8 * NT;
  static constexpr int kRed = kWarps * kHeads * 64 * 4;           // merge buffer: 64 columns at a time
  static constexpr int kSmem = Stages::kBytes + kRed;
  // CTAs an SM, by registers (three leave 168 a thread) and shared memory.
  // More warps beat deeper rings: at head_dim 128 three CTAs of two stages
  // against two of three, bf16 189.8 -> 183.9 us on the batch of 64 (8192
  // rows at most), int8 190.6 -> 143.2 us.
  static constexpr int kCtas = D == 256 ? (KV8 ? 2 : 1) : NT == 2 ? 2 : 3;
};

// XF: scores under a softcap or an additive mask.  MODE: how the units are divided.
template <bool BF16, bool KV8, int D, int NT, bool XF, int MODE>
__global__ void __launch_bounds__(kThreads, Cfg<BF16, KV8, D, NT, MODE>::kCtas) paged_mma_kernel(const Work w) {
  using C = Cfg<BF16, KV8, D, NT, MODE>;
  using T = typename std::conditional<BF16, __nv_bfloat16, __half>::type;
  constexpr bool MBF = BF16 && !KV8;   // MMA type bf16
  using S = Scores<XF>;   // (masks come with XF)
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int st_key[kWarps][C::kStages];         // first key of a warp's stage
  __shared__ uint32_t st_vis[kWarps][C::kStages];    // which of its keys are visible
  __shared__ float red_m[kWarps][C::kHeads], red_l[kWarps][C::kHeads];
  const Problem& p = w.p;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, gid = lane >> 2, tig = lane & 3;
  const int units = p.G * w.n_hc;

  const int cta = blockIdx.x;
  int my;       // tiles of this CTA
  Cursor out;   // the tile being computed
  __shared__ Share share;   // (thread 0's, for its notes of cut units)
  if constexpr (MODE == kCluster) {
    const int unit = cta / w.cluster;
    out.b = unit / units;
    out.u = unit % units;
    out.load(w);
    int end;
    list_part(out.n, cta % w.cluster, w.cluster, out.tile, end);
    my = end - out.tile;
  } else if constexpr (MODE == kWhole) {
    my = 0;
    for (int64_t id = cta + (int64_t)lane * w.stride; id < (int64_t)p.B * units; id += 32 * (int64_t)w.stride)
      my += entry_tiles(w, (int)(id / units));
    my = __reduce_add_sync(kAll, my);
    if (my) out.at_unit(w, units, cta);
  } else {
    let_next_start();
    if (threadIdx.x == 0) w.cuts[cta].b = -1;
    Share s;
    my = find_share(w, units, cta, lane, s, out);
    if (threadIdx.x == 0) share = s;
  }
  if (MODE != kCluster && my == 0) {
    fill_entries<T>(w, cta);
    return;
  }
  typename C::Stages ring(w, out, units, smem, st_key[0], st_vis[0]);
#pragma unroll
  for (int s = 0; s < C::kStages - 1; ++s) {
    if (s < my) ring.issue(s, s + 1 < my);
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
        cs[j][0] = cs[j][1] = p.scale * S::kUnit;
      } else {
        // Channels 4t, 4t + 2 (then 4t + 1, 4t + 3) of a 16-channel block: the order in which the bytes arrive.
        float v[D / 16][4], top = 0.f;
        const float* ks = p.k_scale + (p.kv_per_channel ? g * D : 0);
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          const int d = 16 * c + 4 * tig;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            v[c][e] = hh < nh ? to_f32(row[d + e]) * __ldg(ks + (p.kv_per_channel ? d + e : 0)) : 0.f;
        }
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) top = fmaxf(top, fabsf(v[c][e]));
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
          uint32_t rest[2];
          qh[j][c][0] = pack_split<false>(v[c][0] * up, v[c][2] * up, rest[0]);
          qh[j][c][1] = pack_split<false>(v[c][1] * up, v[c][3] * up, rest[1]);
          ql[j][c][0] = rest[0];
          ql[j][c][1] = rest[1];
        }
        const float down = p.scale * S::kUnit * ldexpf(1.f, -ex);
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
  if constexpr (MODE != kCluster) fill_entries<T>(w, cta);   // (while the first copies are under way)
  const bool capped = XF && p.softcap > 0.f;
  const float cap_inv = capped ? 1.f / p.softcap : 0.f;
  // A row's reference is its maximum, less a lead where P is f16: there p = 2^(x - m_ref) is 2^11 at the maximum
  // the reference was taken from and at most 2^15 when it moves, and what f16 cannot hold (2^-25) is 2^-36 of the
  // row's largest probability: all keys together lose n 2^-36, under a quarter of f16's half step up to 2^23 rows.
  constexpr float kLead = (MBF ? 0.f : 11.f) * (XF ? kLn2 : 1.f);   // in the units of the scores
  constexpr float kRise = (MBF ? kSlack : 15.f) * (XF ? kLn2 : 1.f);
  // ldmatrix source rows and unit offsets of this lane (K: keys x channels; V transposed).
  const int lk_row = (lane & 7) + ((lane >> 3) & 1) * 8, lk_u = lane >> 4;
  const int lv_row = KV8 ? lk_row : (lane & 7) + (lane >> 4) * 8, lv_u = KV8 ? lane >> 4 : (lane >> 3) & 1;

  // Offsets of their first blocks; block c of a row sits at the offset XOR its unit number (times 16).
  const uint32_t lk = swz<C::Stages::kUnits>(lk_row, lk_u), lv = swz<C::Stages::kUnits>(lv_row, lv_u);

  const Part mine(smem, C::kHeads, D);   // (cluster: over the stages, once they are done)
  int first_tile = out.tile, frag = 0;   // where the current fragment began in its unit; its number in this share
  for (int i = 0; i < my; ++i) {
    const int s = i % C::kStages;
    if (i + C::kStages - 1 < my) ring.issue((i + C::kStages - 1) % C::kStages, i + C::kStages < my);
    copy_commit();
    copy_wait<C::kStages - 1>();
    __syncwarp();
    const uint32_t ks = ring.ring + s * C::Stages::kStage, vs = ks + C::kKeys * C::kRow;
    const uint32_t vis = st_vis[warp][s];
    constexpr int MB = C::kKeys / 16;   // 16-key blocks of a stage, in step: their chains of MMAs overlap
    float sc[MB][NT][4];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      // Two accumulators a column tile (even and odd channel blocks): half the chain of dependent MMAs.
      float sd[NT][4];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[mb][j][e] = sd[j][e] = 0.f;
      if constexpr (!KV8) {
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          uint32_t a[4];
          ldsm4(ks + (lk ^ (32 * c)) + 16 * mb * C::kRow, a);
#pragma unroll
          for (int j = 0; j < NT; ++j) mma<MBF>(c % 2 ? sd[j] : sc[mb][j], a, qh[j][c][0], qh[j][c][1]);
        }
      } else {
#pragma unroll
        for (int c = 0; c < D / 16; c += 2) {   // two 16-channel blocks: keys 0-7 and 8-15 of each
          uint32_t kw[4];
          ldsm4(ks + (lk ^ (16 * c)) + 16 * mb * C::kRow, kw);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint32_t a[4] = {half_pair(kw[2 * q], false), half_pair(kw[2 * q + 1], false),
                                   half_pair(kw[2 * q], true), half_pair(kw[2 * q + 1], true)};
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              mma<false>(q ? sd[j] : sc[mb][j], a, qh[j][c + q][0], qh[j][c + q][1]);
              mma<false>(q ? sd[j] : sc[mb][j], a, ql[j][c + q][0], ql[j][c + q][1]);
            }
          }
        }
      }
      // Scores.
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float x = (sc[mb][j][e] + sd[j][e]) * cs[j][e & 1];
          if (XF) {
            const int r = 16 * mb + gid + 8 * (e >> 1);
            if (capped) x = p.softcap * tanh_exp2(x * cap_inv);
            const int hh = 8 * j + 2 * tig + (e & 1);
            const int in_kv = (out.u % w.n_hc) * C::kHeads + hh;
            if (p.M && in_kv < p.qpg && ((vis >> r) & 1u))
              x += p.M[p.m.off + (int64_t)out.b * p.m.bs + (int64_t)(out.u / w.n_hc * p.qpg + in_kv) * p.m.hs +
                       st_key[warp][s] + r];
          }
          sc[mb][j][e] = x;
        }
    }
    if ((vis & C::Stages::kAllKeys) != C::Stages::kAllKeys) {   // hidden keys
#pragma unroll
      for (int mb = 0; mb < MB; ++mb)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!((vis >> (16 * mb + gid + 8 * (e >> 1))) & 1u)) sc[mb][j][e] = -INFINITY;
    }
    // The reference moves only when a score rises above it by more than kRise (by their difference, which is exact
    // where large masks leave no room for kRise beside a reference).
    float top[NT][2];
    bool rise = false;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        top[j][q] = fmaxf(sc[0][j][q], sc[0][j][q + 2]);
#pragma unroll
        for (int mb = 1; mb < MB; ++mb) top[j][q] = fmaxf(top[j][q], fmaxf(sc[mb][j][q], sc[mb][j][q + 2]));
        rise |= top[j][q] - m_ref[j][q] > kRise;
      }
    if (__any_sync(kAll, rise)) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int q = 0; q < 2; ++q) {   // a column's keys are spread over the lanes of a tig
          float mx = top[j][q];
          mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 4));
          mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 8));
          mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, 16));
          if (mx - m_ref[j][q] > kRise) {
            mx -= kLead;
            const float f = S::weight(m_ref[j][q], mx);
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
    uint32_t ph[MB][NT][2], pl[MB][NT][2];   // P^T: keys 2 tig, + 1 (then + 8) x head gid
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const float mu0 = m_ref[j][0] == -INFINITY ? 0.f : m_ref[j][0];
      const float mu1 = m_ref[j][1] == -INFINITY ? 0.f : m_ref[j][1];
#pragma unroll
      for (int mb = 0; mb < MB; ++mb) {
        float e[4];
        e[0] = S::weight(sc[mb][j][0], mu0);
        e[1] = S::weight(sc[mb][j][1], mu1);
        e[2] = S::weight(sc[mb][j][2], mu0);
        e[3] = S::weight(sc[mb][j][3], mu1);
        l[j][0] += e[0] + e[2];
        l[j][1] += e[1] + e[3];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t rest;
          ph[mb][j][q] = movtrans(KV8 ? pack_split<MBF>(e[2 * q], e[2 * q + 1], rest)
                                      : pack_above_zero<MBF>(e[2 * q], e[2 * q + 1], rest));
          pl[mb][j][q] = movtrans(rest);
        }
      }
    }
#pragma unroll
    for (int mb = 0; mb < MB; ++mb) {
      if constexpr (!KV8) {
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          uint32_t a[4];
          ldsm4t(vs + (lv ^ (32 * c)) + 16 * mb * C::kRow, a);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            mma<MBF>(o[c][j], a, ph[mb][j][0], ph[mb][j][1]);
            mma<MBF>(o[c][j], a, pl[mb][j][0], pl[mb][j][1]);
          }
        }
      } else {
#pragma unroll
        for (int c = 0; c < D / 16; c += 2) {
          uint32_t vw[4];   // (block c, keys 0-7), (c, 8-15), (c + 1, 0-7), (c + 1, 8-15)
          ldsm4t(vs + (lv ^ (16 * c)) + 16 * mb * C::kRow, vw);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint32_t a[4] = {half_pair(vw[2 * q], false), half_pair(vw[2 * q], true),
                                   half_pair(vw[2 * q + 1], false), half_pair(vw[2 * q + 1], true)};
#pragma unroll
            for (int j = 0; j < NT; ++j) {
              mma<false>(o[c + q][j], a, ph[mb][j][0], ph[mb][j][1]);
              mma<false>(o[c + q][j], a, pl[mb][j][0], pl[mb][j][1]);
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
      const int slot = frag == 0 ? 0 : 1, b = out.b;
      const int g = out.u / w.n_hc, h0 = g * p.qpg + (out.u % w.n_hc) * C::kHeads;
      const int nh = min(C::kHeads, (g + 1) * p.qpg - h0);
      if constexpr (MODE == kShares)
        if (unit_ends && !whole && threadIdx.x == 0) note_cut(w, share, cta, out, first_tile);
      if (i + 1 < my) {   // the next unit's queries arrive during the merge
        out.template next<MODE>(w, units);
        load_q();
      }
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
      float* red = reinterpret_cast<float*>(smem + C::Stages::kBytes);   // [kWarps][kHeads][64]
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
            const float f = S::weight(red_m[v][hh], mu);
            L = fmaf(f, red_l[v][hh], L);
            a = fmaf(f, red[(v * C::kHeads + hh) * 64 + d], a);
          }
          const int dd = 64 * part + d;
          if (KV8) a *= p.v_scale[p.kv_per_channel ? g * D + dd : 0];
          if constexpr (MODE == kCluster) mine.put(D, hh, dd, M, L, a);
          else put_row<T, XF>(w, whole, cta, slot, b, h0 + hh, hh, dd, M, L, a);
        }
        __syncthreads();
      }
      ++frag;
      first_tile = 0;
      reset();
    } else {
      ++out.tile;
    }
  }
  copy_wait<0>();
  if constexpr (MODE == kCluster) {
    const int g = out.u / w.n_hc, h0 = g * p.qpg + (out.u % w.n_hc) * C::kHeads;
    const int nh = min(C::kHeads, (g + 1) * p.qpg - h0);
    if (my == 0)
      for (int x = threadIdx.x; x < nh * D; x += kThreads) mine.put(D, x / D, x % D, -INFINITY, 0.f, 0.f);
    cluster_join<T, XF>(w, mine, out.b, h0, nh);
  }
}

// Plans the pass; with `launch` enqueues it.
template <bool BF16, bool KV8, int D, int NT>
int pass_cfg(Work& w, bool launch, cudaStream_t st) {
  using C = Cfg<BF16, KV8, D, NT, kShares>;   // (the same sizes for every mode)
  plan_work(w, C::Stages::kTile, C::kHeads, C::kCtas);
  if (!launch) return ATTN_OK;
  const bool xf = w.p.softcap > 0.f || w.p.M != nullptr;
  auto go = [&](auto mode) {
    constexpr int M = decltype(mode)::value;
    return xf ? launch_pass(paged_mma_kernel<BF16, KV8, D, NT, true, M>, w, C::kSmem, st)
              : launch_pass(paged_mma_kernel<BF16, KV8, D, NT, false, M>, w, C::kSmem, st);
  };
  return w.cluster  ? go(std::integral_constant<int, kCluster>())
         : w.stride ? go(std::integral_constant<int, kWhole>())
                    : go(std::integral_constant<int, kShares>());
}

// Two column tiles of heads a unit for more than eight heads a kv head (at
// head_dim 256 they would not fit the registers: the units then take eight
// heads each and read the cache rows again from L2).
template <bool BF16, bool KV8>
bool pick(Work& w, bool launch, cudaStream_t st, int* rc) {
  const bool two = w.p.qpg > 8;
  switch (w.p.D) {
    case 64: *rc = two ? pass_cfg<BF16, KV8, 64, 2>(w, launch, st) : pass_cfg<BF16, KV8, 64, 1>(w, launch, st); return true;
    case 128: *rc = two ? pass_cfg<BF16, KV8, 128, 2>(w, launch, st) : pass_cfg<BF16, KV8, 128, 1>(w, launch, st); return true;
    case 256: *rc = pass_cfg<BF16, KV8, 256, 1>(w, launch, st); return true;
    default: return false;
  }
}

}  // namespace paged
}  // namespace attn
