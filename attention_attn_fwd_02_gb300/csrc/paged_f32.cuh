// paged_f32.cuh -- decode over a paged float32 cache at head_dim 64, 128 or 256.
//
// The same work, shares, rings and joins as the tensor-core pass (paged.cuh);
// the products stay on the CUDA cores, in float32.  A unit has up to 4 or 8
// query heads.  In a stage of 4 KB of keys, 32 / KEYS lanes share a key: each
// takes 32 of its elements against all heads (q from shared memory, one
// broadcast address a lane group) and a butterfly over the group completes the
// scores.  The probabilities pass through shared memory, and every lane sums
// p V for its own 4 (or 8) elements of all heads.
//
// What bounds it: HBM.  At 6 TB/s an SM takes an 8 KB stage every 200 ns; its
// products are 8 x 1024 FMAs (of 128 a cycle) and about 100 shared-memory
// wavefronts at 4 heads, a third of that time.
#pragma once

#include <type_traits>

#include "paged.cuh"

namespace attn {
namespace paged {
namespace {

template <int D, int NH, int MODE>
struct CfgF32 {
  static constexpr int kKeys = 1024 / D;            // keys of a warp's stage: 4 KB of K, 4 KB of V
  static constexpr int kLanes = 32 / kKeys;         // lanes of a key
  static constexpr int kStages = 2;
  using Stages = Ring<D * 4, 4, kKeys, kStages, MODE>;
  static constexpr int kQ = NH * D * 4;             // the unit's queries
  static constexpr int kP = kWarps * kKeys * NH * 4;
  static constexpr int kRed = kWarps * 4 * D * 4;   // merge buffer: 4 heads at a time
  static constexpr int kSmem = Stages::kBytes + kQ + kP + kRed;
  static constexpr int kCtas = kSmem <= 74 * 1024 ? 3 : 2;
};

// XF: scores under a softcap or an additive mask.  OWN: rows are kept for a merge (OwnPart).
template <int D, int NH, bool XF, int MODE, bool OWN>
__global__ void __launch_bounds__(kThreads, CfgF32<D, NH, MODE>::kCtas) paged_f32_kernel(const Work w) {
  using C = CfgF32<D, NH, MODE>;
  constexpr int U = C::Stages::kUnits;              // 16-byte units of a row
  constexpr int KEYS = C::kKeys, LPK = C::kLanes;
  constexpr int VU = U >= 32 ? U / 32 : 1;          // units of a row a lane sums
  constexpr int GROUPS = U >= 32 ? 1 : 32 / U;      // keys side by side in the V sums
  extern __shared__ __align__(128) uint8_t smem[];
  float* q_s = reinterpret_cast<float*>(smem + C::Stages::kBytes);
  float* p_s = q_s + NH * D;
  float* red = p_s + kWarps * KEYS * NH;
  __shared__ int st_key[kWarps][C::kStages];
  __shared__ uint32_t st_vis[kWarps][C::kStages];
  __shared__ float red_m[kWarps][NH], red_l[kWarps][NH];
  const Problem& p = w.p;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
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
    if (!OWN && threadIdx.x == 0) w.cuts[cta].b = -1;
    Share s;
    my = find_share(w, units, cta, lane, s, out);
    if (threadIdx.x == 0) share = s;
  }
  if (MODE != kCluster && my == 0) {
    fill_entries<float, OWN>(w, cta);
    if constexpr (OWN) wait_for_previous();
    return;
  }
  typename C::Stages ring(w, out, units, smem, st_key[0], st_vis[0]);
#pragma unroll
  for (int s = 0; s < C::kStages - 1; ++s) {
    if (s < my) ring.issue(s, s + 1 < my);
    copy_commit();
  }
  using S = Scores<XF>;   // (masks come with XF)
  const bool capped = XF && p.softcap > 0.f;
  const float qscale = p.scale * S::kUnit;
  constexpr float kRise = XF ? kSlack * kLn2 : kSlack;   // in the units of the scores
  auto load_q = [&]() {
    const int g = out.u / w.n_hc, c0 = out.u % w.n_hc * NH;
    for (int x = threadIdx.x; x < NH * D; x += kThreads) {
      const int hh = x / D, d = x % D;
      q_s[x] = c0 + hh < p.qpg ? static_cast<const float*>(p.Q)[p.q.off + (int64_t)out.b * p.q.bs +
                                                                (int64_t)(g * p.qpg + c0 + hh) * p.q.hs + d]
                               : 0.f;
    }
    __syncthreads();
  };
  load_q();
  float o[NH][VU][4], m_ref[NH], l[NH];
  auto reset = [&]() {
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      m_ref[h] = -INFINITY;
      l[h] = 0.f;
#pragma unroll
      for (int v = 0; v < VU; ++v)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[h][v][e] = 0.f;
    }
  };
  reset();
  if constexpr (MODE != kCluster) fill_entries<float, OWN>(w, cta);   // (while the first copies are under way)
  const int key = lane % KEYS, part = lane / KEYS;   // this lane's key of a stage and its share of the elements
  float* my_p = p_s + warp * KEYS * NH;

  const Part mine(smem, NH, D);   // (cluster: over the stages, once they are done)
  int first_tile = out.tile, frag = 0;
  for (int i = 0; i < my; ++i) {
    const int s = i % C::kStages;
    if (i + C::kStages - 1 < my) ring.issue((i + C::kStages - 1) % C::kStages, i + C::kStages < my);
    copy_commit();
    copy_wait<C::kStages - 1>();
    __syncwarp();
    const uint8_t* ks = smem + (warp * C::kStages + s) * C::Stages::kStage;
    const uint8_t* vs = ks + KEYS * D * 4;
    const uint32_t vis = st_vis[warp][s];
    if ((vis & C::Stages::kAllKeys) != 0) {
      float sc[NH];
#pragma unroll
      for (int h = 0; h < NH; ++h) sc[h] = 0.f;
#pragma unroll
      for (int t = 0; t < U / LPK; ++t) {
        const float4 k4 = *reinterpret_cast<const float4*>(ks + swz<U>(key, t * LPK + part));
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          const float4 q4 = *reinterpret_cast<const float4*>(q_s + h * D + (t * LPK + part) * 4);
          sc[h] = fmaf(k4.x, q4.x, fmaf(k4.y, q4.y, fmaf(k4.z, q4.z, fmaf(k4.w, q4.w, sc[h]))));
        }
      }
      const bool seen = (vis >> key) & 1u;
      bool rise = false;
#pragma unroll
      for (int h = 0; h < NH; ++h) {
#pragma unroll
        for (int x = KEYS; x < 32; x <<= 1) sc[h] += __shfl_xor_sync(kAll, sc[h], x);
        float v = sc[h] * qscale;
        if (XF) {
          if (capped) v = p.softcap * tanhf(v / p.softcap);
          const int in_kv = out.u % w.n_hc * NH + h;
          if (p.M && seen && in_kv < p.qpg)
            v += p.M[p.m.off + (int64_t)out.b * p.m.bs + (int64_t)(out.u / w.n_hc * p.qpg + in_kv) * p.m.hs +
                     st_key[warp][s] + key];
        }
        sc[h] = seen ? v : -INFINITY;
        rise |= sc[h] - m_ref[h] > kRise;
      }
      if (__any_sync(kAll, rise)) {
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          float mx = sc[h];
#pragma unroll
          for (int x = 1; x < KEYS; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kAll, mx, x));
          if (mx - m_ref[h] > kRise) {
            const float f = S::weight(m_ref[h], mx);
            l[h] *= f;
#pragma unroll
            for (int v = 0; v < VU; ++v)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[h][v][e] *= f;
            m_ref[h] = mx;
          }
        }
      }
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        sc[h] = S::weight(sc[h], m_ref[h] == -INFINITY ? 0.f : m_ref[h]);
        l[h] += sc[h];   // (the lanes of a key hold the same value: one of them is counted at the end)
      }
      if (part == 0) {
#pragma unroll
        for (int h = 0; h < NH; h += 4)
          *reinterpret_cast<float4*>(my_p + key * NH + h) = make_float4(sc[h], sc[h + 1], sc[h + 2], sc[h + 3]);
      }
      __syncwarp();
#pragma unroll
      for (int kk = 0; kk < KEYS / GROUPS; ++kk) {
        const int r = GROUPS == 1 ? kk : kk * GROUPS + lane / U;
        float4 v4[VU];
#pragma unroll
        for (int v = 0; v < VU; ++v)
          v4[v] = *reinterpret_cast<const float4*>(vs + swz<U>(r, (U >= 32 ? v * 32 : 0) + lane % (U < 32 ? U : 32)));
#pragma unroll
        for (int h = 0; h < NH; h += 4) {
          const float4 p4 = *reinterpret_cast<const float4*>(my_p + r * NH + h);
          const float pv[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
          for (int z = 0; z < 4; ++z)
#pragma unroll
            for (int v = 0; v < VU; ++v) {
              o[h + z][v][0] = fmaf(pv[z], v4[v].x, o[h + z][v][0]);
              o[h + z][v][1] = fmaf(pv[z], v4[v].y, o[h + z][v][1]);
              o[h + z][v][2] = fmaf(pv[z], v4[v].z, o[h + z][v][2]);
              o[h + z][v][3] = fmaf(pv[z], v4[v].w, o[h + z][v][3]);
            }
        }
      }
    }
    __syncwarp();   // the stage and the probabilities are free

    const bool unit_ends = out.tile + 1 == out.n;
    if (unit_ends || i + 1 == my) {
      // The fragment ends: the four warps' results, merged in warp order, four heads at a time.
      const bool whole = unit_ends && first_tile == 0;
      const int slot = frag == 0 ? 0 : 1;
      const int g = out.u / w.n_hc, h0 = g * p.qpg + out.u % w.n_hc * NH;
      const int nh = min(NH, (g + 1) * p.qpg - h0);
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        float x = part == 0 ? l[h] : 0.f;
#pragma unroll
        for (int y = 1; y < 32; y <<= 1) x += __shfl_xor_sync(kAll, x, y);
        if (lane == 0) {
          red_m[warp][h] = m_ref[h];
          red_l[warp][h] = x;
        }
      }
#pragma unroll
      for (int hb = 0; hb < NH; hb += 4) {
#pragma unroll
        for (int z = 0; z < 4; ++z)
#pragma unroll
          for (int v = 0; v < VU; ++v) {
            float4 x = make_float4(o[hb + z][v][0], o[hb + z][v][1], o[hb + z][v][2], o[hb + z][v][3]);
#pragma unroll
            for (int y = U; y < 32; y <<= 1) {   // keys that were summed side by side
              x.x += __shfl_xor_sync(kAll, x.x, y);
              x.y += __shfl_xor_sync(kAll, x.y, y);
              x.z += __shfl_xor_sync(kAll, x.z, y);
              x.w += __shfl_xor_sync(kAll, x.w, y);
            }
            if (lane < U) *reinterpret_cast<float4*>(red + (warp * 4 + z) * D + (v * 32 + lane) * 4) = x;
          }
        __syncthreads();
        for (int x = threadIdx.x; x < min(4, nh - hb) * D; x += kThreads) {
          const int z = x / D, d = x % D;
          float M = -INFINITY;
#pragma unroll
          for (int v = 0; v < kWarps; ++v) M = fmaxf(M, red_m[v][hb + z]);
          const float mu = M == -INFINITY ? 0.f : M;
          float L = 0.f, a = 0.f;
#pragma unroll
          for (int v = 0; v < kWarps; ++v) {
            const float f = S::weight(red_m[v][hb + z], mu);
            L = fmaf(f, red_l[v][hb + z], L);
            a = fmaf(f, red[(v * 4 + z) * D + d], a);
          }
          if constexpr (MODE == kCluster) mine.put(D, hb + z, d, M, L, a);
          else put_row<float, XF, OWN>(w, whole, cta, slot, out.b, h0 + hb + z, hb + z, d, M, L, a);
        }
        __syncthreads();
      }
      if constexpr (MODE == kShares)
        if (unit_ends && threadIdx.x == 0) {
          if (!whole) note_cut<OWN>(w, share, cta, out, first_tile);
          else if (OWN) note_kept(w, out.b, out.u);
        }
      ++frag;
    }
    if (i + 1 < my) {
      out.template next<MODE>(w, units);
      if (unit_ends) {
        first_tile = 0;
        load_q();
        reset();
      }
    }
  }
  copy_wait<0>();
  if constexpr (MODE == kCluster) {
    const int g = out.u / w.n_hc, h0 = g * p.qpg + out.u % w.n_hc * NH;
    const int nh = min(NH, (g + 1) * p.qpg - h0);
    if (my == 0)
      for (int x = threadIdx.x; x < nh * D; x += kThreads) mine.put(D, x / D, x % D, -INFINITY, 0.f, 0.f);
    cluster_join<float, XF, OWN>(w, mine, out.b, h0, nh);
  }
  if constexpr (OWN) wait_for_previous();
}

template <int D, int NH, bool OWN>
int enqueue_f32(const Work& w, cudaStream_t st) {
  using C = CfgF32<D, NH, kShares>;   // (the same sizes for every mode)
  const bool xf = w.p.softcap > 0.f || w.p.M != nullptr;
  auto go = [&](auto mode) {
    constexpr int M = decltype(mode)::value;
    return xf ? launch_pass(paged_f32_kernel<D, NH, true, M, OWN>, w, C::kSmem, st)
              : launch_pass(paged_f32_kernel<D, NH, false, M, OWN>, w, C::kSmem, st);
  };
  return w.cluster  ? go(std::integral_constant<int, kCluster>())
         : w.stride ? go(std::integral_constant<int, kWhole>())
                    : go(std::integral_constant<int, kShares>());
}

}  // namespace

// The pass over own keys behind a shared prefix (paged_own_f32.cu).
template <int D, int NH>
int enqueue_own_f32(const Work& w, cudaStream_t st);

}  // namespace paged
}  // namespace attn
