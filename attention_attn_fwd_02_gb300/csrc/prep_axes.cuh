// prep_axes.cuh -- the step before attention with positions on several axes
// (prep.cuh), for one element type (prep_axes_*.cu).
//
// The vector form is that of prep.cu: NT threads hold a head row, two 16-byte
// chunks of N elements each, so that a rotated pair lies in one thread; a warp
// loads kSteps groups of 32 / NT rows of one kind (Q, K or V) before it computes.
// What is its own:
//   - a thread's N pairs may lie on several axes.  Where every thread's lie on one (ONE:
//     stretches of a multiple of N pairs an axis), its angles are whole vectors
//     at that axis's position; else each is read by itself.  Positions, cache
//     rows and head rows are all under way before the first of them is used,
//     page numbers and angles come next;
//   - few heads leave a warp's rows empty when they are one token's: then (FLAT)
//     rows are taken token after token, each with the angles of its own token.
//
// What bounds it: HBM for long prompts, the chain of loads for one token a
// sequence, and instructions where the heads are narrow.  A video of 16384 tokens
// (32/8 heads, head_dim 128, 411 MB) takes 75.5 us, 5.4 TB/s; both forms of
// angles in one kernel (more registers) 82.  Two batches of 5003 tokens with
// 12/4 heads of 64 and axes in turn: 19.4 us, a token's own items 34.9, places in the
// tables in 64 bits 20.5, three CTAs an SM (spills) 22.5.
#pragma once

#include "prep.cuh"

namespace attn {
namespace {

constexpr int kSteps = 3;

// Division of n < 2^31 by a number that the host knows.
struct Div {
  uint32_t d, mul;
  int shift;
  explicit Div(uint32_t by) : d(by), mul(0), shift(0) {   // as Ext::div_mul (visible.cuh)
    while ((uint64_t)2 << shift < d) ++shift;
    if (d > 1) mul = (uint32_t)((((uint64_t)1 << (32 + shift)) + d - 1) / d);
  }
  __device__ __forceinline__ uint32_t of(uint32_t n) const { return d == 1 ? n : __umulhi(n, mul) >> shift; }
};

// Where the items of a launch are: FLAT, the items of Q and of K and V; else those of a token.
struct Items {
  Div seq, heads, kv_heads, per_token;
  uint32_t q, k, all;
};

// CTAs an SM: three leave 80 registers a thread, enough for whole vectors of one token's angles.
constexpr int ctas_per_sm(bool flat, bool one) { return !flat && one ? 3 : 2; }

template <typename T, int NT, bool KV8, bool INTER, bool FLAT, bool ONE>
__global__ void __launch_bounds__(256, ctas_per_sm(FLAT, ONE)) prep_axes_kernel(const Prep p, const Items it) {
  constexpr int N = Vec<T>::N, P = N / 2, kRows = 32 / NT, D = 2 * N * NT;
  const int lane = threadIdx.x % 32, t = lane % NT, sub = lane / NT;
  const int half = p.rot / 2;
  const bool turned = t * N < half;
  const int d0 = (turned && !INTER ? t : 2 * t) * N;
  const int d1 = turned && !INTER ? d0 + half : d0 + N;
  uint32_t mine[ONE ? 1 : N / 4] = {};   // the axes of the thread's N pairs, a byte each (ONE: their axis)
  if constexpr (ONE) {
    mine[0] = turned ? p.axis[t * N] : 0u;
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) mine[e / 4] |= (turned ? (uint32_t)p.axis[t * N + e] : 0u) << (8 * (e % 4));
  }
  constexpr int kPos = ONE ? 1 : ATTN_MAX_AXES;   // positions of a token that a thread holds
  for (uint32_t id = blockIdx.x * 8 + threadIdx.x / 32; id < it.all; id += gridDim.x * 8) {
    // The kind of the item's rows, and the token and head of this lane's row in each step (head < 0: there is none).
    uint32_t tok[FLAT ? kSteps : 1], part;
    int head[kSteps], kind;
    if constexpr (FLAT) {
      kind = id < it.q ? kQ : id < it.q + it.k ? kK : kV;
      const Div& by = kind == kQ ? it.heads : it.kv_heads;
      part = id - (kind == kQ ? 0 : kind == kK ? it.q : it.q + it.k);
      const uint32_t rows = (uint32_t)p.B * p.S * by.d;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        const uint32_t row = (part * kSteps + s) * kRows + sub;
        tok[s] = by.of(min(row, rows - 1));
        head[s] = row < rows ? (int)(row - tok[s] * by.d) : -1;
      }
    } else {
      tok[0] = it.per_token.of(id);
      part = id - tok[0] * it.per_token.d;
      kind = part < it.q ? kQ : part < it.q + it.k ? kK : kV;
      part -= kind == kQ ? 0 : kind == kK ? it.q : it.q + it.k;
      const int heads = kind == kQ ? p.H : p.G;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) {
        head[s] = (int)(part * kSteps + s) * kRows + sub;
        if (head[s] >= heads) head[s] = -1;
      }
    }
    constexpr int kToks = FLAT ? kSteps : 1;
    const Layout& li = kind == kQ ? p.q : kind == kK ? p.k : p.v;
    const Layout& lo = kind == kQ ? p.qo : kind == kK ? p.ko : p.vo;
    const T* in = static_cast<const T*>(kind == kQ ? p.Q : kind == kK ? p.K : p.V) + li.off;
    void* const out = kind == kQ ? p.QO : kind == kK ? p.KO : p.VO;
    int b[kToks], i[kToks], crow[kToks], pos[kToks][kPos];
    const bool rotates = kind != kV && turned;
#pragma unroll
    for (int s = 0; s < kToks; ++s) {
      b[s] = (int)it.seq.of(tok[s]);
      i[s] = (int)(tok[s] - b[s] * it.seq.d);
      crow[s] = kind != kQ && p.row ? __ldg(p.row + (int64_t)b[s] * p.row_bs + i[s]) : i[s];
#pragma unroll
      for (int a = 0; a < kPos; ++a) {
        const int axis = ONE ? (int)mine[0] : a;
        pos[s][a] = i[s];
        if (rotates && p.pos && axis < p.n_axes)
          pos[s][a] = __ldg(p.pos + axis * p.axis_stride + (int64_t)b[s] * p.pos_bs + i[s]);
      }
    }
    uint4 raw[kSteps][2];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      raw[s][0] = raw[s][1] = make_uint4(0, 0, 0, 0);
      if (head[s] >= 0) {
        const T* x = in + (int64_t)b[FLAT ? s : 0] * li.bs + (int64_t)head[s] * li.hs + (int64_t)i[FLAT ? s : 0] * li.rs;
        raw[s][0] = *reinterpret_cast<const uint4*>(x + d0);
        raw[s][1] = *reinterpret_cast<const uint4*>(x + d1);
      }
    }
    // Where the rows go (outer < 0: nowhere).
    int outer[kToks];
#pragma unroll
    for (int s = 0; s < kToks; ++s) {
      outer[s] = b[s];
      if (kind == kQ) continue;
      if ((uint32_t)crow[s] >= (uint32_t)p.rows_out) {
        outer[s] = -1;
      } else if (p.page_size) {
        const int at = crow[s] / p.page_size;
        const int32_t pg = __ldg(p.table + (int64_t)b[s] * p.table_stride + at);
        outer[s] = (uint32_t)pg < p.n_pages ? pg : -1;
        crow[s] -= at * p.page_size;
      }
    }
    float2 cs[P], sn[P];
    auto angles = [&](int s) {
      if (!rotates) {
#pragma unroll
        for (int e = 0; e < P; ++e) {
          cs[e] = make_float2(1.f, 1.f);
          sn[e] = make_float2(0.f, 0.f);
        }
      } else if constexpr (ONE) {
        const int at = min(max(pos[s][0], 0), p.max_pos - 1) * half + t * N;
#pragma unroll
        for (int e = 0; e < P; e += 2) {
          const float4 c4 = __ldg(reinterpret_cast<const float4*>(p.cos + at + 2 * e));
          const float4 s4 = __ldg(reinterpret_cast<const float4*>(p.sin + at + 2 * e));
          cs[e] = make_float2(c4.x, c4.y);
          cs[e + 1] = make_float2(c4.z, c4.w);
          sn[e] = make_float2(s4.x, s4.y);
          sn[e + 1] = make_float2(s4.z, s4.w);
        }
      } else {
        int at[kPos];   // the token's rows of the tables, from the thread's first pair on
#pragma unroll
        for (int a = 0; a < kPos; ++a) at[a] = min(max(pos[s][a], 0), p.max_pos - 1) * half + t * N;
#pragma unroll
        for (int e = 0; e < N; ++e) {   // each pair at its own axis's position
          const uint32_t a = mine[e / 4] >> (8 * (e % 4)) & 255u;
          const int x = (a & 2u ? (a & 1u ? at[3] : at[2]) : a & 1u ? at[1] : at[0]) + e;
          const float c = __ldg(p.cos + x), y = __ldg(p.sin + x);
          if (e % 2) {
            cs[e / 2].y = c;
            sn[e / 2].y = y;
          } else {
            cs[e / 2].x = c;
            sn[e / 2].x = y;
          }
        }
      }
    };
    if constexpr (!FLAT) angles(0);
    const T* w = kind == kV ? nullptr : static_cast<const T*>(kind == kQ ? p.qw : p.kw);
    const bool weighted = p.norm && w;
    uint4 rw[2];   // the weights, as stored
    if (weighted) {
      rw[0] = __ldg(reinterpret_cast<const uint4*>(w + d0));
      rw[1] = __ldg(reinterpret_cast<const uint4*>(w + d1));
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      if constexpr (FLAT) angles(s);
      const int z = FLAT ? s : 0;
      const int64_t o = lo.off + (int64_t)outer[z] * lo.bs + (int64_t)head[s] * lo.hs + (int64_t)crow[z] * lo.rs;
      const bool writes = head[s] >= 0 && outer[z] >= 0;
      if (kind == kV && !KV8) {
        if (writes) {
          T* y = static_cast<T*>(out) + o;
          *reinterpret_cast<uint4*>(y + d0) = raw[s][0];
          *reinterpret_cast<uint4*>(y + d1) = raw[s][1];
        }
        continue;
      }
      float2 x0[P], x1[P];
      Vec<T>::get(raw[s][0], x0);
      Vec<T>::get(raw[s][1], x1);
      if (kind != kV) {
        if (p.norm) {
          float2 q = mul2(x0[0], x0[0]);
#pragma unroll
          for (int e = 1; e < P; ++e) q = fma2(x0[e], x0[e], q);
#pragma unroll
          for (int e = 0; e < P; ++e) q = fma2(x1[e], x1[e], q);
          float ss = q.x + q.y;
#pragma unroll
          for (int m = NT / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
          const float rs = rsqrtf(fmaf(ss, 1.f / D, p.eps));
          const float2 r2 = make_float2(rs, rs);
#pragma unroll
          for (int e = 0; e < P; ++e) {
            x0[e] = mul2(x0[e], r2);
            x1[e] = mul2(x1[e], r2);
          }
          if (weighted) {
            float2 w0[P], w1[P];
            Vec<T>::get(rw[0], w0);
            Vec<T>::get(rw[1], w1);
#pragma unroll
            for (int e = 0; e < P; ++e) {
              x0[e] = mul2(x0[e], w0[e]);
              x1[e] = mul2(x1[e], w1[e]);
            }
          }
        }
        if (turned) {
          if constexpr (INTER) {   // pairs (2j, 2j + 1) in the thread's 2 N elements: (a, c) cos + (-c, a) sin
#pragma unroll
            for (int e = 0; e < P; ++e) {
              const float ca = e % 2 ? cs[e / 2].y : cs[e / 2].x, sa = e % 2 ? sn[e / 2].y : sn[e / 2].x;
              const float cb = e % 2 ? cs[(P + e) / 2].y : cs[(P + e) / 2].x;
              const float sb = e % 2 ? sn[(P + e) / 2].y : sn[(P + e) / 2].x;
              x0[e] = fma2(make_float2(-x0[e].y, x0[e].x), make_float2(sa, sa), mul2(x0[e], make_float2(ca, ca)));
              x1[e] = fma2(make_float2(-x1[e].y, x1[e].x), make_float2(sb, sb), mul2(x1[e], make_float2(cb, cb)));
            }
          } else {
#pragma unroll
            for (int e = 0; e < P; ++e) {
              const float2 a = x0[e], c = x1[e];
              x0[e] = fma2(make_float2(-c.x, -c.y), sn[e], mul2(a, cs[e]));
              x1[e] = fma2(a, sn[e], mul2(c, cs[e]));
            }
          }
        }
      }
      if (!writes) continue;
      if (KV8 && kind != kQ) {
        const float* sc = (kind == kK ? p.k_scale : p.v_scale) + (p.per_channel ? head[s] * D : 0);
        int8_t* y = static_cast<int8_t*>(out) + o;
        __align__(8) int8_t c0[N], c1[N];
#pragma unroll
        for (int e = 0; e < N; ++e) {
          c0[e] = code_of(e % 2 ? x0[e / 2].y : x0[e / 2].x, sc[p.per_channel ? d0 + e : 0]);
          c1[e] = code_of(e % 2 ? x1[e / 2].y : x1[e / 2].x, sc[p.per_channel ? d1 + e : 0]);
        }
        if constexpr (N == 8) {
          *reinterpret_cast<uint2*>(y + d0) = *reinterpret_cast<const uint2*>(c0);
          *reinterpret_cast<uint2*>(y + d1) = *reinterpret_cast<const uint2*>(c1);
        } else {
          *reinterpret_cast<uint32_t*>(y + d0) = *reinterpret_cast<const uint32_t*>(c0);
          *reinterpret_cast<uint32_t*>(y + d1) = *reinterpret_cast<const uint32_t*>(c1);
        }
      } else {
        T* y = static_cast<T*>(out) + o;
        *reinterpret_cast<uint4*>(y + d0) = Vec<T>::put(x0);
        *reinterpret_cast<uint4*>(y + d1) = Vec<T>::put(x1);
      }
    }
  }
}

template <typename T, int NT, bool FLAT, bool ONE>
cudaError_t launch_items(const Prep& p, const Items& it, bool kv8, cudaStream_t st) {
  const int64_t blocks = ((int64_t)it.all + 7) / 8, most = 152 * ctas_per_sm(FLAT, ONE);
  const unsigned grid = (unsigned)(blocks < most ? blocks : most);
  if (p.inter) {
    if (kv8) prep_axes_kernel<T, NT, true, true, FLAT, ONE><<<grid, 256, 0, st>>>(p, it);
    else prep_axes_kernel<T, NT, false, true, FLAT, ONE><<<grid, 256, 0, st>>>(p, it);
  } else {
    if (kv8) prep_axes_kernel<T, NT, true, false, FLAT, ONE><<<grid, 256, 0, st>>>(p, it);
    else prep_axes_kernel<T, NT, false, false, FLAT, ONE><<<grid, 256, 0, st>>>(p, it);
  }
  return cudaGetLastError();
}

template <typename T, int NT>
cudaError_t launch_axes(const Prep& p, bool kv8, cudaStream_t st) {
  constexpr int kPer = kSteps * (32 / NT);   // rows of an item
  auto up = [](int64_t n) { return (uint32_t)((n + kPer - 1) / kPer); };
  Items it{Div(p.S), Div(p.H), Div(p.G), Div(1), up(p.H), up(p.G), 0};
  const int64_t tokens = (int64_t)p.B * p.S, of_token = it.q + 2 * it.k;
  bool one = true;
  for (int j = 0; j < p.rot / 2; ++j) one = one && p.axis[j] == p.axis[j / Vec<T>::N * Vec<T>::N];
  // A token's own items, where its rows fill 7 tenths of them.
  if (10 * (p.H + 2 * p.G) >= 7 * of_token * kPer) {
    it.per_token = Div((uint32_t)of_token);
    it.all = (uint32_t)(tokens * of_token);
    return one ? launch_items<T, NT, false, true>(p, it, kv8, st) : launch_items<T, NT, false, false>(p, it, kv8, st);
  }
  it.q = up(tokens * p.H);
  it.k = up(tokens * p.G);
  it.all = it.q + 2 * it.k;
  return one ? launch_items<T, NT, true, true>(p, it, kv8, st) : launch_items<T, NT, true, false>(p, it, kv8, st);
}

template <typename T>
cudaError_t launch_type(const Prep& p, bool kv8, cudaStream_t st) {
  // (places in the tables are 32-bit numbers)
  if (!takes_vec<T>(p, kv8) || (int64_t)p.max_pos * (p.rot / 2) > 0x7fffffff) return launch_rows<T, true>(p, kv8, st);
  switch (p.D / (2 * Vec<T>::N)) {
    case 2: return launch_axes<T, 2>(p, kv8, st);
    case 4: return launch_axes<T, 4>(p, kv8, st);
    case 8: return launch_axes<T, 8>(p, kv8, st);
    case 16: return launch_axes<T, 16>(p, kv8, st);
    default:
      if constexpr (Vec<T>::N == 4) return launch_axes<T, 32>(p, kv8, st);   // float32 at head_dim 256
      else return cudaErrorInvalidValue;
  }
}

}  // namespace

}  // namespace attn
