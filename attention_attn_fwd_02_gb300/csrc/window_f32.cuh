// window_f32.cuh -- float32 attention under a sliding window with first keys
// (window_f32.cu), or over a shared prefix and own keys in a paged cache
// (shared_f32.cu), on the CUDA cores at head_dim 32, 64, 128 or 256.
//
// What it computes: O = softmax(scale Q K^T + mask) V and the LSE over each
// row's visible keys (visible.cuh), with the online normaliser of "Attention"
// (recursiveai.org OneGPU docs), opening paragraph, all in float32.
//
// A CTA of 128 threads takes 16 TM rows of one (batch entry, kv head): rows
// are (query, head of the group) pairs, so the group's heads share the tiles.
// It walks its tile list (visible.cuh) 32 keys at a time.  Both products are
// register tiles: thread (ty, tx) of 16 x 8 holds TM rows (ty + 16 r) against
// 4 keys (tx + 8 c) of S, and the same rows against D / 8 columns of O, so a
// shared-memory load feeds 8 FMAs or more; K and Q rows are padded by 16 bytes
// and P is stored by key with a thread's rows side by side, which keeps every
// load free of bank conflicts.  K's next tile is copied (cp.async) while the
// softmax and P V run, V's while the next S runs.
//
// In a paged cache the first warp finds the pages of the next tile's rows while
// the CTA multiplies the current one.
//
// What bounds it: FMA issue (4 head_dim FLOPs a visible pair against 152 x 128
// lanes), for small problems the chain of one CTA's tiles.
#pragma once

#include <limits.h>

#include "paged.cuh"   // cp.async helpers
#include "tma.h"

namespace attn {
namespace {

using paged::copy16;
using paged::copy_commit;
using paged::copy_wait;
using paged::smem_u32;

constexpr int kThreads = 128;
constexpr int BN = 32;
using S = Scores<true>;   // (one instance with and without a mask: a product more for each D of a score)

// acc + a b for both halves, in one instruction (rounded as two).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 acc) {
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%0, %1};\n\t"
      "fma.rn.f32x2 z, x, y, z;\n\tmov.b64 {%0, %1}, z;\n\t}"
      : "+f"(acc.x), "+f"(acc.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return acc;
}

template <int D, int TM>
struct Cfg {
  static constexpr int BM = 16 * TM;
  static constexpr int kPitch = D + 4;                                    // floats
  static constexpr int kPp = BM + 4;                                      // of P, by key
  static constexpr int kSmem = ((BM + BN) * kPitch + BN * D + BN * kPp) * 4;
  static constexpr int kCtas = kSmem <= 74 * 1024 ? 3 : 2;
};

// KIND: contiguous keys, an entry's prefix and own keys in pages, or the prefix alone for the packed rows of all
// entries.  stride: partial results of a row.
enum { kPlain = 0, kPaged = 1, kPacked = 2 };

template <int D, int TM, int KIND>
__global__ void __launch_bounds__(kThreads, Cfg<D, TM>::kCtas)
    window_f32_kernel(const Problem p, const Ext x, const Split sp, const int64_t row_blocks, const int stride) {
  constexpr bool PAGED = KIND != kPlain, PACKED = KIND == kPacked;
  const int first = x.first;
  using C = Cfg<D, TM>;
  constexpr int BM = C::BM, PITCH = C::kPitch, NC = D / 32;
  extern __shared__ __align__(16) float smem[];
  float* q_s = smem;
  float* k_s = q_s + BM * PITCH;
  float* v_s = k_s + BN * PITCH;
  float* p_s = v_s + BN * D;
  __shared__ Vis row_v[BM];
  __shared__ int row_q[BM], row_h[BM], s_f[2], s_w[2];
  __shared__ int row_b[PACKED ? BM : 1];   // PACKED: each row's entry
  // PAGED: where the rows of a tile (even, odd) are in K and V, and which of them have a page.
  __shared__ int64_t at_k[2][BN], at_v[2][BN];
  __shared__ uint32_t paged_keys[2];
  const int tid = threadIdx.x, tx = tid % 8, ty = tid / 8;

  int64_t blk = blockIdx.x;
  const int split = (int)(blk % sp.n_splits);
  blk /= sp.n_splits;
  const int64_t rb = blk % row_blocks;
  blk /= row_blocks;
  const int g = (int)(blk % p.G), b = PACKED ? 0 : (int)(blk / p.G);
  // Query and head of each row (-1: behind the last).
  auto query_of = [&](int row) { return row_q[row]; };
  auto head_of = [&](int row) { return row_h[row]; };
  auto entry_of = [&](int row) { return PACKED ? row_b[PACKED ? row : 0] : b; };
  auto valid = [&](int row) { return row_q[row] >= 0; };

  if (tid == 0) {
    s_f[0] = s_w[0] = INT_MAX;
    s_f[1] = s_w[1] = -1;
  }
  __syncthreads();
  if (tid < BM) {
    const int64_t r = rb * BM + tid;
    int i = (int)(r / p.qpg);
    row_h[tid] = g * p.qpg + (int)(r - (int64_t)i * p.qpg);
    bool here = i < p.Sq;
    if constexpr (PACKED) {
      const int e = i / p.Sq;
      i -= e * p.Sq;
      here = e < p.B;
      row_b[tid] = here ? e : 0;
    }
    row_q[tid] = here ? i : -1;
    const Vis v = !here ? Vis{0, 0, 0, 0} : PACKED ? Vis{0, 0, 0, p.prefix} : row_vis(p, first, b, i);
    row_v[tid] = v;
    if (v.fe > v.lo) {
      atomicMin(&s_f[0], v.lo);
      atomicMax(&s_f[1], v.fe);
    }
    if (v.hi > v.wl) {
      atomicMin(&s_w[0], v.wl);
      atomicMax(&s_w[1], v.hi);
    }
  }
  __syncthreads();
  const Vis uv = vis_union(s_f[0], s_f[1], s_w[0], s_w[1]);
  const TileList tl = tile_list(uv, BN);
  int t0 = 0, t1 = tl.n;
  if (sp.part_o) list_part(tl.n, split, sp.n_splits, t0, t1);

  const float* Q = static_cast<const float*>(p.Q) + p.q.off;
  const float* K = static_cast<const float*>(p.K) + p.k.off + (PAGED ? 0 : (int64_t)b * p.k.bs) + (int64_t)g * p.k.hs;
  const float* V = static_cast<const float*>(p.V) + p.v.off + (PAGED ? 0 : (int64_t)b * p.v.bs) + (int64_t)g * p.v.hs;
  // The page of row `tid` of tile ti, and the row in it (tid < BN).
  auto find = [&](int ti, int& row) {
    const int k = tl.tile(ti) * BN + tid;
    return visible(uv, k) ? page_of(x, b, k, row) : -1;
  };
  auto note = [&](int ti, int page, int row) {
    at_k[ti & 1][tid] = page < 0 ? 0 : (int64_t)page * p.k.bs + (int64_t)row * p.k.rs;
    at_v[ti & 1][tid] = page < 0 ? 0 : (int64_t)page * p.v.bs + (int64_t)row * p.v.rs;
    const uint32_t have = __ballot_sync(0xffffffffu, page >= 0);
    if (tid == 0) paged_keys[ti & 1] = have;
  };
  if (PAGED && t0 < t1) {
    if (tid < BN) {
      int row = 0;
      const int page = find(t0, row);
      note(t0, page, row);
    }
    __syncthreads();
  }
  constexpr int kChunks = D / 4;   // 16-byte chunks of a row
  for (int c = tid; c < BM * kChunks; c += kThreads) {
    const int row = c / kChunks, d = c % kChunks * 4;
    const bool ok = valid(row);
    copy16(smem_u32(q_s + row * PITCH + d),
           ok ? Q + (int64_t)entry_of(row) * p.q.bs + (int64_t)head_of(row) * p.q.hs + (int64_t)query_of(row) * p.q.rs + d
              : Q,
           ok ? 16 : 0);
  }
  // Rows no row of the CTA sees arrive as zeros and are not read.
  auto load = [&](float* dst, int pitch, const float* src, int64_t rs, const int64_t (&at)[2][BN], int ti) {
    const int k0 = tl.tile(ti) * BN;
    for (int c = tid; c < BN * kChunks; c += kThreads) {
      const int row = c / kChunks, d = c % kChunks * 4;
      const bool ok = PAGED ? (paged_keys[ti & 1] >> row) & 1u : visible(uv, k0 + row);
      const int64_t from = PAGED ? at[ti & 1][row] : (int64_t)(k0 + row) * rs;
      copy16(smem_u32(dst + row * pitch + d), ok ? src + from + d : src, ok ? 16 : 0);
    }
  };
  if (t0 < t1) load(k_s, PITCH, K, p.k.rs, at_k, t0);
  copy_commit();
  if (t0 < t1) load(v_s, D, V, p.v.rs, at_v, t0);
  copy_commit();

  float o[TM][NC][4], m[TM], l[TM];
#pragma unroll
  for (int r = 0; r < TM; ++r) {
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int c = 0; c < NC; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[r][c][e] = 0.f;
  }
  for (int ti = t0; ti < t1; ++ti) {
    const int k0 = tl.tile(ti) * BN;
    copy_wait<1>();
    __syncthreads();
    int next_page = -1, next_row = 0;
    if (PAGED && tid < BN && ti + 1 < t1) next_page = find(ti + 1, next_row);
    float s[TM][4];
#pragma unroll
    for (int r = 0; r < TM; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) s[r][c] = 0.f;
#pragma unroll 8
    for (int d = 0; d < D; d += 4) {
      float4 a[TM], k4[4];
#pragma unroll
      for (int r = 0; r < TM; ++r) a[r] = *reinterpret_cast<const float4*>(q_s + (ty + 16 * r) * PITCH + d);
#pragma unroll
      for (int c = 0; c < 4; ++c) k4[c] = *reinterpret_cast<const float4*>(k_s + (tx + 8 * c) * PITCH + d);
#pragma unroll
      for (int r = 0; r < TM; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          s[r][c] = fmaf(a[r].x, k4[c].x,
                         fmaf(a[r].y, k4[c].y, fmaf(a[r].z, k4[c].z, fmaf(a[r].w, k4[c].w, s[r][c]))));
    }
    if (PAGED && tid < BN && ti + 1 < t1) note(ti + 1, next_page, next_row);
    __syncthreads();   // K's tile is free
    if (ti + 1 < t1) load(k_s, PITCH, K, p.k.rs, at_k, ti + 1);
    copy_commit();
    // Scores, hidden ones -inf, and the online softmax of each row (8 lanes a row).
#pragma unroll
    for (int r = 0; r < TM; ++r) {
      const int row = ty + 16 * r;
      const Vis v = row_v[row];
      if (p.softcap > 0.f) {
#pragma unroll
        for (int c = 0; c < 4; ++c) s[r][c] = p.softcap * tanhf(s[r][c] * p.scale / p.softcap);
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) s[r][c] *= p.scale;
      }
      if (p.M && valid(row)) {
        const float* mr = p.M + p.m.off + (int64_t)entry_of(row) * p.m.bs + (int64_t)head_of(row) * p.m.hs +
                          (int64_t)query_of(row) * p.m.rs + k0 + tx;
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (visible(v, k0 + tx + 8 * c)) s[r][c] += mr[8 * c];
      }
      if (!within(v, k0, k0 + BN)) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (!visible(v, k0 + tx + 8 * c)) s[r][c] = -INFINITY;
      }
      if constexpr (PAGED) {
        const uint32_t have = paged_keys[ti & 1];
        if (have != 0xffffffffu) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (!((have >> (tx + 8 * c)) & 1u)) s[r][c] = -INFINITY;
        }
      }
      float mt = fmaxf(fmaxf(s[r][0], s[r][1]), fmaxf(s[r][2], s[r][3]));
#pragma unroll
      for (int x = 1; x < 8; x <<= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, x));
      if (mt > m[r]) {
        const float f = S::weight(m[r], mt);
        m[r] = mt;
        l[r] *= f;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[r][c][e] *= f;
      }
      const float mu = m[r] == -INFINITY ? 0.f : m[r];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        s[r][c] = S::weight(s[r][c], mu);
        l[r] += s[r][c];
      }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      float* dst = p_s + (tx + 8 * c) * C::kPp + ty * TM;
      if constexpr (TM == 4) *reinterpret_cast<float4*>(dst) = make_float4(s[0][c], s[1][c], s[2][c], s[3][c]);
      else *reinterpret_cast<float2*>(dst) = make_float2(s[0][c], s[1][c]);
    }
    copy_wait<1>();
    __syncthreads();
#pragma unroll(D <= 64 ? 8 : 4)
    for (int j = 0; j < BN; ++j) {
      float pr[TM];
      const float* ps = p_s + j * C::kPp + ty * TM;
      if constexpr (TM == 4) {
        const float4 p4 = *reinterpret_cast<const float4*>(ps);
        pr[0] = p4.x, pr[1] = p4.y, pr[2] = p4.z, pr[3] = p4.w;
      } else {
        const float2 p2 = *reinterpret_cast<const float2*>(ps);
        pr[0] = p2.x, pr[1] = p2.y;
      }
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const float4 v4 = *reinterpret_cast<const float4*>(v_s + j * D + c * 32 + tx * 4);
#pragma unroll
        for (int r = 0; r < TM; ++r) {
          const float2 pp = make_float2(pr[r], pr[r]);
          const float2 lo = fma2(pp, make_float2(v4.x, v4.y), make_float2(o[r][c][0], o[r][c][1]));
          const float2 hi = fma2(pp, make_float2(v4.z, v4.w), make_float2(o[r][c][2], o[r][c][3]));
          o[r][c][0] = lo.x;
          o[r][c][1] = lo.y;
          o[r][c][2] = hi.x;
          o[r][c][3] = hi.y;
        }
      }
    }
    __syncthreads();   // V's tile and P are free
    if (ti + 1 < t1) load(v_s, D, V, p.v.rs, at_v, ti + 1);
    copy_commit();
  }
  copy_wait<0>();

#pragma unroll
  for (int r = 0; r < TM; ++r) {
    const int row = ty + 16 * r;
#pragma unroll
    for (int x = 1; x < 8; x <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], x);
    if (!valid(row)) continue;
    const int i = query_of(row), h = head_of(row), e = entry_of(row);
    float f = 1.f, M = S::natural(m[r]);
    if (!sp.part_o && p.sink_on) f = fold_sink<false>(M, l[r], sink_logit(p, h));
    const bool hidden = l[r] == 0.f;
    const float lse = hidden ? -INFINITY : S::lse(M, log2f(l[r]));
    const float fill = sp.part_o || p.masked_zero ? 0.f : NAN;
    const int64_t at = ((int64_t)e * p.H + h) * p.Sq + i;
    float* dst = sp.part_o ? sp.part_o + (at * stride + split) * D
                           : static_cast<float*>(p.O) + p.o.off + (int64_t)e * p.o.bs + (int64_t)h * p.o.hs +
                                 (int64_t)i * p.o.rs;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const float4 y = hidden ? make_float4(fill, fill, fill, fill)
                              : make_float4(o[r][c][0] * f / l[r], o[r][c][1] * f / l[r], o[r][c][2] * f / l[r],
                                            o[r][c][3] * f / l[r]);
      *reinterpret_cast<float4*>(dst + c * 32 + tx * 4) = y;
    }
    if (tx == 0) {
      if (sp.part_o) sp.part_lse[at * stride + split] = sp.part_l && !hidden ? M : lse;
      if (sp.part_l) sp.part_l[at * stride + split] = l[r];
      if (!sp.part_o && p.lse) p.lse[(int64_t)e * p.lse_bs + (int64_t)h * p.lse_hs + i] = lse;
    }
  }
}

template <int D, int TM, int KIND>
int launch(const Problem& p, const Ext& x, const Split& sp, int stride, cudaStream_t st) {
  using C = Cfg<D, TM>;
  const int64_t entries = KIND == kPacked ? 1 : p.B, rows = (int64_t)p.Sq * p.qpg * (KIND == kPacked ? p.B : 1);
  const int64_t row_blocks = (rows + C::BM - 1) / C::BM;
  const int64_t blocks = row_blocks * entries * p.G * sp.n_splits;
  if (blocks > INT_MAX) return -1;
  auto kern = window_f32_kernel<D, TM, KIND>;
  if (ensure_smem((const void*)kern, C::kSmem) != cudaSuccess) return ATTN_ERR_CUDA;
  kern<<<(unsigned)blocks, kThreads, C::kSmem, st>>>(p, x, sp, row_blocks, stride);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

// Four rows a thread when their CTAs fill the SMs, else two: more, shorter CTAs.  (In pages also two where a block has no
// more rows: 77 entries of 28 tokens, 2/2 heads, head_dim 64, with 350 to 430 keys: 60.6 -> 39.6 us.)
inline int row_tiles(int D, int64_t lists, int64_t rows) {
  return D <= 128 && rows > 32 && (rows + 63) / 64 * lists >= 2 * 152 ? 4 : 2;
}

template <int D, int KIND>
int launch_d(const Problem& p, const Ext& x, const Split& sp, int stride, cudaStream_t st) {
  const int64_t entries = KIND == kPacked ? 1 : p.B, rows = (int64_t)p.Sq * p.qpg * (KIND == kPacked ? p.B : 1);
  const int64_t lists = entries * p.G * sp.n_splits;
  if constexpr (D <= 128) {
    if (row_tiles(D, lists, KIND == kPlain && rows <= 32 ? 64 : rows) == 4) return launch<D, 4, KIND>(p, x, sp, stride, st);
  }
  return launch<D, 2, KIND>(p, x, sp, stride, st);
}

// The instance for a head_dim (-1: there is none, or the grid is too large).
template <int KIND>
int launch_head_dim(const Problem& p, const Ext& x, const Split& sp, int stride, cudaStream_t st) {
  switch (p.D) {
    case 32: return launch_d<32, KIND>(p, x, sp, stride, st);
    case 64: return launch_d<64, KIND>(p, x, sp, stride, st);
    case 128: return launch_d<128, KIND>(p, x, sp, stride, st);
    case 256: return launch_d<256, KIND>(p, x, sp, stride, st);
    default: return -1;
  }
}

}  // namespace
}  // namespace attn
