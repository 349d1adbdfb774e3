// window_f32.cu -- float32 attention under a sliding window with first keys, on
// the CUDA cores at head_dim 32, 64, 128 or 256.
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
// What bounds it: FMA issue (4 head_dim FLOPs a visible pair against 152 x 128
// lanes), for small problems the chain of one CTA's tiles.
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

template <int D, int TM>
struct Cfg {
  static constexpr int BM = 16 * TM;
  static constexpr int kPitch = D + 4;                                    // floats
  static constexpr int kPp = BM + 4;                                      // of P, by key
  static constexpr int kSmem = ((BM + BN) * kPitch + BN * D + BN * kPp) * 4;
  static constexpr int kCtas = kSmem <= 74 * 1024 ? 3 : 2;
};

template <int D, int TM>
__global__ void __launch_bounds__(kThreads, Cfg<D, TM>::kCtas)
    window_f32_kernel(const Problem p, const int first, const Split sp, const int64_t row_blocks) {
  using C = Cfg<D, TM>;
  constexpr int BM = C::BM, PITCH = C::kPitch, NC = D / 32;
  extern __shared__ __align__(16) float smem[];
  float* q_s = smem;
  float* k_s = q_s + BM * PITCH;
  float* v_s = k_s + BN * PITCH;
  float* p_s = v_s + BN * D;
  __shared__ Vis row_v[BM];
  __shared__ int row_q[BM], row_h[BM], s_f[2], s_w[2];
  const int tid = threadIdx.x, tx = tid % 8, ty = tid / 8;

  int64_t blk = blockIdx.x;
  const int split = (int)(blk % sp.n_splits);
  blk /= sp.n_splits;
  const int64_t rb = blk % row_blocks;
  blk /= row_blocks;
  const int g = (int)(blk % p.G), b = (int)(blk / p.G);
  // Query and head of each row (-1: behind the last).
  auto query_of = [&](int row) { return row_q[row]; };
  auto head_of = [&](int row) { return row_h[row]; };
  auto valid = [&](int row) { return row_q[row] >= 0; };

  if (tid == 0) {
    s_f[0] = s_w[0] = INT_MAX;
    s_f[1] = s_w[1] = -1;
  }
  __syncthreads();
  if (tid < BM) {
    const int64_t r = rb * BM + tid;
    const int i = (int)(r / p.qpg);
    row_q[tid] = i < p.Sq ? i : -1;
    row_h[tid] = g * p.qpg + (int)(r - (int64_t)i * p.qpg);
    const Vis v = i < p.Sq ? row_vis(p, first, b, i) : Vis{0, 0, 0, 0};
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

  const float* Q = static_cast<const float*>(p.Q) + p.q.off + (int64_t)b * p.q.bs;
  const float* K = static_cast<const float*>(p.K) + p.k.off + (int64_t)b * p.k.bs + (int64_t)g * p.k.hs;
  const float* V = static_cast<const float*>(p.V) + p.v.off + (int64_t)b * p.v.bs + (int64_t)g * p.v.hs;
  constexpr int kChunks = D / 4;   // 16-byte chunks of a row
  for (int c = tid; c < BM * kChunks; c += kThreads) {
    const int row = c / kChunks, d = c % kChunks * 4;
    const bool ok = valid(row);
    copy16(smem_u32(q_s + row * PITCH + d),
           ok ? Q + (int64_t)head_of(row) * p.q.hs + (int64_t)query_of(row) * p.q.rs + d : Q, ok ? 16 : 0);
  }
  // Rows no row of the CTA sees arrive as zeros and are not read.
  auto load = [&](float* dst, int pitch, const float* src, int64_t rs, int ti) {
    const int k0 = tl.tile(ti) * BN;
    for (int c = tid; c < BN * kChunks; c += kThreads) {
      const int row = c / kChunks, d = c % kChunks * 4;
      const bool ok = visible(uv, k0 + row);
      copy16(smem_u32(dst + row * pitch + d), ok ? src + (int64_t)(k0 + row) * rs + d : src, ok ? 16 : 0);
    }
  };
  if (t0 < t1) load(k_s, PITCH, K, p.k.rs, t0);
  copy_commit();
  if (t0 < t1) load(v_s, D, V, p.v.rs, t0);
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
    __syncthreads();   // K's tile is free
    if (ti + 1 < t1) load(k_s, PITCH, K, p.k.rs, ti + 1);
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
        const float* mr = p.M + p.m.off + (int64_t)b * p.m.bs + (int64_t)head_of(row) * p.m.hs +
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
#pragma unroll
      for (int r = 0; r < TM; ++r) pr[r] = p_s[j * C::kPp + ty * TM + r];
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        const float4 v4 = *reinterpret_cast<const float4*>(v_s + j * D + c * 32 + tx * 4);
#pragma unroll
        for (int r = 0; r < TM; ++r) {
          o[r][c][0] = fmaf(pr[r], v4.x, o[r][c][0]);
          o[r][c][1] = fmaf(pr[r], v4.y, o[r][c][1]);
          o[r][c][2] = fmaf(pr[r], v4.z, o[r][c][2]);
          o[r][c][3] = fmaf(pr[r], v4.w, o[r][c][3]);
        }
      }
    }
    __syncthreads();   // V's tile and P are free
    if (ti + 1 < t1) load(v_s, D, V, p.v.rs, ti + 1);
    copy_commit();
  }
  copy_wait<0>();

#pragma unroll
  for (int r = 0; r < TM; ++r) {
    const int row = ty + 16 * r;
#pragma unroll
    for (int x = 1; x < 8; x <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], x);
    if (!valid(row)) continue;
    const int i = query_of(row), h = head_of(row);
    float f = 1.f, M = S::natural(m[r]);
    if (!sp.part_o && p.sink_on) f = fold_sink<false>(M, l[r], sink_logit(p, h));
    const bool hidden = l[r] == 0.f;
    const float lse = hidden ? -INFINITY : S::lse(M, log2f(l[r]));
    const float fill = sp.part_o || p.masked_zero ? 0.f : NAN;
    const int64_t at = ((int64_t)b * p.H + h) * p.Sq + i;
    float* dst = sp.part_o ? sp.part_o + (at * sp.n_splits + split) * D
                           : static_cast<float*>(p.O) + p.o.off + (int64_t)b * p.o.bs + (int64_t)h * p.o.hs +
                                 (int64_t)i * p.o.rs;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const float4 y = hidden ? make_float4(fill, fill, fill, fill)
                              : make_float4(o[r][c][0] * f / l[r], o[r][c][1] * f / l[r], o[r][c][2] * f / l[r],
                                            o[r][c][3] * f / l[r]);
      *reinterpret_cast<float4*>(dst + c * 32 + tx * 4) = y;
    }
    if (tx == 0) {
      if (sp.part_o) sp.part_lse[at * sp.n_splits + split] = sp.part_l && !hidden ? M : lse;
      if (sp.part_l) sp.part_l[at * sp.n_splits + split] = l[r];
      if (!sp.part_o && p.lse) p.lse[(int64_t)b * p.lse_bs + (int64_t)h * p.lse_hs + i] = lse;
    }
  }
}

template <int D, int TM>
int launch(const Problem& p, int first, const Split& sp, cudaStream_t st) {
  using C = Cfg<D, TM>;
  const int64_t row_blocks = ((int64_t)p.Sq * p.qpg + C::BM - 1) / C::BM;
  const int64_t blocks = row_blocks * p.B * p.G * sp.n_splits;
  if (blocks > INT_MAX) return -1;
  auto kern = window_f32_kernel<D, TM>;
  if (ensure_smem((const void*)kern, C::kSmem) != cudaSuccess) return ATTN_ERR_CUDA;
  kern<<<(unsigned)blocks, kThreads, C::kSmem, st>>>(p, first, sp, row_blocks);
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

// Four rows a thread when their CTAs fill the SMs, else two: more, shorter CTAs.
template <int D>
int launch_d(const Problem& p, int first, const Split& sp, cudaStream_t st) {
  const int64_t big = ((int64_t)p.Sq * p.qpg + 63) / 64 * p.B * p.G * sp.n_splits;
  if constexpr (D <= 128) {
    if (big >= 2 * 152) return launch<D, 4>(p, first, sp, st);
  }
  return launch<D, 2>(p, first, sp, st);
}

}  // namespace

int window_f32_try(const Problem& p, int first, const Split& sp, cudaStream_t st, int* used) {
  *used = 0;
  if (p.dtype != ATTN_F32 || p.kv_int8 || p.Sk < 1) return ATTN_OK;
  if (!tma_layout_ok_es(p.Q, p.q, p.Sq, p.H, p.B, 4) || !tma_layout_ok_es(p.K, p.k, p.Sk, p.G, p.B, 4) ||
      !tma_layout_ok_es(p.V, p.v, p.Sk, p.G, p.B, 4) || !tma_layout_ok_es(p.O, p.o, p.Sq, p.H, p.B, 4))
    return ATTN_OK;   // 16-byte loads and stores of rows
  const float sc = p.scale * S::kLog2;
  if (!(sc == sc) || isinf(sc)) return ATTN_OK;
  int rc = -1;
  switch (p.D) {
    case 32: rc = launch_d<32>(p, first, sp, st); break;
    case 64: rc = launch_d<64>(p, first, sp, st); break;
    case 128: rc = launch_d<128>(p, first, sp, st); break;
    case 256: rc = launch_d<256>(p, first, sp, st); break;
  }
  if (rc < 0) return ATTN_OK;
  *used = 1;
  return rc;
}

}  // namespace attn
