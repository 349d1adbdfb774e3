// simt.cu -- CUDA-core kernels: the exact float32 forward (also the generic
// fallback for half/bfloat16 layouts the tensor-core path cannot take), the
// generic split-range decode pass, and the partial-result combine.  The
// forward kernel itself is in simt_fwd.cuh; this file launches its general
// layout and hands head_dim 8 x threads-per-row to the chunked form
// (simt_full.cu).
#include "simt_fwd.cuh"

namespace attn {

namespace {

// Where the ranges give LSEs under a mask: a maximum of 2^28 or more, which the
// mask brought in, has absorbed the scores beside it and in the LSE the
// logarithm of the sum, so the keys that carry it are counted.
struct Ranges {
  static constexpr bool kOn = true;
  Problem p;
  int split_len;
  // Visible keys of range r whose mask is M, counted by a warp.
  __device__ float count(int b, int h, int i, int r, float M, int lane) const {
    int64_t lo, hi;
    row_range(p, b, i, lo, hi);
    lo = max(lo, (int64_t)r * split_len);
    hi = min(hi, (int64_t)(r + 1) * split_len);
    const float* m = p.M + p.m.off + (int64_t)b * p.m.bs + (int64_t)h * p.m.hs + (int64_t)i * p.m.rs;
    int n = 0;
    for (int64_t k = lo + lane; k < hi; k += 32) n += m[k] == M;
    return (float)max(__reduce_add_sync(0xffffffffu, n), 1);
  }
};
struct NoMask {
  static constexpr bool kOn = false;
};

// One warp per row: merge the row's range partials in range order.
// With sink_on the head's sink logit enters as one more range with an
// empty numerator (the sink term of the denominator, added once per row).
// The lanes read the ranges' LSEs in parallel (lane r: ranges r, r + 32, ...)
// and broadcast the weights; the partial rows of four ranges are loaded
// before they are summed, so the loads overlap instead of queueing behind one
// another.  Ranges with weight 0 (empty, or underflowed) are left out of the
// sum by a select, so an unwritten partial never reaches it.  With part_l the
// ranges give maxima and sums in place of LSEs (Split).
template <typename T, typename Mask>
__global__ void __launch_bounds__(128) combine_kernel(int n_splits, int64_t rows, int D, const float* part_o,
                                                      const float* part_lse, const float* part_l, T* O,
                                                      Layout ol, int H, int Sq, float* lse, int64_t lse_bs,
                                                      int64_t lse_hs, int64_t lse_rs, int masked_zero, int sink_on,
                                                      const float* sink, const Mask mask) {
  constexpr unsigned kAll = 0xffffffffu;
  const int64_t row = (int64_t)blockIdx.x * 4 + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  if (row >= rows) return;
  const float* pl = part_lse + row * n_splits;
  const float* sums = part_l ? part_l + row * n_splits : nullptr;
  const int i = (int)(row % Sq);
  const int h = (int)((row / Sq) % H);
  const float sg = sink_on ? (sink ? sink[h] : 0.f) : -INFINITY;
  bool bad = isnan(sg) || sg == INFINITY;
  float M = bad ? -INFINITY : sg;
  for (int r = lane; r < n_splits; r += 32) {
    const float x = pl[r];
    if (isnan(x) || x == INFINITY || (sums && isnan(sums[r]))) bad = true;
    else M = fmaxf(M, x);
  }
  bad = __any_sync(kAll, bad);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kAll, M, o));
  const int64_t b = row / ((int64_t)Sq * H);
  const int64_t ob = ol.off + b * ol.bs + (int64_t)h * ol.hs + (int64_t)i * ol.rs;
  const bool normal = !bad && M != -INFINITY;
  float acc[8];
#pragma unroll
  for (int s = 0; s < 8; ++s) acc[s] = 0.f;
  float ws = 0.f;
  if (normal) {
    for (int base = 0; base < n_splits; base += 32) {
      const int r = base + lane;
      const float x = r < n_splits ? pl[r] : -INFINITY;
      float wr = x == -INFINITY ? 0.f : expf(x - M);
      if (sums && wr != 0.f) wr *= sums[r];
      if constexpr (Mask::kOn)
        if (fabsf(M) >= 0x1p28f)
          for (uint32_t top = __ballot_sync(kAll, x == M && r < n_splits); top; top &= top - 1) {
            const int at = __ffs(top) - 1;
            const float n = mask.count((int)b, h, i, base + at, M, lane);
            if (lane == at) wr *= n;
          }
      ws += wr;
      const int nr = min(32, n_splits - base);
      for (int k = 0; k < nr; k += 4) {
        float w[4], v[4][8];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          w[u] = __shfl_sync(kAll, wr, k + u);   // lanes past the last range hold 0
          const float* src = part_o + (row * n_splits + min(base + k + u, n_splits - 1)) * D;
#pragma unroll
          for (int s = 0; s < 8; ++s) {
            const int d = lane + 32 * s;
            v[u][s] = d < D ? src[d] : 0.f;
          }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int s = 0; s < 8; ++s) acc[s] = w[u] != 0.f ? fmaf(w[u], v[u][s], acc[s]) : acc[s];
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ws += __shfl_xor_sync(kAll, ws, o);
    if (sg > -INFINITY) ws += expf(sg - M);
  }
  const float val_fill = (!bad && M == -INFINITY) ? (masked_zero ? 0.f : NAN) : NAN;
#pragma unroll
  for (int s = 0; s < 8; ++s) {
    const int d = lane + 32 * s;
    if (d < D) O[ob + d] = from_f32<T>(normal ? acc[s] / ws : val_fill);
  }
  if (lse && lane == 0)
    lse[b * lse_bs + (int64_t)h * lse_hs + (int64_t)i * lse_rs] =
        bad ? NAN : (M == -INFINITY ? -INFINITY : M + logf(ws));
}

template <typename T, typename Mask>
cudaError_t launch_combine_t(int n_splits, int64_t rows, int D, const float* po, const float* pl, const float* sums,
                             void* o,
                             Layout ol, int H, int Sq, float* lse, int64_t lbs, int64_t lhs, int64_t lrs,
                             int masked_zero, int sink_on, const float* sink, const Mask& mask, cudaStream_t st) {
  if (rows <= 0) return cudaSuccess;
  const int64_t blocks = (rows + 3) / 4;
  if (blocks > INT_MAX) return cudaErrorInvalidConfiguration;
  combine_kernel<T, Mask><<<(unsigned)blocks, 128, 0, st>>>(n_splits, rows, D, po, pl, sums, static_cast<T*>(o), ol, H,
                                                            Sq, lse, lbs, lhs, lrs, masked_zero, sink_on, sink, mask);
  return cudaGetLastError();
}

template <typename Mask>
cudaError_t combine_dispatch(int32_t dt, int n_splits, int64_t rows, int D, const float* po, const float* pl,
                             const float* sums, void* o, Layout ol, int H, int Sq, float* lse, int64_t lbs, int64_t lhs,
                             int64_t lrs, int masked_zero, int sink_on, const float* sink, const Mask& mask,
                             cudaStream_t st) {
  switch (dt) {
    case ATTN_F32:
      return launch_combine_t<float>(n_splits, rows, D, po, pl, sums, o, ol, H, Sq, lse, lbs, lhs, lrs, masked_zero,
                                     sink_on, sink, mask, st);
    case ATTN_F16:
      return launch_combine_t<__half>(n_splits, rows, D, po, pl, sums, o, ol, H, Sq, lse, lbs, lhs, lrs, masked_zero,
                                      sink_on, sink, mask, st);
    default:
      return launch_combine_t<__nv_bfloat16>(n_splits, rows, D, po, pl, sums, o, ol, H, Sq, lse, lbs, lhs, lrs,
                                             masked_zero, sink_on, sink, mask, st);
  }
}

}  // namespace

cudaError_t launch_simt(const Problem& p, const Split& s, cudaStream_t st) {
  if (p.D == 32 || p.D == 64 || p.D == 128 || p.D == 256) return launch_simt_full(p, s, st);
  return launch_simt_all<false, false>(p, s, st, Ext{});
}

cudaError_t launch_combine(const Problem& p, const Split& s, int32_t out_dtype, cudaStream_t st) {
  const int64_t rows = (int64_t)p.B * p.H * p.Sq;
  auto go = [&](const auto& mask) {
    return combine_dispatch(out_dtype, s.n_splits, rows, p.D, s.part_o, s.part_lse, s.part_l, p.O, p.o, p.H, p.Sq,
                            p.lse, p.lse_bs, p.lse_hs, 1, p.masked_zero, p.sink_on, p.sink, mask, st);
  };
  return p.M && !s.part_l ? go(Ranges{p, s.split_len}) : go(NoMask{});
}

cudaError_t launch_combine_flat(int n_splits, int rows, int D, const float* part_o, const float* part_lse,
                                int32_t out_dtype, void* o, int64_t o_row_stride, float* lse, int masked_zero,
                                cudaStream_t st) {
  Layout ol{0, 0, 0, o_row_stride};
  return combine_dispatch(out_dtype, n_splits, rows, D, part_o, part_lse, nullptr, o, ol, 1, rows, lse, 0, 0, 1,
                          masked_zero, 0, nullptr, NoMask{}, st);
}

}  // namespace attn
