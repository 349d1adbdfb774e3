// paged_join.cu -- joins the fragments of a paged decode (paged.cuh).
//
// A unit is cut when its tile list crosses the end of a share; the share that
// ends it has noted where it began.  One warp a row of O merges the partial
// results in list order: O = sum_f exp(lse_f - M) O_f / sum_f exp(lse_f - M),
// with the sink's logit as one more term of the denominator.  The kernel is
// launched as the pass's programmatic dependent: its CTAs are in place when
// the pass ends.
#include "paged.cuh"

namespace attn {
namespace paged {
namespace {

constexpr int kJoinWarps = 8;

template <typename T>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const Work w) {
  const Problem& p = w.p;
  const int lane = threadIdx.x % 32, cta = blockIdx.x;
  wait_for_previous();
  const CutUnit cut = w.cuts[cta];
  if (cut.b < 0) return;
  const int g = cut.u / w.n_hc, h0 = g * p.qpg + cut.u % w.n_hc * w.heads;
  const int nh = min(w.heads, (g + 1) * p.qpg - h0), count = cta - cut.c0 + 1;
  for (int hh = threadIdx.x / 32; hh < nh; hh += kJoinWarps) {
    const int h = h0 + hh;
    const float sg = p.sink_on ? sink_logit(p, h) : -INFINITY;
    auto slot_row = [&](int f) { return ((int64_t)(cut.c0 + f) * 2 + (f == 0 ? cut.late : 0)) * w.heads + hh; };
    bool bad = isnan(sg) || sg == INFINITY;
    float M = bad ? -INFINITY : sg;
    for (int f = lane; f < count; f += 32) {
      const float x = w.part_lse[slot_row(f)];
      if (isnan(x) || x == INFINITY) bad = true;
      else M = fmaxf(M, x);
    }
    bad = __any_sync(kAll, bad);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kAll, M, o));
    float acc[8], ws = 0.f;
#pragma unroll
    for (int s = 0; s < 8; ++s) acc[s] = 0.f;
    const bool normal = !bad && M != -INFINITY;
    if (normal) {
      for (int base = 0; base < count; base += 32) {
        const float x = base + lane < count ? w.part_lse[slot_row(base + lane)] : -INFINITY;
        const float wr = x == -INFINITY ? 0.f : expf(x - M);
        ws += wr;
        const int nr = min(32, count - base);
        for (int k = 0; k < nr; k += 4) {
          float wk[4], v[4][8];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            wk[q] = __shfl_sync(kAll, wr, k + q);   // lanes past the last fragment hold 0
            const float* src = w.part_o + slot_row(min(base + k + q, count - 1)) * p.D;
#pragma unroll
            for (int s = 0; s < 8; ++s) v[q][s] = lane + 32 * s < p.D ? src[lane + 32 * s] : 0.f;
          }
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int s = 0; s < 8; ++s) acc[s] = wk[q] != 0.f ? fmaf(wk[q], v[q][s], acc[s]) : acc[s];
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ws += __shfl_xor_sync(kAll, ws, o);
      if (sg > -INFINITY) ws += expf(sg - M);
    }
    const float fill = !bad && p.masked_zero ? 0.f : NAN;
    T* out = static_cast<T*>(p.O) + p.o.off + (int64_t)cut.b * p.o.bs + (int64_t)h * p.o.hs;
#pragma unroll
    for (int s = 0; s < 8; ++s)
      if (lane + 32 * s < p.D) out[lane + 32 * s] = from_f32<T>(normal ? acc[s] / ws : fill);
    if (p.lse && lane == 0)
      p.lse[(int64_t)cut.b * p.lse_bs + (int64_t)h * p.lse_hs] =
          bad ? NAN : (M == -INFINITY ? -INFINITY : M + logf(ws));
  }
}

}  // namespace

cudaError_t launch_join(const Work& w, cudaStream_t st) {
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)w.ctas);
  c.blockDim = dim3(32 * kJoinWarps);
  c.stream = st;
  c.attrs = &at;
  c.numAttrs = 1;
  if (w.p.dtype == ATTN_F32) return cudaLaunchKernelEx(&c, join_kernel<float>, w);
  if (w.p.dtype == ATTN_F16) return cudaLaunchKernelEx(&c, join_kernel<__half>, w);
  return cudaLaunchKernelEx(&c, join_kernel<__nv_bfloat16>, w);
}

}  // namespace paged
}  // namespace attn
