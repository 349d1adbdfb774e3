// paged_join.cu -- joins the fragments of a paged decode (paged.cuh).
//
// A unit is cut when its tile list crosses the end of a share; the share that
// ends it has noted where it began, and the CTA of that share's number merges
// the unit: O = sum_f l_f exp(m_f - M) O_f / sum_f l_f exp(m_f - M), in an order
// fixed by the cut, with the sink's logit as one more term of the denominator.
// The kernel is launched as the pass's programmatic dependent: its CTAs are in
// place when the pass ends.  Its time is the latency of the fragments' loads,
// so a thread has up to eight in flight.
#include "paged.cuh"

namespace attn {
namespace paged {
namespace {

constexpr int kJoinWarps = 8;
constexpr int kJoinThreads = 32 * kJoinWarps;
constexpr int kMaxHeads = 16;   // query heads of a unit

template <typename T>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const Work w) {
  __shared__ float s_top[kMaxHeads], s_sum[kMaxHeads];   // of each row's fragments and sink
  __shared__ float4 s_acc[kJoinThreads];
  const Problem& p = w.p;
  const int tid = threadIdx.x, lane = tid % 32, cta = blockIdx.x, D = p.D;
  wait_for_previous();
  const CutUnit cut = w.cuts[cta];
  if (cut.b < 0) return;
  const int g = cut.u / w.n_hc, h0 = g * p.qpg + cut.u % w.n_hc * w.heads;
  const int nh = min(w.heads, (g + 1) * p.qpg - h0), count = cta - cut.c0 + 1;
  auto slot_row = [&](int f, int hh) {
    return ((int64_t)(cut.c0 + f) * 2 + (f == 0 ? cut.late : 0)) * w.heads + hh;
  };
  // A row's maximum and sum: one warp a row, its lanes over the fragments.  A NaN top marks a NaN row.
  for (int hh = tid / 32; hh < nh; hh += kJoinWarps) {
    const float sg = p.sink_on ? sink_logit(p, h0 + hh) : -INFINITY;
    bool bad = isnan(sg) || sg == INFINITY;
    float M = bad ? -INFINITY : sg;
    for (int f = lane; f < count; f += 32) {
      const int64_t at = slot_row(f, hh);
      const float x = w.part_m[at];
      if (x == INFINITY || isnan(w.part_l[at])) bad = true;
      else M = fmaxf(M, x);
    }
    bad = __any_sync(kAll, bad);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kAll, M, o));
    float sum = 0.f;
    if (!bad && M != -INFINITY) {
      for (int f = lane; f < count; f += 32) {
        const int64_t at = slot_row(f, hh);
        const float x = w.part_m[at];
        sum += x == -INFINITY ? 0.f : w.part_l[at] * expf(x - M);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
      if (sg > -INFINITY) sum += expf(sg - M);
    }
    if (lane == 0) {
      s_top[hh] = bad ? NAN : M;
      s_sum[hh] = sum;
      if (p.lse)
        p.lse[(int64_t)cut.b * p.lse_bs + (int64_t)(h0 + hh) * p.lse_hs] =
            bad ? NAN : (M == -INFINITY ? -INFINITY : M + logf(sum));
    }
  }
  __syncthreads();
  // Four columns a thread; groups of threads that hold the same columns take
  // the fragments in turn and add up in group order.
  const int cols = nh * (D / 4), groups = max(1, kJoinThreads / cols), group = tid / cols;
  for (int c0 = 0; c0 < cols; c0 += kJoinThreads) {
    const int c = groups > 1 ? tid % cols : c0 + tid, hh = c / (D / 4), d = c % (D / 4) * 4;
    const bool mine = groups > 1 ? group < groups : c < cols;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    const float M = mine ? s_top[hh] : NAN;
    const bool normal = M == M && M != -INFINITY;
    if (normal) {
      for (int f0 = groups > 1 ? group : 0; f0 < count; f0 += 8 * groups) {
        float x[8], l[8];
        float4 v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const int f = f0 + q * groups;
          x[q] = -INFINITY;
          if (f < count) {
            const int64_t at = slot_row(f, hh);
            x[q] = w.part_m[at];
            l[q] = w.part_l[at];
            v[q] = *reinterpret_cast<const float4*>(w.part_o + at * D + d);
          }
        }
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          if (x[q] == -INFINITY) continue;   // an empty fragment
          const float k = l[q] * expf(x[q] - M);
          acc.x = fmaf(k, v[q].x, acc.x);
          acc.y = fmaf(k, v[q].y, acc.y);
          acc.z = fmaf(k, v[q].z, acc.z);
          acc.w = fmaf(k, v[q].w, acc.w);
        }
      }
    }
    if (groups > 1) {
      s_acc[tid] = acc;
      __syncthreads();
      if (tid < cols)
        for (int k = 1; k < groups; ++k) {
          const float4 y = s_acc[k * cols + tid];
          acc.x += y.x;
          acc.y += y.y;
          acc.z += y.z;
          acc.w += y.w;
        }
    }
    if (mine && (groups == 1 || tid < cols)) {
      const float fill = M == M && p.masked_zero ? 0.f : NAN, sum = s_sum[hh];
      T* out = static_cast<T*>(p.O) + p.o.off + (int64_t)cut.b * p.o.bs + (int64_t)(h0 + hh) * p.o.hs + d;
      const float a[4] = {acc.x, acc.y, acc.z, acc.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) out[e] = from_f32<T>(normal ? a[e] / sum : fill);
    }
  }
}

}  // namespace

cudaError_t launch_join(const Work& w, cudaStream_t st) {
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)w.ctas);
  c.blockDim = dim3(kJoinThreads);
  c.stream = st;
  c.attrs = &at;
  c.numAttrs = 1;
  if (w.p.dtype == ATTN_F32) return cudaLaunchKernelEx(&c, join_kernel<float>, w);
  if (w.p.dtype == ATTN_F16) return cudaLaunchKernelEx(&c, join_kernel<__half>, w);
  return cudaLaunchKernelEx(&c, join_kernel<__nv_bfloat16>, w);
}

}  // namespace paged
}  // namespace attn
