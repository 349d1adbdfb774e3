// paged_join.cu -- joins the fragments of a paged decode (paged.cuh).
//
// One warp a row of O: it finds which shares hold its unit's tile list from
// the lengths alone, as the pass did, and merges their partial results in list
// order: O = sum_f exp(lse_f - M) O_f / sum_f exp(lse_f - M), with the sink's
// logit as one more term of the denominator.  Rows that one share held are
// already written; rows of entries without a visible key are filled here.
#include "paged.cuh"

namespace attn {
namespace paged {
namespace {

template <typename T>
__global__ void __launch_bounds__(128) join_kernel(const Work w) {
  const Problem& p = w.p;
  const int lane = threadIdx.x % 32;
  const int64_t row = (int64_t)blockIdx.x * 4 + threadIdx.x / 32;
  if (row >= (int64_t)p.B * p.H) return;
  const int b = (int)(row / p.H), h = (int)(row % p.H);
  const int g = h / p.qpg, hc = (h % p.qpg) / w.heads, hh = (h % p.qpg) % w.heads;
  const int units = p.G * w.n_hc, u = g * w.n_hc + hc;
  const int n = entry_tiles(w, b);
  const float sg = p.sink_on ? sink_logit(p, h) : -INFINITY;
  int c0 = 0, count = 0;
  bool late = false;   // the first fragment is not the first of its share
  if (n > 0) {
    const int64_t total = tiles_before(w, p.B, lane) * units;
    const int shares = (int)min((int64_t)w.ctas, total);
    const int64_t at = tiles_before(w, b, lane) * units + (int64_t)u * n;
    c0 = share_of(total, shares, at);
    count = share_of(total, shares, at + n - 1) - c0 + 1;
    if (count == 1) return;
    late = share_begin(total, shares, c0) < at;
  }
  auto slot_row = [&](int f) { return ((int64_t)(c0 + f) * 2 + (f == 0 && late ? 1 : 0)) * w.heads + hh; };
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
  T* out = static_cast<T*>(p.O) + p.o.off + (int64_t)b * p.o.bs + (int64_t)h * p.o.hs;
#pragma unroll
  for (int s = 0; s < 8; ++s)
    if (lane + 32 * s < p.D) out[lane + 32 * s] = from_f32<T>(normal ? acc[s] / ws : fill);
  if (p.lse && lane == 0)
    p.lse[(int64_t)b * p.lse_bs + (int64_t)h * p.lse_hs] = bad ? NAN : (M == -INFINITY ? -INFINITY : M + logf(ws));
}

}  // namespace

cudaError_t launch_join(const Work& w, cudaStream_t st) {
  const int64_t blocks = ((int64_t)w.p.B * w.p.H + 3) / 4;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  if (w.p.dtype == ATTN_F32) join_kernel<float><<<(unsigned)blocks, 128, 0, st>>>(w);
  else if (w.p.dtype == ATTN_F16) join_kernel<__half><<<(unsigned)blocks, 128, 0, st>>>(w);
  else join_kernel<__nv_bfloat16><<<(unsigned)blocks, 128, 0, st>>>(w);
  return cudaGetLastError();
}

}  // namespace paged
}  // namespace attn
