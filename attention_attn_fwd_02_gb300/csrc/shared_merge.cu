// shared_merge.cu -- merges the partial results of a batch over a shared prefix.
//
// What it computes: O = sum_s l_s exp(m_s - M) O_s / sum_s l_s exp(m_s - M) over
// a row's partial results s, with the sink's logit as one more term of the
// denominator, and LSE = M + log of that sum.  Which there are follows from the
// plan (shared.h) and, for own keys that the decode pass cut, from its notes
// (paged.cuh).  A maximum of +inf or NaN or a sum of NaN makes the row NaN: the
// passes' maxima pass over NaN scores, so that a part without any other has a
// maximum of -inf, as an empty one does, and a sum of NaN.
//
// What bounds it: the latency of its loads.  A row of a decode step has up to some
// twenty results: four warps take a row, each every fourth result; a lane reads
// a result's maximum and sum, then four columns each of up to four at a time (at
// head_dim 64 a warp's halves take every other one), and the warps meet in
// shared memory.  Up to four results of a row, those of prompts, have all their
// loads of two rows a warp under way together.  (64 entries of 32 heads, 7 results:
// 4.5 us, one warp a row and eight columns at a time 13; 51200 rows of three: 19 us
// against 42 with 64-bit row numbers and four rows a warp.)
#include "shared.h"

namespace attn {
namespace shr {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kWarps = 4;
constexpr int kFlight = 4;   // results of a row that a team has on their way

// Cut units of own keys (note null: there are none).
struct Cuts {
  const float *o, *m, *l;
  const int2* note;
  int heads, n_hc;
};

// Four elements of a row of O (on a 16-byte boundary).
template <typename T>
__device__ __forceinline__ void store4(T* out, const T (&y)[4]) {
  if constexpr (sizeof(T) == 4) *reinterpret_cast<uint4*>(out) = *reinterpret_cast<const uint4*>(y);
  else *reinterpret_cast<uint2*>(out) = *reinterpret_cast<const uint2*>(y);
}

// Merges the n results of a row (WARPS warps; every thread of them comes here).  load_m, load_l: a result's maximum and
// sum; load_o: four columns of it.
template <typename T, int D, int WARPS, typename M_, typename L_, typename O_>
__device__ __forceinline__ void merge_row(const Problem& p, bool here, int64_t b, int h, int i, int n, M_ load_m,
                                          L_ load_l, O_ load_o) {
  constexpr int kCols = D / 4, kTeams = 32 / kCols;   // lanes of a result's row, results side by side
  __shared__ float s_m[kWarps], s_l[kWarps];
  __shared__ float4 s_acc[kWarps][kCols];
  const int warp = threadIdx.x / 32, part = warp % WARPS;
  const int lane = threadIdx.x % 32, team = lane / kCols, d = lane % kCols * 4;
  const float sg = p.sink_on && part == 0 && here ? sink_logit(p, h) : -INFINITY;
  bool bad = isnan(sg) || sg == INFINITY;
  // This warp's results: part, part + WARPS, ...; the first 32 of them a lane each.
  const int mine = (n - part + WARPS - 1) / WARPS;
  const bool one = lane < mine;
  const float m0 = one ? load_m(part + lane * WARPS) : -INFINITY;
  const float l0 = one ? load_l(part + lane * WARPS) : 0.f;
  float M = bad ? -INFINITY : sg;
  for (int k = lane; k < mine; k += 32) {
    const float m = k < 32 ? m0 : load_m(part + k * WARPS), l = k < 32 ? l0 : load_l(part + k * WARPS);
    if (!(m < INFINITY) || isnan(l)) bad = true;
    else M = fmaxf(M, m);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kAll, M, o));
  const float mu = M == -INFINITY ? 0.f : M;
  float sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int base = 0; base < mine; base += 32) {
    float wt = 0.f;
    if (base + lane < mine) {
      const int k = part + (base + lane) * WARPS;
      const float m = base ? load_m(k) : m0;
      if (m > -INFINITY) wt = (base ? load_l(k) : l0) * expf(m - mu);
    }
    bad = bad || isnan(wt);
    sum += wt;
    const int nr = min(32, mine - base);
    for (int k0 = 0; k0 < nr; k0 += kFlight * kTeams) {
      float f[kFlight];
      float4 v[kFlight];
#pragma unroll
      for (int q = 0; q < kFlight; ++q) {
        const int k = k0 + q * kTeams + team;
        f[q] = __shfl_sync(kAll, wt, k & 31);
        if (k >= nr) f[q] = 0.f;
        if (f[q] != 0.f) v[q] = load_o(part + (base + k) * WARPS, d);
      }
#pragma unroll
      for (int q = 0; q < kFlight; ++q)
        if (f[q] != 0.f) {   // (an empty result was not written)
          acc.x = fmaf(f[q], v[q].x, acc.x);
          acc.y = fmaf(f[q], v[q].y, acc.y);
          acc.z = fmaf(f[q], v[q].z, acc.z);
          acc.w = fmaf(f[q], v[q].w, acc.w);
        }
    }
  }
  bad = __any_sync(kAll, bad);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
  if (!bad && sg > -INFINITY) sum += expf(sg - mu);
  if (bad) sum = NAN;
  if constexpr (kTeams == 2) {
    acc.x += __shfl_xor_sync(kAll, acc.x, 16);
    acc.y += __shfl_xor_sync(kAll, acc.y, 16);
    acc.z += __shfl_xor_sync(kAll, acc.z, 16);
    acc.w += __shfl_xor_sync(kAll, acc.w, 16);
  }
  if constexpr (WARPS > 1) {
    if (lane == 0) {
      s_m[warp] = M;
      s_l[warp] = sum;
    }
    if (team == 0) s_acc[warp][lane % kCols] = acc;
    __syncthreads();
    if (part > 0) return;
    float f[WARPS], top = -INFINITY;
#pragma unroll
    for (int q = 0; q < WARPS; ++q) top = fmaxf(top, s_m[warp + q]);
    const float to = top == -INFINITY ? 0.f : top;
    sum = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int q = 0; q < WARPS; ++q) {
      f[q] = s_m[warp + q] == -INFINITY ? 0.f : expf(s_m[warp + q] - to);
      const float l = s_l[warp + q];
      sum += isnan(l) ? l : f[q] * l;
      const float4 v = s_acc[warp + q][lane % kCols];
      acc.x = fmaf(f[q], v.x, acc.x);
      acc.y = fmaf(f[q], v.y, acc.y);
      acc.z = fmaf(f[q], v.z, acc.z);
      acc.w = fmaf(f[q], v.w, acc.w);
    }
    M = top;
  }
  if (!here) return;
  const bool nan = isnan(sum), none = !nan && M == -INFINITY;
  if (team == 0) {
    const float fill = none && p.masked_zero ? 0.f : NAN, inv = 1.f / sum;
    const bool plain = !nan && !none;
    T* out = static_cast<T*>(p.O) + p.o.off + b * p.o.bs + (int64_t)h * p.o.hs + (int64_t)i * p.o.rs + d;
    const float a[4] = {acc.x, acc.y, acc.z, acc.w};
    __align__(16) T y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = from_f32<T>(plain ? a[e] * inv : fill);
    store4(out, y);
  }
  if (p.lse && lane == 0)
    p.lse[b * p.lse_bs + (int64_t)h * p.lse_hs + i] = nan ? NAN : none ? -INFINITY : M + logf(sum);
}

// The same for up to kFew results of a row: a lane takes the same four columns of kRowsFew rows (of two rows in turn at
// head_dim 64), whose loads are all under way together.  row_of: a row's place, its results' places and how many there
// are (0: there is no such row), without a look at the maxima and sums that it fetches meanwhile.
constexpr int kFew = 4;
constexpr int kRowsFew = 2;

struct FewRow {
  bool here;
  int b, h, i, n;
  int64_t at[kFew];
  float m[kFew], l[kFew];
  __device__ __forceinline__ void fetch(const Work& w, int most) {
#pragma unroll
    for (int k = 0; k < kFew; ++k) {
      m[k] = here && k < most ? w.part_m[at[k]] : -INFINITY;
      l[k] = here && k < most ? w.part_l[at[k]] : 0.f;
    }
  }
};

template <typename T, int D>
__device__ __forceinline__ void merge_few(const Problem& p, const Work& w, FewRow (&row)[kRowsFew]) {
  constexpr int kCols = D / 4;
  const int d = threadIdx.x % kCols * 4;
  float4 v[kRowsFew][kFew];
#pragma unroll
  for (int q = 0; q < kRowsFew; ++q)
#pragma unroll
    for (int k = 0; k < kFew; ++k) {
      if (k >= row[q].n) row[q].m[k] = -INFINITY, row[q].l[k] = 0.f;
      v[q][k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (row[q].m[k] != -INFINITY) v[q][k] = *reinterpret_cast<const float4*>(w.part_o + row[q].at[k] * D + d);
    }
#pragma unroll
  for (int q = 0; q < kRowsFew; ++q) {
    const FewRow& r = row[q];
    if (!r.here) continue;
    const float sg = p.sink_on ? sink_logit(p, r.h) : -INFINITY;
    bool bad = isnan(sg) || sg == INFINITY;
    float M = bad ? -INFINITY : sg;
#pragma unroll
    for (int k = 0; k < kFew; ++k) {
      if (!(r.m[k] < INFINITY) || isnan(r.l[k])) bad = true;
      else M = fmaxf(M, r.m[k]);
    }
    const float mu = M == -INFINITY ? 0.f : M;
    float sum = sg > -INFINITY ? expf(sg - mu) : 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kFew; ++k) {
      if (r.m[k] == -INFINITY) continue;
      const float f = r.l[k] * expf(r.m[k] - mu);
      sum += f;
      acc.x = fmaf(f, v[q][k].x, acc.x);
      acc.y = fmaf(f, v[q][k].y, acc.y);
      acc.z = fmaf(f, v[q][k].z, acc.z);
      acc.w = fmaf(f, v[q][k].w, acc.w);
    }
    const bool nan = bad || isnan(sum), none = !nan && M == -INFINITY;
    const float fill = none && p.masked_zero ? 0.f : NAN, inv = 1.f / sum;
    T* out = static_cast<T*>(p.O) + p.o.off + r.b * p.o.bs + r.h * p.o.hs + r.i * p.o.rs + d;
    const float a[4] = {acc.x, acc.y, acc.z, acc.w};
    __align__(16) T y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = from_f32<T>(nan || none ? fill : a[e] * inv);
    store4(out, y);
    if (p.lse && d == 0)
      p.lse[r.b * p.lse_bs + r.h * p.lse_hs + r.i] = nan ? NAN : none ? -INFINITY : M + logf(sum);
  }
}

// packed, with at most kFew results of a row (no decode pass among them).
template <typename T, int D>
__global__ void __launch_bounds__(32 * kWarps, 6) merge_few_kernel(const Problem p, const __grid_constant__ Work w) {
  constexpr int kTeams = 128 / D;   // rows that a warp's lanes hold side by side
  const uint32_t rows = (uint32_t)p.B * p.H * p.Sq, per_entry = (uint32_t)p.H * p.Sq;
  const uint32_t row0 = (blockIdx.x * kWarps + threadIdx.x / 32) * (kRowsFew * kTeams) + threadIdx.x % 32 / (D / 4);
  FewRow row[kRowsFew];
  const int* note[kRowsFew];
#pragma unroll
  for (int q = 0; q < kRowsFew; ++q) {
    FewRow& r = row[q];
    const uint32_t id = row0 + q * kTeams;
    r.here = id < rows;
    const uint32_t in = id % per_entry;
    r.b = (int)(id / per_entry);
    r.h = (int)(in / (uint32_t)p.Sq);
    r.i = (int)(in - r.h * (uint32_t)p.Sq);
    note[q] = nullptr;
    const uint32_t g = (uint32_t)r.h / p.qpg, packed = ((uint32_t)r.b * p.Sq + r.i) * p.qpg + r.h - g * p.qpg;
    if (w.note) note[q] = w.note + (r.here ? g * w.blocks + packed / (2 * kRows) : 0);
#pragma unroll
    for (int k = 0; k < kFew; ++k) r.at[k] = (int64_t)id * w.splits + k;   // (by slot, so far)
  }
  paged::wait_for_previous();
  int n_a[kRowsFew];
#pragma unroll
  for (int q = 0; q < kRowsFew; ++q) {
    n_a[q] = note[q] ? *note[q] : w.own_slot;
    row[q].fetch(w, w.splits);
  }
#pragma unroll
  for (int q = 0; q < kRowsFew; ++q) {   // slots that the row does not use count as empty
    row[q].n = row[q].here ? w.splits : 0;
#pragma unroll
    for (int k = 0; k < kFew; ++k)
      if (k >= n_a[q] && k < w.own_slot) row[q].m[k] = -INFINITY, row[q].l[k] = 0.f;
  }
  merge_few<T, D>(p, w, row);
}

// joined, with at most kFew fragments of a unit.
template <typename T, int D>
__global__ void __launch_bounds__(32 * kWarps, 6) join_few_kernel(const Problem p, const __grid_constant__ Work w) {
  constexpr int kTeams = 128 / D, kPer = kWarps * kRowsFew * kTeams;   // rows of a CTA
  const int c = w.list.cut[blockIdx.x / (2 * kRows / kPer)];
  const int local0 =
      blockIdx.x % (2 * kRows / kPer) * kPer + threadIdx.x / 32 * (kRowsFew * kTeams) + threadIdx.x % 32 / (D / 4);
  const int u = w.list.unit[c], n = w.list.frag[c] + 1, c0 = c - w.list.frag[c];
  const int row0 = w.block_of(u, p.B, p.G) * 2 * kRows, g = u % p.G, b = u / p.G % p.B;
  FewRow row[kRowsFew];
#pragma unroll
  for (int q = 0; q < kRowsFew; ++q) {
    FewRow& r = row[q];
    const int local = local0 + q * kTeams;
    r.b = b;
    r.i = (row0 + local) / p.qpg;
    r.h = g * p.qpg + row0 + local - r.i * p.qpg;
    r.here = r.i < p.Sq;
    r.n = r.here ? n : 0;
#pragma unroll
    for (int f = 0; f < kFew; ++f) r.at[f] = ((int64_t)(c0 + f) * 2 + (f == 0 ? 1 : 0)) * (2 * kRows) + local;
  }
  paged::wait_for_previous();
#pragma unroll
  for (int q = 0; q < kRowsFew; ++q) row[q].fetch(w, n);
  merge_few<T, D>(p, w, row);
}

// packed: a row's results are its unit's fragments and then its own keys' (shared.h).
template <typename T, int D, int WARPS>
__global__ void __launch_bounds__(32 * kWarps, 8)
    merge_kernel(const Problem p, const __grid_constant__ Work w, const Cuts cuts) {
  const int64_t row = (int64_t)blockIdx.x * (kWarps / WARPS) + threadIdx.x / 32 / WARPS;
  const int i = (int)(row % p.Sq), h = (int)(row / p.Sq % p.H);
  const int64_t b = row / ((int64_t)p.Sq * p.H);
  const bool here = b < p.B;
  const int64_t r = (b * p.Sq + i) * p.qpg + h % p.qpg;
  const int unit = w.note ? h / p.qpg * w.blocks + (int)(r / (2 * kRows)) : 0;
  const int j = h % p.qpg, u = cuts.note ? h / p.qpg * cuts.n_hc + j / cuts.heads : 0;
  paged::wait_for_previous();
  int n_a = 0, n_b = w.parts_b;
  int64_t first = 0, rest = 0;   // rows of a cut unit's first fragment and of the others
  bool cut = false;
  if (here) {
    n_a = w.note ? w.note[unit] : w.own_slot;
    if (cuts.note) {
      const int2 note = cuts.note[b * p.G * cuts.n_hc + u];
      cut = note.y > 0;
      if (cut) {
        n_b = note.y;
        first = (int64_t)note.x * cuts.heads + j % cuts.heads;
        rest = (int64_t)(note.x / 2) * 2 * cuts.heads + j % cuts.heads;
      }
    }
  }
  // Result k of the row: own ones of a cut unit are in the decode pass's arrays.
  auto own_row = [&](int f) { return f == 0 ? first : rest + (int64_t)f * 2 * cuts.heads; };
  auto kept = [&](int k) { return row * w.splits + (k < n_a ? k : w.own_slot + k - n_a); };
  merge_row<T, D, WARPS>(
      p, here, b, h, i, here ? n_a + n_b : 0,
      [&](int k) { return cut && k >= n_a ? cuts.m[own_row(k - n_a)] : w.part_m[kept(k)]; },
      [&](int k) { return cut && k >= n_a ? cuts.l[own_row(k - n_a)] : w.part_l[kept(k)]; },
      [&](int k, int d) {
        const float* o = cut && k >= n_a ? cuts.o + own_row(k - n_a) * D : w.part_o + kept(k) * D;
        return *reinterpret_cast<const float4*>(o + d);
      });
}

// joined: the fragments of the unit that share c began in the middle of and ends.
template <typename T, int D, int WARPS>
__global__ void __launch_bounds__(32 * kWarps, 8) join_kernel(const Problem p, const __grid_constant__ Work w) {
  constexpr int kPer = kWarps / WARPS;   // rows of a CTA
  const int c = w.list.cut[blockIdx.x / (2 * kRows / kPer)];
  const int local = blockIdx.x % (2 * kRows / kPer) * kPer + threadIdx.x / 32 / WARPS;
  const int u = w.list.unit[c], n = w.list.frag[c] + 1, c0 = c - w.list.frag[c];
  const int row = w.block_of(u, p.B, p.G) * 2 * kRows + local, i = row / p.qpg;
  const int h = u % p.G * p.qpg + row - i * p.qpg;
  const bool here = i < p.Sq;
  if (kPer == 1 && !here) return;   // (all of the CTA's threads)
  paged::wait_for_previous();
  // The first fragment is the last of its share, the others are their shares' first.
  auto at = [&](int f) { return ((int64_t)(c0 + f) * 2 + (f == 0 ? 1 : 0)) * (2 * kRows) + local; };
  merge_row<T, D, WARPS>(
      p, here, u / p.G % p.B, h, i, here ? n : 0, [&](int f) { return w.part_m[at(f)]; },
      [&](int f) { return w.part_l[at(f)]; },
      [&](int f, int d) { return *reinterpret_cast<const float4*>(w.part_o + at(f) * D + d); });
}

template <typename... Args>
cudaError_t launch(void (*kern)(Args...), int64_t blocks, cudaStream_t st, Args... args) {
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)blocks);
  c.blockDim = dim3(32 * kWarps);
  c.stream = st;
  c.attrs = &at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kern, args...);
}

template <typename T, int D>
cudaError_t merge(const Problem& p, const Work& w, const Cuts& cuts, cudaStream_t st) {
  constexpr int kPer = kWarps * kRowsFew * (128 / D);   // rows of a CTA that merges few results of each
  if (w.joined) {
    int most = 0;
    for (int c = 0; c < w.list.ctas; ++c) most = w.list.frag[c] > most ? w.list.frag[c] : most;
    // CTAs for the cut units alone (over all shares: 20 us for 20 units of 256 rows, 7 fragments each, against 6).
    const int64_t rows = (int64_t)w.list.n_cut * 2 * kRows;
    if (most >= 8 && rows <= 16 * kSms) return launch(join_kernel<T, D, 4>, rows, st, p, w);
    if (most >= kFew) return launch(join_kernel<T, D, 1>, rows / kWarps, st, p, w);
    return launch(join_few_kernel<T, D>, (int64_t)w.list.n_cut * 2 * kRows / kPer, st, p, w);
  }
  const int64_t rows = (int64_t)p.B * p.H * p.Sq;
  if (w.splits <= kFew && !cuts.note) return launch(merge_few_kernel<T, D>, (rows + kPer - 1) / kPer, st, p, w);
  if (w.splits > 8 && rows <= 8 * kSms) return launch(merge_kernel<T, D, 4>, rows, st, p, w, cuts);   // while all run at once
  return launch(merge_kernel<T, D, 1>, (rows + kWarps - 1) / kWarps, st, p, w, cuts);
}

}  // namespace
}  // namespace shr

cudaError_t launch_shared_merge(const Problem& p, const shr::Work& w, const paged::Work* own, cudaStream_t st) {
  shr::Cuts cuts{};
  if (own && own->own.note) cuts = {own->part_o, own->part_m, own->part_l, own->own.note, own->heads, own->n_hc};
  if (p.dtype == ATTN_F32)
    return p.D == 64 ? shr::merge<float, 64>(p, w, cuts, st) : shr::merge<float, 128>(p, w, cuts, st);
  if (p.dtype == ATTN_F16)
    return p.D == 64 ? shr::merge<__half, 64>(p, w, cuts, st) : shr::merge<__half, 128>(p, w, cuts, st);
  return p.D == 64 ? shr::merge<__nv_bfloat16, 64>(p, w, cuts, st) : shr::merge<__nv_bfloat16, 128>(p, w, cuts, st);
}

}  // namespace attn
