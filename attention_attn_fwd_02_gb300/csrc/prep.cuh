// prep.cuh -- the step before attention in one pass: RMS norms of Q and K for
// each head, rotary position rotation, and the write of K and V into the
// (paged or contiguous, float or int8) cache.  Here is what the vector forms of
// prep.cu (one position a token) and prep_axes.cuh (one on each axis) share, and the form
// of one warp a row that both fall back to.
//
// What it computes, for every token and every head row x of Q and K
// ("com.microsoft.GroupQueryAttention" (webgpu-kernels README): rotary
// embedding from cos / sin caches, half-split or interleaved, and RMS norms of
// Q and K for each head):
//   y = x * w / sqrt(sum(x^2) / D + eps),
//   (y_a, y_c) <- (y_a cos - y_c sin, y_c cos + y_a sin)
// for the pairs (a, c) of the first rot_dim elements; V passes through.  With
// axes, pair j takes its angle at the token's position on axis j's axis.
// Everything between the loads and the one rounding at the end is float32.
//
// What bounds it: memory.  A row is read once and written once, with about
// seven float operations an element.
#pragma once

#include <math.h>
#include <string.h>

#include "prep.h"

namespace attn {
namespace {

enum { kQ = 0, kK = 1, kV = 2 };

// Which of Q, K, V the head row r of a token is, and its head.
__device__ __forceinline__ int row_kind(const Prep& p, int r, int& head) {
  if (r < p.H) {
    head = r;
    return kQ;
  }
  if (r < p.H + p.G) {
    head = r - p.H;
    return kK;
  }
  head = r - p.H - p.G;
  return kV;
}

// Where token (b, i)'s rows go in the cache: the batch (or page) index and the
// row in it.  False when the token writes no K and V.
__device__ __forceinline__ bool cache_slot(const Prep& p, int b, int i, int64_t& outer, int64_t& row) {
  const int64_t r = p.row ? p.row[(int64_t)b * p.row_bs + i] : i;
  if (r < 0 || r >= p.rows_out) return false;
  outer = b;
  row = r;
  if (p.page_size) {
    const int32_t pg = p.table[(int64_t)b * p.table_stride + r / p.page_size];
    if ((uint32_t)pg >= p.n_pages) return false;
    outer = pg;
    row = r % p.page_size;
  }
  return true;
}

__device__ __forceinline__ int64_t clamped_pos(const Prep& p, int b, int i, int axis = 0) {
  return clamp64(p.pos ? p.pos[axis * p.axis_stride + (int64_t)b * p.pos_bs + i] : i, 0, p.max_pos - 1);
}

// The int8 code of x: x / scale rounded to the nearest integer (ties to even)
// and saturated.
__device__ __forceinline__ int8_t code_of(float x, float scale) {
  return (int8_t)fminf(fmaxf(rintf(x / scale), -128.f), 127.f);
}

// One warp per head row, any head_dim, layout and alignment.  Lane j takes the
// pairs j, j + 32, ... of the rotated part and then the other elements; a
// lane reads and writes the same elements, so q_out may be q.
template <typename T, bool KV8, bool AXES>
__global__ void __launch_bounds__(128) prep_row_kernel(const Prep p, const int64_t n_rows) {
  const int64_t id = (int64_t)blockIdx.x * 4 + threadIdx.x / 32;
  const int lane = threadIdx.x % 32;
  if (id >= n_rows) return;
  const int rows = p.H + 2 * p.G;
  const int64_t tok = id / rows;
  const int b = (int)(tok / p.S), i = (int)(tok % p.S);
  int head;
  const int kind = row_kind(p, (int)(id % rows), head);
  int64_t outer = b, orow = i;
  if (kind != kQ && !cache_slot(p, b, i, outer, orow)) return;
  const Layout& li = kind == kQ ? p.q : kind == kK ? p.k : p.v;
  const Layout& lo = kind == kQ ? p.qo : kind == kK ? p.ko : p.vo;
  const T* x = static_cast<const T*>(kind == kQ ? p.Q : kind == kK ? p.K : p.V) + li.off + b * li.bs + head * li.hs +
               i * li.rs;
  const int64_t o = lo.off + outer * lo.bs + head * lo.hs + orow * lo.rs;
  void* const out = kind == kQ ? p.QO : kind == kK ? p.KO : p.VO;
  const float* scale = kind == kK ? p.k_scale : p.v_scale;
  auto put = [&](int d, float y) {
    if (KV8 && kind != kQ)
      static_cast<int8_t*>(out)[o + d] = code_of(y, scale[p.per_channel ? head * p.D + d : 0]);
    else
      static_cast<T*>(out)[o + d] = from_f32<T>(y);
  };
  if (kind == kV) {
    for (int d = lane; d < p.D; d += 32) put(d, to_f32(x[d]));
    return;
  }
  float rs = 1.f;
  if (p.norm) {
    float ss = 0.f;
    for (int d = lane; d < p.D; d += 32) ss = fmaf(to_f32(x[d]), to_f32(x[d]), ss);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    rs = 1.f / sqrtf(ss / (float)p.D + p.eps);
  }
  const T* w = p.norm ? static_cast<const T*>(kind == kQ ? p.qw : p.kw) : nullptr;
  auto get = [&](int d) { return to_f32(x[d]) * rs * (w ? to_f32(w[d]) : 1.f); };
  const int half = p.rot / 2;
  if (half > 0) {
    const int64_t one = AXES ? 0 : clamped_pos(p, b, i);
    for (int j = lane; j < half; j += 32) {
      const int a = p.inter ? 2 * j : j, c = p.inter ? 2 * j + 1 : j + half;
      const int64_t pos = AXES ? clamped_pos(p, b, i, p.axis[j]) : one;
      const float cs = p.cos[pos * half + j], sn = p.sin[pos * half + j];
      const float ya = get(a), yc = get(c);
      put(a, ya * cs - yc * sn);
      put(c, yc * cs + ya * sn);
    }
  }
  for (int d = p.rot + lane; d < p.D; d += 32) put(d, get(d));
}

// Pairs of floats in one 64-bit register, as the packed instructions take them.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\t"
      "mul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}

// 16 bytes of T as pairs of floats, and back.
template <typename T>
struct Vec;
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void get(const uint4& u, float2 (&x)[2]) {
    x[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
    x[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
  }
  static __device__ __forceinline__ uint4 put(const float2 (&x)[2]) {
    return make_uint4(__float_as_uint(x[0].x), __float_as_uint(x[0].y), __float_as_uint(x[1].x),
                      __float_as_uint(x[1].y));
  }
};
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(const uint4& u, float2 (&x)[4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  static __device__ __forceinline__ uint4 put(const float2 (&x)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[i].x, x[i].y);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec<__half> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(const uint4& u, float2 (&x)[4]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
  }
  static __device__ __forceinline__ uint4 put(const float2 (&x)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(x[i].x, x[i].y);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// Whether a strided view takes accesses of `bytes` bytes: its start and the
// strides that are used (their extents exceed 1) are multiples.
bool vec_ok(const void* base, const Layout& l, int64_t outer, int heads, int64_t rows, int es, int bytes) {
  auto ok = [=](int64_t stride, int64_t extent) { return extent <= 1 || stride * es % bytes == 0; };
  return ((uintptr_t)base + (uintptr_t)l.off * es) % bytes == 0 && ok(l.bs, outer) && ok(l.hs, heads) &&
         ok(l.rs, rows);
}

// The vector form wants whole chunks on both sides of a rotated pair, and aligned views.
template <typename T>
bool takes_vec(const Prep& p, bool kv8) {
  constexpr int N = Vec<T>::N;
  const int nt = p.D / (2 * N);
  if (p.D % (2 * N) || nt < 2 || nt > 32 || (nt & (nt - 1)) || (p.rot / 2) % N) return false;
  const int es = sizeof(T), ces = kv8 ? 1 : es;
  const int64_t outer = p.page_size ? p.n_pages : p.B, orows = p.page_size ? p.page_size : p.rows_out;
  return vec_ok(p.Q, p.q, p.B, p.H, p.S, es, 16) && vec_ok(p.K, p.k, p.B, p.G, p.S, es, 16) &&
         vec_ok(p.V, p.v, p.B, p.G, p.S, es, 16) && vec_ok(p.QO, p.qo, p.B, p.H, p.S, es, 16) &&
         vec_ok(p.KO, p.ko, outer, p.G, orows, ces, N * ces) && vec_ok(p.VO, p.vo, outer, p.G, orows, ces, N * ces) &&
         (uintptr_t)p.qw % 16 == 0 && (uintptr_t)p.kw % 16 == 0 && (uintptr_t)p.cos % 16 == 0 &&
         (uintptr_t)p.sin % 16 == 0 && (int64_t)p.B * p.S * (p.H + 2 * p.G) < 0x40000000;
}

template <typename T, bool AXES>
cudaError_t launch_rows(const Prep& p, bool kv8, cudaStream_t st) {
  const int64_t n = (int64_t)p.B * p.S * (p.H + 2 * p.G);
  const int64_t blocks = (n + 3) / 4;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  if (kv8)
    prep_row_kernel<T, true, AXES><<<(unsigned)blocks, 128, 0, st>>>(p, n);
  else
    prep_row_kernel<T, false, AXES><<<(unsigned)blocks, 128, 0, st>>>(p, n);
  return cudaGetLastError();
}

}  // namespace
}  // namespace attn
