// prep.cu -- the step before attention in one pass: RMS norms of Q and K for
// each head, rotary position rotation, and the write of K and V into the
// (paged or contiguous, float or int8) cache.
//
// What it computes, for every token and every head row x of Q and K
// ("com.microsoft.GroupQueryAttention" (webgpu-kernels README): rotary
// embedding from cos / sin caches, half-split or interleaved, and RMS norms of
// Q and K for each head):
//   y = x * w / sqrt(sum(x^2) / D + eps),
//   (y_a, y_c) <- (y_a cos - y_c sin, y_c cos + y_a sin)
// for the pairs (a, c) of the first rot_dim elements; V passes through.
// Everything between the loads and the one rounding at the end is float32.
//
// What bounds it: memory.  A row is read once and written once, with about
// seven float operations an element.
#include <math.h>

#include "prep.h"

namespace attn {
namespace {

// A validated attn_prep with its pointers, passed by value to the kernels.
struct Prep {
  int B, S, H, G, D, rot, inter, rows_out, max_pos, norm;
  float eps;
  Layout q, k, v, qo, ko, vo;
  int64_t pos_bs, row_bs;
  const void *Q, *K, *V, *qw, *kw;
  const float *cos, *sin;
  const int32_t *pos, *row;
  void *QO, *KO, *VO;
  const float *k_scale, *v_scale;
  int per_channel;
  int page_size;          // 0: contiguous caches
  uint32_t n_pages;
  const int32_t* table;
  int64_t table_stride;
};

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

__device__ __forceinline__ int64_t clamped_pos(const Prep& p, int b, int i) {
  return clamp64(p.pos ? p.pos[(int64_t)b * p.pos_bs + i] : i, 0, p.max_pos - 1);
}

// The int8 code of x: x / scale rounded to the nearest integer (ties to even)
// and saturated.
__device__ __forceinline__ int8_t code_of(float x, float scale) {
  return (int8_t)fminf(fmaxf(rintf(x / scale), -128.f), 127.f);
}

// One warp per head row, any head_dim, layout and alignment.  Lane j takes the
// pairs j, j + 32, ... of the rotated part and then the other elements; a
// lane reads and writes the same elements, so q_out may be q.
template <typename T, bool KV8>
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
    const int64_t pos = clamped_pos(p, b, i);
    for (int j = lane; j < half; j += 32) {
      const int a = p.inter ? 2 * j : j, c = p.inter ? 2 * j + 1 : j + half;
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

// The vector form: NT = head_dim / (2 N) threads hold a head row, two 16-byte
// chunks of N elements each.  Thread t of a row takes chunks t and t + rot / 2N
// while that is a rotated pair of halves, else chunks 2t and 2t + 1 (pairs of
// the interleaved form, or elements behind the rotated part), so a rotation
// needs no exchange between threads and its N angles load as whole vectors.
// A warp takes up to kSteps groups of 32 / NT head rows of one token, all of
// Q, K or V -- an item: it loads all of them before it computes (the reads in
// flight are what a memory-bound kernel is made of), and the angles and weights
// once.  The grid is what the SMs hold; warps stride over the items.
//
// Measured on two prompts of 8192 tokens (32/8 heads, head_dim 128, bf16, 405
// MB): one warp a row and scalar loads 422 us; this form with one item a warp,
// Q, K and V mixed 121 us; of one kind, packed arithmetic 96 us; striding
// 71.6 us (5.66 TB/s) with 3 groups and 3 CTAs an SM (2 and 4: 74.0, 4 and 2:
// 88).  Three CTAs leave 80 registers a thread, where the f16/bf16 instances
// spill 20 to 36 bytes: with two CTAs and no spills 80.0 against 70.3 us.  Into
// an int8 cache 100.5 us (a division and a rounding an element).  The form of
// one warp a row, which head_dim 80 and 96 take: 404 and 422 us for such prompts.
constexpr int kSteps = 3;
constexpr int kCtasPerSm = 3;

__host__ __device__ __forceinline__ int warps_of(int heads, int per) {
  return ((heads + per - 1) / per + kSteps - 1) / kSteps;
}

template <typename T, int NT, bool KV8, bool INTER>
__global__ void __launch_bounds__(256, kCtasPerSm) prep_vec_kernel(const Prep p) {
  constexpr int N = Vec<T>::N, P = N / 2, kRows = 32 / NT, D = 2 * N * NT;
  const int lane = threadIdx.x % 32, t = lane % NT;
  const uint32_t wq = warps_of(p.H, kRows), wk = warps_of(p.G, kRows), parts = wq + 2 * wk;   // items of a token
  const uint32_t items = (uint32_t)p.B * p.S * parts;
  const int half = p.rot / 2;
  const bool turned = t * N < half;
  const int d0 = (turned && !INTER ? t : 2 * t) * N;
  const int d1 = turned && !INTER ? d0 + half : d0 + N;
  for (uint32_t id = blockIdx.x * 8 + threadIdx.x / 32; id < items; id += gridDim.x * 8) {
    const uint32_t tok = id / parts;
    uint32_t part = id - tok * parts;
    const int b = tok / (uint32_t)p.S, i = tok - b * p.S;
    const int kind = part < wq ? kQ : part < wq + wk ? kK : kV;
    part -= kind == kQ ? 0 : kind == kK ? wq : wq + wk;
    const int heads = kind == kQ ? p.H : p.G;
    const int head0 = part * kSteps * kRows + lane / NT;
    const Layout& li = kind == kQ ? p.q : kind == kK ? p.k : p.v;
    const Layout& lo = kind == kQ ? p.qo : kind == kK ? p.ko : p.vo;
    const T* x = static_cast<const T*>(kind == kQ ? p.Q : kind == kK ? p.K : p.V) + li.off + (int64_t)b * li.bs +
                 (int64_t)head0 * li.hs + (int64_t)i * li.rs;
    void* const out = kind == kQ ? p.QO : kind == kK ? p.KO : p.VO;
    uint4 raw[kSteps][2];
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      raw[s][0] = raw[s][1] = make_uint4(0, 0, 0, 0);
      if (head0 + s * kRows < heads) {
        raw[s][0] = *reinterpret_cast<const uint4*>(x + s * kRows * li.hs + d0);
        raw[s][1] = *reinterpret_cast<const uint4*>(x + s * kRows * li.hs + d1);
      }
    }
    int64_t outer = b, orow = i;
    if (kind != kQ && !cache_slot(p, b, i, outer, orow)) continue;
    const int64_t o = lo.off + outer * lo.bs + (int64_t)head0 * lo.hs + orow * lo.rs;
    if (kind == kV && !KV8) {
      T* y = static_cast<T*>(out) + o;
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
        if (head0 + s * kRows < heads) {
          *reinterpret_cast<uint4*>(y + s * kRows * lo.hs + d0) = raw[s][0];
          *reinterpret_cast<uint4*>(y + s * kRows * lo.hs + d1) = raw[s][1];
        }
      continue;
    }
    float2 cs[P], sn[P];
#pragma unroll
    for (int e = 0; e < P; ++e) {
      cs[e] = make_float2(1.f, 1.f);
      sn[e] = make_float2(0.f, 0.f);
    }
    uint4 rw[2];   // the weights, as stored
    bool weighted = false;
    if (kind != kV) {
      if (turned) {
        const int64_t at = clamped_pos(p, b, i) * half + t * N;
#pragma unroll
        for (int e = 0; e < P; e += 2) {
          const float4 c4 = __ldg(reinterpret_cast<const float4*>(p.cos + at + 2 * e));
          const float4 s4 = __ldg(reinterpret_cast<const float4*>(p.sin + at + 2 * e));
          cs[e] = make_float2(c4.x, c4.y);
          cs[e + 1] = make_float2(c4.z, c4.w);
          sn[e] = make_float2(s4.x, s4.y);
          sn[e + 1] = make_float2(s4.z, s4.w);
        }
      }
      const T* w = static_cast<const T*>(kind == kQ ? p.qw : p.kw);
      weighted = p.norm && w;
      if (weighted) {
        rw[0] = __ldg(reinterpret_cast<const uint4*>(w + d0));
        rw[1] = __ldg(reinterpret_cast<const uint4*>(w + d1));
      }
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
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
        if constexpr (INTER) {   // pairs (2j, 2j + 1) in the thread's 2 N elements: (a, c) cos + (-c, a) sin
#pragma unroll
          for (int e = 0; e < P; ++e) {
            const float ca = e % 2 ? cs[e / 2].y : cs[e / 2].x, sa = e % 2 ? sn[e / 2].y : sn[e / 2].x;
            const float cb = e % 2 ? cs[(P + e) / 2].y : cs[(P + e) / 2].x;
            const float sb = e % 2 ? sn[(P + e) / 2].y : sn[(P + e) / 2].x;
            if (turned) {
              x0[e] = fma2(make_float2(-x0[e].y, x0[e].x), make_float2(sa, sa), mul2(x0[e], make_float2(ca, ca)));
              x1[e] = fma2(make_float2(-x1[e].y, x1[e].x), make_float2(sb, sb), mul2(x1[e], make_float2(cb, cb)));
            }
          }
        } else if (turned) {
#pragma unroll
          for (int e = 0; e < P; ++e) {
            const float2 a = x0[e], c = x1[e];
            x0[e] = fma2(make_float2(-c.x, -c.y), sn[e], mul2(a, cs[e]));
            x1[e] = fma2(a, sn[e], mul2(c, cs[e]));
          }
        }
      }
      if (head0 + s * kRows >= heads) continue;
      if (KV8 && kind != kQ) {
        const int head = head0 + s * kRows;
        const float* sc = (kind == kK ? p.k_scale : p.v_scale) + (p.per_channel ? head * D : 0);
        int8_t* y = static_cast<int8_t*>(out) + o + s * kRows * lo.hs;
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
        T* y = static_cast<T*>(out) + o + s * kRows * lo.hs;
        *reinterpret_cast<uint4*>(y + d0) = Vec<T>::put(x0);
        *reinterpret_cast<uint4*>(y + d1) = Vec<T>::put(x1);
      }
    }
  }
}

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

template <typename T, int NT>
cudaError_t launch_vec(const Prep& p, bool kv8, cudaStream_t st) {
  constexpr int kRows = 32 / NT;
  const int64_t items = (int64_t)p.B * p.S * (warps_of(p.H, kRows) + 2 * warps_of(p.G, kRows));
  const int64_t blocks = (items + 7) / 8;
  const unsigned grid = (unsigned)(blocks < 152 * kCtasPerSm ? blocks : 152 * kCtasPerSm);
  if (p.inter) {
    if (kv8) prep_vec_kernel<T, NT, true, true><<<grid, 256, 0, st>>>(p);
    else prep_vec_kernel<T, NT, false, true><<<grid, 256, 0, st>>>(p);
  } else {
    if (kv8) prep_vec_kernel<T, NT, true, false><<<grid, 256, 0, st>>>(p);
    else prep_vec_kernel<T, NT, false, false><<<grid, 256, 0, st>>>(p);
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_rows(const Prep& p, bool kv8, cudaStream_t st);

template <typename T>
cudaError_t launch(const Prep& p, bool kv8, cudaStream_t st) {
  if (!takes_vec<T>(p, kv8)) return launch_rows<T>(p, kv8, st);
  switch (p.D / (2 * Vec<T>::N)) {
    case 2: return launch_vec<T, 2>(p, kv8, st);
    case 4: return launch_vec<T, 4>(p, kv8, st);
    case 8: return launch_vec<T, 8>(p, kv8, st);
    case 16: return launch_vec<T, 16>(p, kv8, st);
    default:
      if constexpr (Vec<T>::N == 4) return launch_vec<T, 32>(p, kv8, st);   // float32 at head_dim 256
      else return cudaErrorInvalidValue;
  }
}

template <typename T>
cudaError_t launch_rows(const Prep& p, bool kv8, cudaStream_t st) {
  const int64_t n = (int64_t)p.B * p.S * (p.H + 2 * p.G);
  const int64_t blocks = (n + 3) / 4;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  if (kv8)
    prep_row_kernel<T, true><<<(unsigned)blocks, 128, 0, st>>>(p, n);
  else
    prep_row_kernel<T, false><<<(unsigned)blocks, 128, 0, st>>>(p, n);
  return cudaGetLastError();
}

bool layout_ok(const attn_layout& l) {
  return l.offset >= 0 && l.batch_stride >= 0 && l.head_stride >= 0 && l.row_stride >= 0;
}

Layout layout_of(const attn_layout& l) { return {l.offset, l.batch_stride, l.head_stride, l.row_stride}; }

bool off_alignment(const void* ptr, size_t a) { return (uintptr_t)ptr % a != 0; }

int check_prep(const attn_prep* p) {
  if (!p) return ATTN_ERR_INVALID_ARG;
  if (p->batch < 0 || p->seq_len < 0 || p->heads < 1 || p->kv_heads < 1 || p->heads % p->kv_heads)
    return ATTN_ERR_INVALID_ARG;
  if (p->dtype != ATTN_F32 && p->dtype != ATTN_F16 && p->dtype != ATTN_BF16) return ATTN_ERR_INVALID_ARG;
  if (p->head_dim < 1 || p->head_dim > 256 || (p->dtype != ATTN_F32 && (p->head_dim & 1)))
    return ATTN_ERR_INVALID_ARG;
  if (p->rot_dim < 0 || p->rot_dim > p->head_dim || (p->rot_dim & 1)) return ATTN_ERR_INVALID_ARG;
  if ((p->interleaved & ~1) || (p->norm & ~1)) return ATTN_ERR_INVALID_ARG;
  if (!(p->eps >= 0.f) || isinf(p->eps)) return ATTN_ERR_INVALID_ARG;
  if (p->cache_rows < 0 || (p->rot_dim > 0 && p->max_pos < 1)) return ATTN_ERR_INVALID_ARG;
  for (const attn_layout* l : {&p->q, &p->k, &p->v, &p->q_out, &p->k_out, &p->v_out})
    if (!layout_ok(*l)) return ATTN_ERR_INVALID_ARG;
  if (p->pos_batch_stride < 0 || p->row_batch_stride < 0) return ATTN_ERR_INVALID_ARG;
  if (p->kv_dtype != ATTN_KV_AS_Q && p->kv_dtype != ATTN_KV_INT8) return ATTN_ERR_INVALID_ARG;
  if (p->kv_scale_kind != ATTN_KV_SCALE_TENSOR && p->kv_scale_kind != ATTN_KV_SCALE_CHANNEL)
    return ATTN_ERR_INVALID_ARG;
  if (p->kv_dtype == ATTN_KV_INT8) {
    if (!p->k_scale || !p->v_scale) return ATTN_ERR_INVALID_ARG;
    if (off_alignment(p->k_scale, 4) || off_alignment(p->v_scale, 4)) return ATTN_ERR_ALIGNMENT;
  }
  return ATTN_OK;
}

}  // namespace
}  // namespace attn

extern "C" int attn_qkv_prep(const attn_prep* p, const attn_pages* pages, const void* q, const void* k, const void* v,
                             const void* q_weight, const void* k_weight, const float* cos, const float* sin,
                             const int32_t* positions, const int32_t* rows, void* q_out, void* k_out, void* v_out,
                             attn_stream stream) {
  using namespace attn;
  int rc = check_prep(p);
  if (rc) return rc;
  if (pages && (rc = check_pages(pages, p->cache_rows))) return rc;
  if (p->batch == 0 || p->seq_len == 0) return ATTN_OK;
  const size_t es = p->dtype == ATTN_F32 ? 4 : 2, kv_es = p->kv_dtype == ATTN_KV_INT8 ? 1 : es;
  if (!q || !k || !v || !q_out || !k_out || !v_out) return ATTN_ERR_INVALID_ARG;
  if (p->rot_dim > 0 && (!cos || !sin)) return ATTN_ERR_INVALID_ARG;
  if (off_alignment(q, es) || off_alignment(k, es) || off_alignment(v, es) || off_alignment(q_weight, es) ||
      off_alignment(k_weight, es) || off_alignment(q_out, es) || off_alignment(k_out, kv_es) ||
      off_alignment(v_out, kv_es) || off_alignment(cos, 4) || off_alignment(sin, 4) || off_alignment(positions, 4) ||
      off_alignment(rows, 4))
    return ATTN_ERR_ALIGNMENT;
  Prep r;
  r.B = p->batch;
  r.S = p->seq_len;
  r.H = p->heads;
  r.G = p->kv_heads;
  r.D = p->head_dim;
  r.rot = p->rot_dim;
  r.inter = p->interleaved;
  r.rows_out = p->cache_rows;
  r.max_pos = p->max_pos;
  r.norm = p->norm;
  r.eps = p->eps;
  r.q = layout_of(p->q);
  r.k = layout_of(p->k);
  r.v = layout_of(p->v);
  r.qo = layout_of(p->q_out);
  r.ko = layout_of(p->k_out);
  r.vo = layout_of(p->v_out);
  r.pos_bs = p->pos_batch_stride;
  r.row_bs = p->row_batch_stride;
  r.Q = q;
  r.K = k;
  r.V = v;
  r.qw = q_weight;
  r.kw = k_weight;
  r.cos = cos;
  r.sin = sin;
  r.pos = positions;
  r.row = rows;
  r.QO = q_out;
  r.KO = k_out;
  r.VO = v_out;
  r.k_scale = p->k_scale;
  r.v_scale = p->v_scale;
  r.per_channel = p->kv_scale_kind == ATTN_KV_SCALE_CHANNEL;
  r.page_size = pages ? pages->page_size : 0;
  r.n_pages = pages ? (uint32_t)pages->n_pages : 0u;
  r.table = pages ? pages->table : nullptr;
  r.table_stride = pages ? pages->table_stride : 0;
  const bool kv8 = p->kv_dtype == ATTN_KV_INT8;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = p->dtype == ATTN_F32   ? launch<float>(r, kv8, st)
                        : p->dtype == ATTN_F16 ? launch<__half>(r, kv8, st)
                                               : launch<__nv_bfloat16>(r, kv8, st);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}
