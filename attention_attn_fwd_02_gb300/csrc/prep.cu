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
  const cudaError_t e = p->dtype == ATTN_F32   ? launch_rows<float>(r, kv8, st)
                        : p->dtype == ATTN_F16 ? launch_rows<__half>(r, kv8, st)
                                               : launch_rows<__nv_bfloat16>(r, kv8, st);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}
