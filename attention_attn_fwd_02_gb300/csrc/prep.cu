// prep.cu -- the step before attention: argument checks, and the instances with
// one position a token (prep.cuh).
#include "prep.cuh"

namespace attn {
namespace {

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

namespace attn {
namespace {

// attn_qkv_prep (axes null) and attn_qkv_prep_axes.
int prep_impl(const attn_prep* p, const attn_pages* pages, const attn_axes* axes, const void* q, const void* k,
              const void* v, const void* q_weight, const void* k_weight, const float* cos, const float* sin,
              const int32_t* positions, const int32_t* rows, void* q_out, void* k_out, void* v_out,
              attn_stream stream) {
  int rc = check_prep(p);
  if (rc) return rc;
  if (axes) {
    if (axes->n_axes < 1 || axes->n_axes > ATTN_MAX_AXES || axes->pos_axis_stride < 0) return ATTN_ERR_INVALID_ARG;
    for (int j = 0; j < p->rot_dim / 2; ++j)
      if (axes->axis[j] >= axes->n_axes) return ATTN_ERR_INVALID_ARG;
  }
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
  r.n_axes = axes ? axes->n_axes : 1;
  r.axis_stride = axes ? axes->pos_axis_stride : 0;
  memset(r.axis, 0, sizeof r.axis);
  if (axes) memcpy(r.axis, axes->axis, p->rot_dim / 2);
  const bool kv8 = p->kv_dtype == ATTN_KV_INT8;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // (one axis is one position a token)
  const cudaError_t e = r.n_axes > 1 ? prep_axes(r, kv8, p->dtype, st) : launch_prep<false>(r, kv8, p->dtype, st);
  return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

}  // namespace
}  // namespace attn

extern "C" int attn_qkv_prep(const attn_prep* p, const attn_pages* pages, const void* q, const void* k, const void* v,
                             const void* q_weight, const void* k_weight, const float* cos, const float* sin,
                             const int32_t* positions, const int32_t* rows, void* q_out, void* k_out, void* v_out,
                             attn_stream stream) {
  return attn::prep_impl(p, pages, nullptr, q, k, v, q_weight, k_weight, cos, sin, positions, rows, q_out, k_out,
                         v_out, stream);
}

extern "C" int attn_qkv_prep_axes(const attn_prep* p, const attn_pages* pages, const attn_axes* axes, const void* q,
                                  const void* k, const void* v, const void* q_weight, const void* k_weight,
                                  const float* cos, const float* sin, const int32_t* positions, const int32_t* rows,
                                  void* q_out, void* k_out, void* v_out, attn_stream stream) {
  if (!axes) return ATTN_ERR_INVALID_ARG;
  return attn::prep_impl(p, pages, axes, q, k, v, q_weight, k_weight, cos, sin, positions, rows, q_out, k_out, v_out,
                         stream);
}
