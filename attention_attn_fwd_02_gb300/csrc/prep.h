// prep.h -- the step before attention: Q/K norms, rotation and cache write.
#pragma once
#include "common.cuh"

namespace attn {

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
  int n_axes;             // 1: one position a token
  int64_t axis_stride;    // of the positions
  uint8_t axis[128];      // of each rotated pair
};

// Enqueue the step with positions on several axes (prep_axes_*.cu).
cudaError_t prep_axes_f32(const Prep& p, bool kv8, cudaStream_t st);
cudaError_t prep_axes_f16(const Prep& p, bool kv8, cudaStream_t st);
cudaError_t prep_axes_bf16(const Prep& p, bool kv8, cudaStream_t st);

// Checks of a page list that holds `rows` rows an entry (defined in api.cu).
int check_pages(const attn_pages* pages, int64_t rows);

}  // namespace attn
