// prep.h -- the step before attention: Q/K norms, rotation and cache write.
#pragma once
#include "common.cuh"

namespace attn {
// Checks of a page list that holds `rows` rows an entry (defined in api.cu).
int check_pages(const attn_pages* pages, int64_t rows);
}  // namespace attn
