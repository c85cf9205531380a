// Host interface of the tree attention kernels: what tl_tree_attention checks
// and what a context's speculation passes directly.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/tl.h"

namespace tl {

struct TreeAttnArgs {
  const void* q;
  int64_t q_stride;
  const int32_t* table;      // [R][max_pages]
  int32_t max_pages;
  const int32_t* ctx;
  const int32_t* cu;
  int32_t R, n_rows, H, Hk, max_nodes;
  const uint32_t* masks;
  int32_t words;
  float scale_log2;          // softmax scale times log2(e)
  void* out;
  int32_t out_f32;
  int64_t out_stride;
  float* lse;
  __half* out16;             // NULL, or a second copy of fp32 outputs as the projections take it (act16_put)
  int32_t split16;
  int64_t n_pages;
  int32_t page_shift;
  char* ws;
  int32_t* status;
};

// Checked arguments (as tl_tree_attention documents); pool describes the cache.
int tree_attn_run(TreeAttnArgs a, const tl_kv_pool& pool, cudaStream_t s, int64_t* launches = nullptr);

size_t tree_attn_workspace(int hd, int64_t rows_per_head, int n_sms);

}  // namespace tl
