// Host interface of the tree kernels for a context's own passes: what the
// public calls check and pass on, and what tl_speculate_tree passes directly.
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
  int32_t node0;             // R = 1: the rows are nodes node0, node0 + 1, ... of a tree whose earlier nodes are cached
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
  int32_t max_sms;           // 0, or the SMs that the workspace is for
  int32_t* status;
};

// Rotation and append of projection rows [q | k | v] (fp32, every head its own
// keys) to one cache slot of a lane: slots[row] is a position, map the pages of
// the cache slot.  Queries go to q_out in fp16.
int norm_rope_lane(const float* qkv, int64_t rows, int32_t n_heads, const float2* table, int32_t length,
                   const int32_t* positions, const int64_t* slots, const tl_kv_pool& pool, const int32_t* map,
                   int32_t map_pages, __half* q_out, int32_t* status, cudaStream_t s);

// Checked arguments (as tl_tree_attention documents); pool describes the cache.
int tree_attn_run(TreeAttnArgs a, const tl_kv_pool& pool, cudaStream_t s, int64_t* launches = nullptr);

size_t tree_attn_workspace(int hd, int64_t rows_per_head, int n_sms);

}  // namespace tl
