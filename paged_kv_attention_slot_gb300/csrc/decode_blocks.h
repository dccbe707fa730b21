// Declarations of the calls around decode over selected pages: key bounds, selection, rotary KV write, token map.
#pragma once

#include "divider.cuh"
#include "pkv_internal.h"

namespace pkv {

constexpr int32_t kBlocksMinPage = 8;         // smallest page that has bounds: 2 D bytes beside a key's row
constexpr int32_t kSelectMaxBlocks = 49152;   // pages of the longest request whose scores one CTA's shared memory holds
constexpr int32_t kSelectMaxGroup = 128;      // query heads per KV head: codes of 32767 / 128 levels at least

struct BoundsParams {
  const ReqInfo* req;
  const int32_t* max_page;  // largest entry of kv_indices
  const int32_t* kv_indices;
  const char* k_pool;
  const char* k_sf;  // null unless NVFP4
  int64_t stride_page_b, stride_token_b, stride_head_b;
  int64_t sf_page_b, sf_token_b, sf_head_b;
  int8_t* codes;       // [num_pages, num_kv_heads, 2, head_dim]
  const float* scale;  // [num_kv_heads, head_dim]
  float k_scale;       // of the pool (1 for bf16)
  int64_t pages;       // entries of the page list to look at (last_only: requests)
  uint32_t last_page;  // of the pool
  int32_t* err;        // set by the launcher
  int32_t batch, num_kv_heads, page_size;
  int32_t last_only;   // a page per request, its last one
  int32_t new_only;    // pages that hold a new token
  int32_t shared_page; // the warps of a CTA share a page (set by the launcher)
  Divider by_page;     // set by the launcher
};
cudaError_t launch_key_bounds(BoundsParams p, int dtype, int head_dim, int num_sms, cudaStream_t s);

struct SelectParams {
  const ReqInfo* req;
  const int32_t* max_page;  // largest entry of kv_indices
  const int32_t* kv_indices;
  const void* q;
  const int8_t* codes;
  const float* scale;
  int32_t* blocks;  // [total_tokens, num_kv_heads, num_blocks]
  int32_t num_kv_heads, group, head_dim, page_size;
  int32_t num_blocks, num_sink, num_recent;
  uint32_t last_page;  // that codes has
  int32_t key_cap;  // competing pages that the launch has room for (set by the launcher, as the members behind it)
  Divider by_page;
  int32_t* err;
};
// max_blocks: pages of the longest request
cudaError_t launch_block_select(SelectParams p, int32_t batch, int32_t max_blocks, int num_sms, cudaStream_t s);

cudaError_t launch_rope_store(const pkv_rope_args& a, const pkv_cache& c, float inv_k, float inv_v, cudaStream_t s);
cudaError_t launch_token_map(const ReqInfo* req, const int32_t* kv_indices, int32_t batch, int64_t tokens, int32_t page_size,
                             const int64_t* offsets, int64_t* positions, int64_t* slots, cudaStream_t s);
cudaError_t launch_decode_blocks(const RunParams& p, int kv_dtype, cudaStream_t s);

}  // namespace pkv
