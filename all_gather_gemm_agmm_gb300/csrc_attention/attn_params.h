// attn_params.h -- parameter blocks shared by the host side (attn_api.cpp) and
// the kernels of the attention operators.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace agmm {

constexpr int kMaxHeadDim = 256;
constexpr int kMaxAxes = 4;

struct NormRopeParams {
  const uint16_t* qkv;
  const uint16_t* q_weight;
  const uint16_t* k_weight;
  const void* positions;
  uint16_t* q;
  uint16_t* k;
  uint16_t* k_cache;
  uint16_t* v_cache;
  const int64_t* slots;
  int64_t tokens;
  int64_t qkv_ts, qkv_hs, q_ts, q_hs, k_ts, k_hs;  // token and head strides, elements
  int64_t cache_ps, cache_ts, cache_hs;            // page, place and head strides
  int64_t num_slots, position_axis_stride;
  int q_heads, kv_heads, pairs, page_size;
  int page_shift;  // log2(page_size), or -1
  int adjacent, position64;
  float eps;
  double turns[kMaxHeadDim / 2];      // inv_freq / (2 pi): turns per position
  uint8_t axis[kMaxHeadDim / 2];      // position axis of each pair
};

cudaError_t launch_norm_rope(const NormRopeParams& p, int head_dim, bool f16, cudaStream_t stream);

constexpr int kRows = 128;        // query rows of a tile (MMA M, TMEM lanes)
constexpr int kKeys = 128;        // keys of a tile
constexpr int kMostItems = 1 << 30;  // of a run of prompts
constexpr int kAttnThreads = 384;  // 2 x 4 softmax warps, then producer, MMA and scheduler warps and an idle one

// Workspace: status words and the counter that prompts draw from, which a run that gave
// up leaves somewhere and agmm_query_status zeroes with the words; then a join record
// per CTA and the partial results of split work, which every run writes before it reads.
constexpr size_t kAttnStatusBytes = 256;
constexpr size_t kCounterOffset = 128;
constexpr int kJoinInts = 8;  // 1 (or 0: no join); first tile's token, rows, head; last CTA; second tile's token, rows, head

// One attention problem.  Prompts: packed rows of keys and values.  Trees: a
// paged cache, whose places take the part of the key rows.
struct __align__(128) AttnParams {
  CUtensorMap qmap;  // {head_dim, q_heads, tokens}: a box is 64 columns of one tile's rows
  CUtensorMap kmap;  // {head_dim, tokens or places, kv_heads, pages}: 64 columns of up to 128 rows
  CUtensorMap vmap;
  const uint16_t* q;  // the same again, for plain loads
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* out;
  const int32_t* starts;     // query rows of each sequence (nodes of a tree)
  const int32_t* kv_starts;  // prompts: key rows of each sequence
  const int32_t* context_lens;
  const int32_t* page_table;
  const int64_t* mask;
  int* status;
  int* counter;    // prompts: items drawn
  int* joins;      // [CTAs][kJoinInts]
  float* partial;  // [CTAs][2][rows][head_dim], then [CTAs][2][rows][2] (maximum, sum)
  int64_t tokens, kv_tokens;
  int64_t q_ts, q_hs;        // token and head strides
  int64_t k_ts, k_hs, k_ps;  // token (place), head and page strides
  int64_t v_ts, v_hs, v_ps;
  int64_t out_ts, out_hs;
  int64_t table_stride, table_pages, pages;
  uint64_t wait_limit_cycles;
  int sequences;
  int mask_words, page_shift;
  int q_heads, kv_heads, group;  // group: query heads of a key head
  int pack;                      // heads a tile packs per token: group for trees, 1 for prompts
  int tile_tokens;               // tokens of a row tile: 128 / pack
  int causal, max_nodes;
  int pair_heads;                // prompts: one-tile items have two heads
  int by_draw;                   // prompts: whole items from the counter, no cuts
  int min_tiles;                 // least key tiles of an item on either side of a cut
  int partial_rows;              // rows of a partial slot
  float scale_log2;              // scale * log2(e)
  int test_drop_first_load;      // test hook: the producer skips its first load, so a wait runs out
};

// One instantiation of the kernel, and its shared memory.
struct AttnFn {
  void (*fn)(AttnParams);
  size_t smem;
};
AttnFn prompt_kernel(int head_dim, bool f16);
AttnFn tree_kernel(int head_dim, bool f16);

cudaError_t prepare_attention(const AttnFn& k);
cudaError_t launch_attention(const AttnFn& k, const AttnParams& p, int ctas, cudaStream_t stream);
// Sums the parts of split work, after launch_attention on the same stream.
cudaError_t launch_join(const AttnParams& p, int head_dim, bool f16, int ctas, cudaStream_t stream);

}  // namespace agmm
