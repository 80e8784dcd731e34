/*
 * agmm_attention.h -- C ABI of the operators behind a column-parallel QKV
 * product (agmm.h): head norms with rotary positions, attention of packed
 * prompts, and attention of drafted tokens over a paged cache.
 *
 * Types: every matrix is bf16 (AGMM_BF16) or fp16 (AGMM_F16), fixed by the
 * plan; sums, softmax statistics and norms are held in float32 and rounded
 * once, to the nearest, at the output.  The weights of a softmax are rounded to
 * that type too, as an operand of the tensor cores, and summed as they are
 * rounded; in fp16 as numbers 2^7 times as large, so that a weight of 2^-21 of
 * its row's largest has all its bits, and one of 2^-32 still counts.
 *
 * Strides count elements; the innermost (head_dim) stride is 1.  Data
 * pointers are 16-byte aligned and strides are multiples of 8 elements
 * (16 bytes), else AGMM_ERR_ALIGNMENT.  Grouped heads: query head h reads
 * key/value head h / (q_heads / kv_heads).
 *
 * Ownership, streams, errors: as in agmm.h.  The caller owns every buffer;
 * runs are asynchronous on the given stream; every call returns a status and
 * nothing throws; agmm_last_error() has the detail.  A plan holds no device
 * memory, belongs to the device that was current when it was made, and may be
 * used by several host threads at once.  A workspace is zero-filled before
 * its first use, and runs that overlap on the device need one each; its status
 * words are read with agmm_query_status(NULL, workspace, stream), which
 * reports a device-side wait that ran out: the results since the last query are
 * then not valid, and the query leaves the workspace ready for its next use.  A
 * call with nothing to do (no tokens) returns AGMM_OK and launches nothing.
 *
 * Values in device memory (starts, lengths, page numbers, slots) are not read
 * by the host.  The kernels bound them: starts are clamped to the tokens there
 * are (where they fall, a sequence is empty; when they stand for 2^30 tiles of
 * work or more so, prompts are not worked on), lengths to what the page table
 * covers, a page number outside the cache reads zeros, and a slot outside the
 * cache is not written.
 */
#ifndef AGMM_ATTENTION_H_
#define AGMM_ATTENTION_H_

#include "agmm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---------------------------------------------------------------- norm_rope
 *
 * For each token t and each query or key head x (head_dim values):
 *     y = x / sqrt(mean(x^2) + eps) * weight       (weight NULL: y = x)
 *     angle_i = positions[axis_of_pair[i]][t] * inv_freq[i],  i < rotary_dim / 2
 *     (a, b) -> (a cos - b sin, b cos + a sin)
 * where (a, b) are y's values (i, i + rotary_dim / 2), or (2i, 2i + 1) when
 * `adjacent` is set; values from rotary_dim on are not rotated.  Angles are
 * reduced in float64, so far positions lose nothing.
 */
typedef struct {
  int q_heads, kv_heads;
  int head_dim;            /* 64, 128 or 256                                   */
  int rotary_dim;          /* a multiple of 16, 0..head_dim                    */
  int adjacent;            /* 0: pairs (i, i + rotary_dim / 2); 1: (2i, 2i + 1) */
  int axes;                /* position axes, 1..4                              */
  agmm_dtype_t dtype;      /* AGMM_BF16 or AGMM_F16                            */
  float eps;               /* >= 0                                             */
  const double* inv_freq;  /* host, rotary_dim / 2 radians per position        */
  const int* axis_of_pair; /* host, rotary_dim / 2 axes; NULL: all axis 0      */
} agmm_norm_rope_desc_t;

typedef struct {
  int64_t tokens;
  const void* qkv;             /* [tokens, q_heads + 2 kv_heads, head_dim]: queries, keys, values */
  int64_t qkv_token_stride, qkv_head_stride;
  const void* q_weight;        /* [head_dim] in the plan's type; both NULL: no norm        */
  const void* k_weight;
  const void* positions;       /* [axes, tokens] of int32 or int64                          */
  int64_t position_bytes;      /* 4 or 8                                                    */
  int64_t position_axis_stride;
  void* q;                     /* out [tokens, q_heads, head_dim]; may be qkv's own queries */
  int64_t q_token_stride, q_head_stride;
  void* k;                     /* out [tokens, kv_heads, head_dim] or NULL; may be qkv's own keys */
  int64_t k_token_stride, k_head_stride;
  void* k_cache;               /* [pages, page_size, kv_heads, head_dim] or NULL            */
  void* v_cache;               /* the same shape and strides; NULL with k_cache             */
  int64_t pages, page_size;
  int64_t cache_page_stride, cache_token_stride, cache_head_stride;
  const int64_t* slots;        /* [tokens]: page * page_size + place; outside the cache: not written */
} agmm_norm_rope_args_t;

typedef struct agmm_norm_rope_s* agmm_norm_rope_t;

agmm_status_t agmm_norm_rope_plan(const agmm_norm_rope_desc_t* desc, agmm_norm_rope_t* out_plan);
agmm_status_t agmm_norm_rope_run(agmm_norm_rope_t plan, const agmm_norm_rope_args_t* args, void* stream);
void agmm_norm_rope_destroy(agmm_norm_rope_t plan);

/* ------------------------------------------------------------------- prompt
 *
 * Sequence s has the query rows [starts[s], starts[s+1]) and the key/value
 * rows [kv_starts[s], kv_starts[s+1]).  With n and m of them, query row i sees
 * key rows j <= i + m - n (causal: the last query sees the last key) or all
 * (not causal):
 *     out_i = sum_j softmax_j(scale * q_i . k_j) v_j
 * A row that sees no key is zero.  A key or value row that no row of a
 * 128-row tile sees, or that lies outside the sequence, is never used, whatever
 * it holds; a non-finite value in a row that some rows see reaches those only.
 * (The others of its tile are then computed again one by one, in time that grows
 * with their keys: 54 ms for 8000.  That is not a wait that runs out.)
 */
typedef struct {
  int q_heads, kv_heads; /* q_heads a multiple of kv_heads */
  int head_dim;          /* 64 or 128                      */
  int causal;
  agmm_dtype_t dtype;    /* AGMM_BF16 or AGMM_F16          */
  float scale;           /* > 0                            */
} agmm_prompt_desc_t;

typedef struct {
  int64_t tokens, kv_tokens, sequences; /* up to 2^31 - 4097 rows, 2^20 sequences */
  const void* q;             /* [tokens, q_heads, head_dim]     */
  int64_t q_token_stride, q_head_stride;
  const void* k;             /* [kv_tokens, kv_heads, head_dim] */
  int64_t k_token_stride, k_head_stride;
  const void* v;             /* [kv_tokens, kv_heads, head_dim] */
  int64_t v_token_stride, v_head_stride;
  void* out;                 /* [tokens, q_heads, head_dim]     */
  int64_t out_token_stride, out_head_stride;
  const int32_t* starts;     /* [sequences + 1], not falling    */
  const int32_t* kv_starts;  /* [sequences + 1]; NULL: starts   */
  void* workspace;
} agmm_prompt_args_t;

typedef struct agmm_prompt_s* agmm_prompt_t;

agmm_status_t agmm_prompt_plan(const agmm_prompt_desc_t* desc, agmm_prompt_t* out_plan);
size_t agmm_prompt_workspace_bytes(agmm_prompt_t plan);
agmm_status_t agmm_prompt_run(agmm_prompt_t plan, const agmm_prompt_args_t* args, void* stream);
void agmm_prompt_destroy(agmm_prompt_t plan);

/* --------------------------------------------------------------------- tree
 *
 * Sequence s has context_lens[s] tokens in the cache and, at the places after
 * them, the keys and values of its drafted tokens (nodes) [node_starts[s],
 * node_starts[s+1]).  Place p of a sequence is row p % page_size of page
 * page_table[s][p / page_size].  Node i (counted in its sequence) sees the
 * whole context and the nodes j whose bit is set: bit j % 64 of word j / 64 of
 * its mask row; without a mask it sees the nodes up to itself.  One node
 * without a mask is the ordinary decode step.  A node that sees nothing is
 * zero.  max_nodes bounds a sequence's nodes: nodes past it are not computed, but
 * a mask may let others see them.
 */
typedef struct {
  int q_heads, kv_heads; /* q_heads a multiple of kv_heads, at most 128 heads to a group */
  int head_dim;          /* 64 or 128                              */
  int page_size;         /* a power of two, 8..256                 */
  int max_nodes;         /* 1..1024                                */
  agmm_dtype_t dtype;    /* AGMM_BF16 or AGMM_F16                  */
  float scale;           /* > 0                                    */
} agmm_tree_desc_t;

typedef struct {
  int64_t tokens, sequences;    /* drafted tokens of all sequences          */
  const void* q;                /* [tokens, q_heads, head_dim]              */
  int64_t q_token_stride, q_head_stride;
  const void* k_cache;          /* [pages, page_size, kv_heads, head_dim]   */
  const void* v_cache;          /* the same shape and strides               */
  int64_t pages, cache_page_stride, cache_token_stride, cache_head_stride;
  const int32_t* page_table;    /* [sequences, table_pages]                 */
  int64_t table_pages;          /* pages a sequence can have, up to 2^31 - 4097 places */
  int64_t table_stride;         /* entries from one sequence to the next    */
  const int32_t* context_lens;  /* [sequences]                              */
  const int32_t* node_starts;   /* [sequences + 1], not falling             */
  const int64_t* mask;          /* [tokens, mask_words] or NULL             */
  int64_t mask_words;
  void* out;                    /* [tokens, q_heads, head_dim]              */
  int64_t out_token_stride, out_head_stride;
  void* workspace;
} agmm_tree_args_t;

typedef struct agmm_tree_s* agmm_tree_t;

agmm_status_t agmm_tree_plan(const agmm_tree_desc_t* desc, agmm_tree_t* out_plan);
size_t agmm_tree_workspace_bytes(agmm_tree_t plan);
agmm_status_t agmm_tree_run(agmm_tree_t plan, const agmm_tree_args_t* args, void* stream);
void agmm_tree_destroy(agmm_tree_t plan);

#ifdef __cplusplus
}
#endif

#endif /* AGMM_ATTENTION_H_ */
