/*
 * agmm_feedforward.h -- C ABI of the feed-forward half of a transformer block
 * around the gathered product (agmm.h): layer norm, the gated product, and the
 * product with bias, activation and residual, each with its backward pass.
 *
 * Types: every matrix is bf16 (AGMM_BF16) or fp16 (AGMM_F16), fixed by the
 * plan; sums, statistics and activations are held in float32 and rounded once,
 * to the nearest, at the output.  Two more roundings to that type are part of
 * the backward passes: of what the forward pass saves (gate, up, pre), unless the
 * plan has it in float32 (agmm_gated_save_float, agmm_linear_save_float), and of
 * the gradients that the tensor cores multiply (d_gate, d_up, d_pre).  An fp16
 * value past 65504 is infinite there, as in any output.
 *
 * Rows of X come as for agmm_run: `shards` separate buffers of `rows` rows,
 * 1..8 of them; one buffer of all rows is one shard.  All other matrices with a
 * row for each token have shards * rows rows, in the order of the shards.  A
 * weight is stored [k, n], or [n, k] with rhs_transpose, and its gradient alike.
 *
 * Strides count elements from one row to the next, 2^29 at most; rows are
 * contiguous and do not overlap.  Pointers are 16-byte aligned, and strides, k, n and columns are
 * multiples of 8, else AGMM_ERR_ALIGNMENT (k, n, columns: AGMM_ERR_INVALID_ARG).
 * An output must not overlap an input, but where it is said that it may.
 *
 * Activations a(z): none, relu, silu z / (1 + e^-z), gelu z Phi(z), and gelu_tanh
 * z / 2 (1 + tanh(sqrt(2 / pi) (z + 0.044715 z^3))).
 *
 * Ownership, streams, errors: as in agmm.h.  The caller owns every buffer; runs
 * are asynchronous on the given stream; every call returns a status and nothing
 * throws; agmm_last_error() has the detail.  A plan holds no device memory,
 * belongs to the device that was current when it was made, and may be used by
 * several host threads at once.  The first AGMM_FEEDFORWARD_HEAD_BYTES of a
 * workspace are zero-filled before its first use, and runs that overlap on the
 * device need one each.  Its status words are read with agmm_query_status(NULL,
 * workspace, stream); after that has reported a device-side wait that ran out,
 * the results since the last query are not valid and those bytes are zero-filled
 * again before the next use.  A call
 * without tokens writes nothing, but gradients of weights, which are then zero.
 * Results do not depend on the order in which the GPU does the work.
 */
#ifndef AGMM_FEEDFORWARD_H_
#define AGMM_FEEDFORWARD_H_

#include "agmm.h"

#ifdef __cplusplus
extern "C" {
#endif

#define AGMM_FEEDFORWARD_HEAD_BYTES 65536

typedef enum {
  AGMM_ACT_NONE = 0,
  AGMM_ACT_RELU = 1,
  AGMM_ACT_SILU = 2,
  AGMM_ACT_GELU = 3,
  AGMM_ACT_GELU_TANH = 4
} agmm_activation_t;

/* --------------------------------------------------------------- layer_norm
 *
 * For each row x of `columns` values:
 *     mean = sum(x) / columns,  rstd = 1 / sqrt(sum((x - mean)^2) / columns + eps)
 *     out = (x - mean) * rstd * weight + bias      (weight NULL: 1, bias NULL: 0)
 * and backwards, with g = d_out * weight and xhat = (x - mean) * rstd:
 *     dx = rstd * (g - sum(g) / columns - xhat * sum(g * xhat) / columns) + add
 *     d_weight = sum over rows of d_out * xhat,  d_bias = sum over rows of d_out
 */
typedef struct {
  int columns;        /* a multiple of 8, 8..16384 */
  agmm_dtype_t dtype; /* AGMM_BF16 or AGMM_F16     */
  float eps;          /* >= 0                      */
} agmm_layer_norm_desc_t;

typedef struct {
  int64_t rows;       /* up to 2^31 - 1                                */
  const void* x;      /* [rows, columns]                               */
  int64_t x_stride;
  const void* weight; /* [columns] or NULL                             */
  const void* bias;   /* [columns] or NULL                             */
  void* out;          /* [rows, columns]; may be x                     */
  int64_t out_stride;
  float* mean;        /* out, [rows] or NULL: what the backward pass   */
  float* rstd;        /* reads                                         */
} agmm_layer_norm_args_t;

typedef struct {
  int64_t rows;
  const void* d_out;  /* [rows, columns]                               */
  int64_t d_out_stride;
  const void* x;      /* [rows, columns], as the forward pass had it   */
  int64_t x_stride;
  const float* mean;  /* [rows]                                        */
  const float* rstd;  /* [rows]                                        */
  const void* weight; /* [columns] or NULL                             */
  const void* add;    /* [rows, columns] or NULL: added to dx          */
  int64_t add_stride;
  void* dx;           /* [rows, columns] or NULL; may be d_out or add  */
  int64_t dx_stride;
  void* d_weight;     /* [columns] or NULL                             */
  void* d_bias;       /* [columns] or NULL                             */
  int64_t f32_grads;  /* d_weight and d_bias are float32               */
  void* workspace;
} agmm_layer_norm_grad_args_t;

typedef struct agmm_layer_norm_s* agmm_layer_norm_t;

agmm_status_t agmm_layer_norm_plan(const agmm_layer_norm_desc_t* desc, agmm_layer_norm_t* out_plan);
size_t agmm_layer_norm_workspace_bytes(agmm_layer_norm_t plan);
agmm_status_t agmm_layer_norm_run(agmm_layer_norm_t plan, const agmm_layer_norm_args_t* args, void* stream);
agmm_status_t agmm_layer_norm_backward(agmm_layer_norm_t plan, const agmm_layer_norm_grad_args_t* args, void* stream);
void agmm_layer_norm_destroy(agmm_layer_norm_t plan);

/* -------------------------------------------------------------------- gated
 *
 *     gate = X Wgate,  up = X Wup,  out = a(gate) * up
 * in one kernel; gate and up are written (rounded) when they are asked for.
 * Backwards, from those:
 *     d_gate = d_out * up * a'(gate),  d_up = d_out * a(gate)
 *     dx = d_gate Wgate^T + d_up Wup^T,  dw_gate = X^T d_gate,  dw_up = X^T d_up
 */
typedef struct {
  int k, n;                     /* multiples of 8, 8..2^20          */
  agmm_activation_t activation; /* not AGMM_ACT_NONE                */
  int rhs_transpose;            /* weights stored [n, k]            */
  agmm_dtype_t dtype;           /* AGMM_BF16 or AGMM_F16            */
} agmm_gated_desc_t;

typedef struct {
  int64_t shards, rows;    /* shards * rows up to 2^31 - 1024       */
  const void* x[8];        /* [rows, k] each                        */
  int64_t x_stride;
  const void* w_gate;
  const void* w_up;        /* may be halves of one tensor           */
  int64_t w_stride;
  void* out;               /* [shards * rows, n]                    */
  int64_t out_stride;
  void* gate;              /* out, [shards * rows, n]; both or none */
  void* up;
  int64_t saved_stride;
  void* workspace;
} agmm_gated_args_t;

typedef struct {
  int64_t shards, rows;
  const void* x[8];        /* read for dw_gate and dw_up            */
  int64_t x_stride;
  const void* w_gate;      /* read for dx                           */
  const void* w_up;
  int64_t w_stride;
  const void* d_out;       /* [shards * rows, n]                    */
  int64_t d_out_stride;
  const void* gate;        /* as the forward pass wrote them        */
  const void* up;
  int64_t saved_stride;
  void* d_gate;            /* out, [shards * rows, n]; may be gate  */
  void* d_up;              /* and up (unless those are float32), or */
                           /* one of them d_out                     */
  int64_t d_stride;
  void* dx;                /* [shards * rows, k] or NULL            */
  int64_t dx_stride;
  void* dw_gate;           /* like the weights; both or none        */
  void* dw_up;
  int64_t dw_stride;
  int64_t f32_grads;       /* dw_gate and dw_up are float32         */
  void* workspace;
} agmm_gated_grad_args_t;

typedef struct agmm_gated_s* agmm_gated_t;

agmm_status_t agmm_gated_plan(const agmm_gated_desc_t* desc, agmm_gated_t* out_plan);
/* gate and up of the plan's runs and backward passes are float32 (1), or of its
 * type (0, as a new plan has it).  Before the plan is used. */
agmm_status_t agmm_gated_save_float(agmm_gated_t plan, int on);
size_t agmm_gated_workspace_bytes(agmm_gated_t plan);
agmm_status_t agmm_gated_run(agmm_gated_t plan, const agmm_gated_args_t* args, void* stream);
agmm_status_t agmm_gated_backward(agmm_gated_t plan, const agmm_gated_grad_args_t* args, void* stream);
void agmm_gated_destroy(agmm_gated_t plan);

/* ------------------------------------------------------------------- linear
 *
 *     pre = X W + bias,  out = a(pre) + residual
 * in one kernel; pre is written (rounded) when it is asked for.  Backwards, from
 * that (the residual's gradient is d_out itself):
 *     d_pre = d_out * a'(pre)     (no activation: d_out, and neither is given)
 *     dx = d_pre W^T,  dw = X^T d_pre,  d_bias = sum over rows of d_pre
 */
typedef struct {
  int k, n;                     /* multiples of 8, 8..2^20          */
  agmm_activation_t activation;
  int rhs_transpose;            /* the weight is stored [n, k]      */
  agmm_dtype_t dtype;           /* AGMM_BF16 or AGMM_F16            */
} agmm_linear_desc_t;

typedef struct {
  int64_t shards, rows;    /* shards * rows up to 2^31 - 1024       */
  const void* x[8];        /* [rows, k] each                        */
  int64_t x_stride;
  const void* w;
  int64_t w_stride;
  const void* bias;        /* [n] or NULL                           */
  const void* residual;    /* [shards * rows, n] or NULL            */
  int64_t residual_stride;
  void* out;               /* [shards * rows, n]; may be residual   */
  int64_t out_stride;
  void* pre;               /* out, [shards * rows, n] or NULL       */
  int64_t pre_stride;
  void* workspace;
} agmm_linear_args_t;

typedef struct {
  int64_t shards, rows;
  const void* x[8];        /* read for dw                           */
  int64_t x_stride;
  const void* w;           /* read for dx                           */
  int64_t w_stride;
  const void* d_out;       /* [shards * rows, n]                    */
  int64_t d_out_stride;
  const void* pre;         /* with an activation: as the forward pass wrote it */
  int64_t pre_stride;
  void* d_pre;             /* with an activation: out, [shards * rows, n]; may */
  int64_t d_pre_stride;    /* be pre (unless that is float32) or d_out         */
  void* dx;                /* [shards * rows, k] or NULL            */
  int64_t dx_stride;
  void* dw;                /* like the weight, or NULL              */
  int64_t dw_stride;
  void* d_bias;            /* [n] or NULL                           */
  int64_t f32_grads;       /* dw and d_bias are float32             */
  void* workspace;
} agmm_linear_grad_args_t;

typedef struct agmm_linear_s* agmm_linear_t;

agmm_status_t agmm_linear_plan(const agmm_linear_desc_t* desc, agmm_linear_t* out_plan);
/* pre of the plan's runs and backward passes is float32 (1), or of its type (0,
 * as a new plan has it).  Before the plan is used. */
agmm_status_t agmm_linear_save_float(agmm_linear_t plan, int on);
size_t agmm_linear_workspace_bytes(agmm_linear_t plan);
agmm_status_t agmm_linear_run(agmm_linear_t plan, const agmm_linear_args_t* args, void* stream);
agmm_status_t agmm_linear_backward(agmm_linear_t plan, const agmm_linear_grad_args_t* args, void* stream);
void agmm_linear_destroy(agmm_linear_t plan);

#ifdef __cplusplus
}
#endif

#endif /* AGMM_FEEDFORWARD_H_ */
