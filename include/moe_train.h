/*
 * moe_train.h -- C ABI of the training side of the routed experts (GB300,
 * sm_103a): the expert products in 16 bits with their gradients, the SwiGLU
 * gradient, the rows' way to the experts and back, and the AdamW step of the
 * weights.  Weights trained here are quantised for moe_fp8_block_scale_forward
 * by moe_quantize_weight_128x128.
 *
 * Conventions are those of moe_fp8.h (device pointers owned by the caller,
 * asynchronous on `stream`, host-side argument errors returned before any
 * launch, device-side conditions OR-ed into *device_status).  16-bit values
 * are passed as their uint16 bit patterns, BF16 or FP16 by a dtype argument.
 * Sums are held in FP32 and each output is rounded once, to nearest even.
 * No entry point uses atomics on data or allocates memory: the same inputs
 * give the same bits, and calls on different streams do not share anything.
 *
 * Plan order: rows of an expert are contiguous "slots" of a row buffer.  The
 * layout moe_plan makes is one such order (moe_plan_groups reads it); any
 * other is described by group_start and group_rows directly.
 *
 * Where buffers must not overlap, row buffers of one row stride may be columns of
 * one wider buffer; rows of different strides must not interleave.
 */
#ifndef MOE_TRAIN_H
#define MOE_TRAIN_H

#include <stddef.h>
#include <stdint.h>

#include "moe_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_TYPE_BF16 0
#define MOE_TYPE_FP16 1
#define MOE_TYPE_FP32 2

/* A group lies outside the row buffer (start < 0, rows < 0 or start + rows
 * beyond it): it is treated as empty. */
#define MOE_DEV_BAD_GROUP 0x8

/* ------------------------------------------------------------------------
 * The groups of a plan (moe_plan or moe_route_plan): for expert e its first
 * slot group_start[e] and its number of routes group_rows[e] (0 and 0 where
 * it has none), and for route r its slot route_slot[r] (-1 if the plan does
 * not hold it).
 *  sorted_token_ids [sorted_cap], expert_ids [blocks_cap],
 *  num_tokens_post_padded [1]   the plan; R = M * top_k its route count
 *  group_start, group_rows      [E] int32 out
 *  route_slot                   nullable [R] int32 out
 * 1 <= E <= 2048; 8 <= block_m <= 1024, block_m % 8 == 0;
 * sorted_cap >= blocks_cap * block_m. */
moe_status moe_plan_groups(const int32_t* sorted_token_ids, int64_t sorted_cap, const int32_t* expert_ids,
                           int64_t blocks_cap, const int32_t* num_tokens_post_padded, int block_m, int64_t R, int E,
                           int32_t* group_start, int32_t* group_rows, int32_t* route_slot, moe_stream_t stream);

/* ------------------------------------------------------------------------
 * Dispatch and combine of rows; each is the other's gradient.
 * ------------------------------------------------------------------------ */

/* xs[s] = x[route_ids[s] / top_k] for every slot s below num_rows whose route
 * id is in [0, M * top_k); the other slots below num_rows become zero, slots
 * at and past it are not touched.
 *  x          [M, ldx], xs [rows, ldxs]: `width` elements of each row
 *  route_ids  [rows] (sorted_token_ids of a plan)
 *  num_rows   nullable [1] device scalar (num_tokens_post_padded); NULL: rows
 * dtype BF16, FP16 or FP32; width, ldx and ldxs multiples of 16 bytes' worth
 * of elements, x and xs 16-byte aligned; x and xs do not overlap.  x may be
 * NULL where M is 0. */
moe_status moe_gather_rows(const void* x, int64_t M, int width, int64_t ldx, void* xs, int64_t rows, int64_t ldxs,
                           const int32_t* route_ids, int top_k, const int32_t* num_rows, int dtype,
                           moe_stream_t stream);

/* out[t] = sum over j of y[route_slot[t * top_k + j]], added in FP32 in the
 * order of j (first out[t] itself if accumulate != 0) and rounded once.
 * Slots outside [0, rows) add nothing; a token without any gives zero.
 *  y [rows, ldy], out [M, ldout], route_slot [M, top_k]
 * Types, widths and alignment as above; y and out do not overlap.  y may be
 * NULL where rows is 0. */
moe_status moe_sum_routes(const void* y, int64_t rows, int width, int64_t ldy, void* out, int64_t M, int64_t ldout,
                          const int32_t* route_slot, int top_k, int accumulate, int dtype, moe_stream_t stream);

/* ------------------------------------------------------------------------
 * Products grouped by expert, ragged in the rows of each group.
 *
 *  MOE_GROUPED_FORWARD          y[s, n] = sum_k x[s, k] w[e, n, k]
 *  MOE_GROUPED_INPUT_GRADIENT   y[s, k] = sum_n x[s, n] w[e, n, k]
 *                               (x is the gradient of the forward's y)
 * for every slot s of every group e.  Slots outside the groups are not
 * written, and what they hold in x has no influence, NaN included.
 *
 * Epilogue MOE_GROUPED_SWIGLU (forward only; rows [0, N/2) of w are the gate,
 * [N/2, N) the up projection):
 *   y[s, i] = silu(gate) * up * weight(s)     [rows, N / 2]
 *   pre[s]  = gate | up                       [rows, N], if pre is not NULL
 * with the FP32 sums, before any rounding.  weight(s) = 1 without
 * route_weights, else route_weights[route_ids[s]] (0 for an id outside
 * [0, R)), or route_weights[s] without route_ids.
 * ------------------------------------------------------------------------ */
#define MOE_GROUPED_FORWARD 0
#define MOE_GROUPED_INPUT_GRADIENT 1
#define MOE_GROUPED_PLAIN 0
#define MOE_GROUPED_SWIGLU 1

typedef struct moe_grouped_args {
  const uint16_t* x;           /* [rows, ldx]                                             */
  const uint16_t* w;           /* [E, N, K] dense                                         */
  uint16_t* y;                 /* [rows, ldy]                                             */
  uint16_t* pre;               /* SWIGLU, nullable: [rows, ldpre]                         */
  const int32_t* group_start;  /* [E] first slot of each group                            */
  const int32_t* group_rows;   /* [E] slots of each group; groups do not overlap          */
  const int32_t* route_ids;    /* SWIGLU, nullable: [rows]                                */
  const float* route_weights;  /* SWIGLU, nullable: [R], or [rows] without route_ids      */
  int32_t* device_status;      /* nullable [1]: MOE_DEV_* bits are OR-ed in               */
  int64_t rows;                /* slots of x, y and pre                                   */
  int64_t ldx, ldy, ldpre;     /* elements from one row to the next                       */
  int64_t R;                   /* routes (SWIGLU with route_ids)                          */
  int32_t E, N, K;
  int32_t dtype;               /* MOE_TYPE_BF16 or MOE_TYPE_FP16                          */
  int32_t direction;           /* MOE_GROUPED_FORWARD or _INPUT_GRADIENT                  */
  int32_t epilogue;            /* MOE_GROUPED_PLAIN or _SWIGLU                            */
} moe_grouped_args;

/* 1 <= E <= 2048; N and K multiples of 8 (N of 16 with SWIGLU); row strides
 * multiples of 8 and at least the row's width; pointers 16-byte aligned
 * (those to 4-byte elements: 4 bytes);
 * 0 <= rows < 2^31.  y and pre overlap no input and not one another. */
moe_status moe_grouped_gemm(const moe_grouped_args* args, moe_stream_t stream);

/* dw[e, n, k] = sum over the slots s of group e of dy[s, n] x[s, k]; zero for
 * an empty group.  accumulate != 0 (FP32 output only): added to what dw
 * holds, one addition per element; empty groups leave dw as it is. */
typedef struct moe_grouped_wgrad_args {
  const uint16_t* dy;          /* [rows, lddy], N wide                                    */
  const uint16_t* x;           /* [rows, ldx], K wide                                     */
  void* dw;                    /* [E, N, K] dense                                         */
  const int32_t* group_start;  /* [E]                                                     */
  const int32_t* group_rows;   /* [E]                                                     */
  int32_t* device_status;      /* nullable [1]                                            */
  int64_t rows;
  int64_t lddy, ldx;
  int32_t E, N, K;
  int32_t dtype;               /* of dy and x: MOE_TYPE_BF16 or MOE_TYPE_FP16             */
  int32_t dw_dtype;            /* dtype, or MOE_TYPE_FP32                                 */
  int32_t accumulate;
} moe_grouped_wgrad_args;

/* Constraints as for moe_grouped_gemm. */
moe_status moe_grouped_wgrad(const moe_grouped_wgrad_args* args, moe_stream_t stream);

/* ------------------------------------------------------------------------
 * The gradient of h = silu(gate) * up * weight, by rows.  With
 * sig = 1 / (1 + exp(-gate)):
 *   dpre[s]      = dh * weight * up * sig * (1 + gate * (1 - sig))  |
 *                  dh * weight * gate * sig
 *   h[s]         = silu(gate) * up * weight    (recomputed, if h is not NULL)
 *   dweights[r]  = sum_i dh * silu(gate) * up  (if dweights is not NULL)
 * for every slot s below num_rows whose route id r is in [0, R); without
 * route_ids for every slot below num_rows, with r = s.  Other rows are not
 * written.
 * ------------------------------------------------------------------------ */
typedef struct moe_swiglu_backward_args {
  const uint16_t* dh;          /* [rows, lddh], I wide                                    */
  const uint16_t* pre;         /* [rows, ldpre], 2 I wide: gate | up                      */
  uint16_t* dpre;              /* [rows, lddpre], 2 I wide; may be pre itself             */
  uint16_t* h;                 /* nullable [rows, ldh], I wide; may be dh itself          */
  const int32_t* route_ids;    /* nullable [rows]                                         */
  const int32_t* num_rows;     /* nullable [1] device scalar; NULL: rows                  */
  const float* route_weights;  /* nullable [R] ([rows] without route_ids); NULL: 1        */
  float* dweights;             /* nullable [R] ([rows] without route_ids)                 */
  int64_t rows;
  int64_t lddh, ldpre, lddpre, ldh;
  int64_t R;
  int32_t I;
  int32_t dtype;               /* MOE_TYPE_BF16 or MOE_TYPE_FP16                          */
} moe_swiglu_backward_args;

/* I and the row strides multiples of 8; dh, pre, dpre and h 16-byte aligned. */
moe_status moe_swiglu_backward(const moe_swiglu_backward_args* args, moe_stream_t stream);

/* ------------------------------------------------------------------------
 * AdamW over many tensors in one launch (one for each type of gradient).  Per element, in FP32:
 *   g = grad * *grad_scale                      (1 without grad_scale)
 *   m = beta1 m + (1 - beta1) g
 *   v = beta2 v + (1 - beta2) g^2
 *   p = p (1 - lr weight_decay) - (lr / (1 - beta1^step)) m / (sqrt(v) / sqrt(1 - beta2^step) + eps)
 * and the rounded copy of p in `model`, where there is one.
 * The update is right to a few roundings down to the smallest v, whatever eps;
 * with eps = 0 an element whose v is 0 gets 0 / 0.
 *
 * State bits 32: exp_avg and exp_avg_sq hold m and v in FP32.
 * State bits 8: they hold E4M3 codes of m and of r = sqrt(v), with one FP32
 * scale per 128 consecutive elements (the largest magnitude times 1/448; a
 * group of zeros has scale 0), each rewritten after the step's own update has used the
 * unrounded values.  m is rounded to nearest even.  r moves by less than half
 * a code per step when beta2 is near 1, and would stand still under rounding
 * to nearest; it is rounded up with the probability of the part cut off, from
 * an integer hash of (seed, tensor, element): give every step its own seed.
 * A positive r never becomes code 0 (m / (0 + eps) would follow).
 * A NaN becomes code 0x7F and stays in its element.  Where v passes FP32 the
 * update is m / inf = 0, as with FP32 states, but r is held (formed without its
 * square), so that v returns; m or r beyond FP32 are held as its largest value.
 * Such an element decides its group's scale: its neighbours' m become 0 and
 * their r the smallest code, 2^-9 of the scale, until it has decayed.  A step
 * whose gradients overflow is better left out by `skip`.
 * ------------------------------------------------------------------------ */
typedef struct moe_adamw_tensor {
  float* param;                /* [n] FP32                                                */
  uint16_t* model;             /* nullable [n]: rounded copy, written only                */
  const void* grad;            /* [n] grad_dtype                                          */
  void* exp_avg;               /* [n] FP32, or E4M3 codes                                 */
  void* exp_avg_sq;            /* [n] FP32, or E4M3 codes of the root                     */
  float* exp_avg_scale;        /* state bits 8: [ceil(n / 128)]                           */
  float* exp_avg_sq_scale;     /* state bits 8: [ceil(n / 128)]                           */
  int64_t n;                   /* elements, >= 0                                          */
  double weight_decay;
  int32_t grad_dtype;          /* MOE_TYPE_*                                              */
  int32_t model_dtype;         /* MOE_TYPE_BF16 or MOE_TYPE_FP16 (model given)            */
} moe_adamw_tensor;

/* Device bytes of a table of `count` tensors (host-only; 0 for count < 1). */
size_t moe_adamw_table_bytes(int count);

/* Check `tensors` (HOST array) and copy their table to the device.  Pointers
 * 16-byte aligned (scales: 4-byte), no two tensors overlapping; the array may
 * be reused when the call returns, the device buffers it names have to live
 * as long as the table.  Writes, through the host pointers, the table's number
 * of work chunks and which gradient types it has (bit MOE_TYPE_*).  1 <= count <= 65536; state_bits 32 or 8. */
moe_status moe_adamw_table_init(const moe_adamw_tensor* tensors, int count, int state_bits, void* table,
                                size_t table_bytes, int64_t* chunks, int32_t* grad_types, moe_stream_t stream);

typedef struct moe_adamw_args {
  const void* table;           /* written by moe_adamw_table_init                         */
  const float* grad_scale;     /* nullable [1] device scalar                              */
  const int32_t* skip;         /* nullable [1]: not 0: the step changes nothing           */
  int64_t chunks;              /* from moe_adamw_table_init                               */
  int64_t step;                /* 1 for the first step; one that `skip` left out does not count */
  double lr, beta1, beta2, eps; /* (1 - beta is formed in double, then rounded)           */
  uint32_t seed;               /* state bits 8                                            */
  int32_t count;
  int32_t state_bits;          /* as given to moe_adamw_table_init                        */
  int32_t grad_types;          /* from moe_adamw_table_init                               */
} moe_adamw_args;

/* A table of other state bits is left as it is, and chunks past the table's are
 * none.  lr, eps >= 0 and finite; 0 <= beta1, beta2 < 1; step >= 1.  lr, step and seed
 * are taken when the call is made: a captured graph repeats those of its capture
 * (grad_scale and skip are read by the device). */
moe_status moe_adamw_step(const moe_adamw_args* args, moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_TRAIN_H */
