/*
 * moe_block.h -- C ABI of what stands between the residual stream and the
 * routed experts (GB300, sm_103a): the choice of experts from scores, with its
 * gradient and the step of its balance bias, and the norms before and after a
 * block fused with its gate, its residual scale and the quantisation of the
 * experts' input, with their gradient.
 *
 * Conventions are those of moe_fp8.h and moe_train.h: device pointers owned by
 * the caller, asynchronous on `stream`, host-side argument errors returned
 * before any launch; 16-bit values as bit patterns, their type (MOE_TYPE_*) by
 * an argument.  Arithmetic and sums are in FP32 (64 bits where this header says
 * so), each output is rounded once.  No entry point uses atomics on data or
 * allocates memory: the same inputs give the same bits.
 *
 * A padded batch: num_tokens and num_rows are nullable device scalars, read by
 * the kernel, so that a captured graph follows them; only the tokens or rows
 * below count (values outside [0, M] are taken as the nearer end).
 */
#ifndef MOE_BLOCK_H
#define MOE_BLOCK_H

#include <stddef.h>
#include <stdint.h>

#include "moe_fp8.h"
#include "moe_train.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * Routing by scores.  For a token's logits l [E]:
 *   s_e = 1 / (1 + exp(-l_e))                     MOE_SCORE_SIGMOID
 *   s_e = exp(l_e) / sum_i exp(l_i)               MOE_SCORE_SOFTMAX
 *   c_e = s_e + bias[e]; without a bias experts are compared by l_e itself
 * An expert whose logit or bias is -inf is left out.  The E experts form
 * `groups` runs of E / groups; a group's value is the largest c of its experts
 * (MOE_GROUP_MAX) or the sum of its two largest (MOE_GROUP_TOP2; one alone
 * counts by itself; without a bias c = s here).  Of the topk_groups largest
 * groups, the top_k experts with the largest c are chosen, in falling order.
 * Values are compared as in 64 bits; of equal ones the lower index comes first.  (A bias
 * beside which scores vanish in FP32 is right but slow, 50 times at its type's lowest
 * value: leave experts out by -inf.)
 *   topk_weights[t, j] = routed_scale * s_j / (sum of s over the chosen)
 *                                                 with renormalize
 *   topk_weights[t, j] = routed_scale * s_j       without
 * The bias has no part in the weights.  Where fewer than top_k experts can be
 * chosen, and for padding tokens, the rest of the row has id -1 (which moe_plan
 * leaves out) and weight 0.  Renormalised weights are right however small
 * the scores are.  A NaN, in the logits or the bias, counts as the largest value and
 * stays in the weights that its score is part of; ids are always distinct.
 *
 * Accuracy, in units of 2^-23 and with x the distance of a logit from the largest one (softmax) or
 * from 0 (sigmoid): a score is within 4 + |x| / 2 units of itself, a renormalised weight within
 * twice that and 5 more.  A plain softmax weight is divided by a total of hardware exponentials, off
 * by up to 2 + 1.7 ln E units and half a unit for each of E / 32 + 5 additions (groups: up to 133).
 * ------------------------------------------------------------------------ */
#define MOE_SCORE_SOFTMAX 0
#define MOE_SCORE_SIGMOID 1
#define MOE_GROUP_MAX 0
#define MOE_GROUP_TOP2 1

typedef struct moe_route_scores_args {
  const void* logits;          /* [M, ldlogits] dtype                                     */
  const float* bias;           /* nullable [E]                                            */
  void* topk_ids;              /* [M, top_k] int32 or int64 (id_bits)                     */
  float* topk_weights;         /* [M, top_k]                                              */
  const int32_t* num_tokens;   /* nullable [1]                                            */
  int64_t M;
  int64_t ldlogits;            /* elements from one token's logits to the next's          */
  int32_t E, top_k;
  int32_t groups, topk_groups; /* 1 and 1: no groups                                      */
  int32_t group_score;         /* MOE_GROUP_*                                             */
  int32_t score;               /* MOE_SCORE_*                                             */
  int32_t renormalize;
  int32_t dtype;               /* MOE_TYPE_*                                              */
  int32_t id_bits;             /* 32 or 64                                                */
  float routed_scale;
} moe_route_scores_args;

/* 1 <= E <= 2048; 1 <= groups <= 32, E % groups == 0; 1 <= topk_groups <=
 * groups; 1 <= top_k <= min(32, topk_groups * E / groups); E <= ldlogits < 2^31;
 * M * top_k < 2^31.  Pointers aligned to their elements; the outputs overlap
 * no input and not one another. */
moe_status moe_route_scores(const moe_route_scores_args* args, moe_stream_t stream);

/* The logits' gradient from the weights' (dweights).  With the token's listed
 * experts j (ids in [0, E) whose logit is not -inf; other ids and their
 * dweights have no part), p_j = s_j / (sum of s over them):
 *   sigmoid, renormalize: dl_j = scale p_j (1 - s_j) (dw_j - sum_i dw_i p_i)
 *   sigmoid:              dl_j = scale dw_j s_j (1 - s_j)
 *   softmax, renormalize: dl_j = scale p_j (dw_j - sum_i dw_i p_i)
 *   softmax:              dl_e = scale s_e ([e listed] dw_e - sum_i dw_i s_i), every e
 * and zero for the other logits and for padding tokens.  An expert listed twice
 * counts as two terms.  Plain softmax forms its scores by hardware exponentials, within (2 +
 * 1.7 |x|) 2^-23 of themselves before the total's error; what lies below 2^-126 may be 0. */
typedef struct moe_route_scores_backward_args {
  const void* logits;          /* [M, ldlogits] dtype                                     */
  const void* topk_ids;        /* [M, top_k] int32 or int64                               */
  const float* dweights;       /* [M, top_k]                                              */
  void* dlogits;               /* [M, lddlogits] dtype; may be logits itself              */
  const int32_t* num_tokens;   /* nullable [1]                                            */
  int64_t M;
  int64_t ldlogits, lddlogits;
  int32_t E, top_k;
  int32_t score;
  int32_t renormalize;
  int32_t dtype;
  int32_t id_bits;
  float routed_scale;
} moe_route_scores_backward_args;

/* Constraints as above (1 <= top_k <= 32; here top_k may pass E). */
moe_status moe_route_scores_backward(const moe_route_scores_backward_args* args, moe_stream_t stream);

/* out[e] = bias[e] + rate * sign(sum of load - E load[e]): the bias of an expert
 * with less than its even share of routes rises, that of one with more falls.
 * load [E] int32 (a plan's group_rows); out may be bias itself.
 * 1 <= E <= 2048; rate finite. */
moe_status moe_route_balance(const int32_t* load, const float* bias, float* out, int E, float rate,
                             moe_stream_t stream);

/* ------------------------------------------------------------------------
 * A block's exit and the next one's entry, row by row in one pass.  With
 * N(x; w) = x / sqrt(mean(x^2) + eps) * (w + weight_offset)  (w NULL: 1):
 *   u = N(y; w_post) if post_norm, else y
 *   h = residual_scale * r + gate * u              (r NULL: gate * u)
 *   z = N(h; w_pre)
 *   q, q_scale = z in E4M3 with one scale per 128 columns, as
 *                moe_quantize_act_1x128 (or _ue8m0) forms them; a NaN in a group
 *                makes its scale NaN
 * z and q come from the unrounded h, and q from the unrounded z.  h, z and q
 * are nullable (one of them is written at least); r, gate and the weights are
 * too.  Padding rows are not touched.
 *
 * Squares are added in FP32: rows whose sum of squares passes its range
 * (magnitudes beyond about 1e17) are normed to 0, and with eps = 0 rows of magnitudes
 * below about 1e-19 lose bits; a NaN or an infinity stays in its row.
 * ------------------------------------------------------------------------ */
#define MOE_GATE_NONE 0
#define MOE_GATE_CHANNEL 1   /* gate [H], weight_dtype     */
#define MOE_GATE_TOKEN 2     /* gate [M], FP32             */
#define MOE_GATE_FULL 3      /* gate [M, ldgate], dtype    */

typedef struct moe_norm_args {
  const void* y;               /* [M, ldy] dtype: the block's output, the branch          */
  const void* r;               /* nullable [M, ldr] stream_dtype: the residual stream     */
  const void* gate;            /* by gate_mode                                            */
  const void* w_post;          /* nullable [H] weight_dtype                               */
  const void* w_pre;           /* nullable [H] weight_dtype                               */
  void* h;                     /* nullable [M, ldh] stream_dtype; may be r itself         */
  void* z;                     /* nullable [M, ldz] dtype; may be y itself                */
  uint8_t* q;                  /* nullable [M, H] E4M3; H % 128 == 0                      */
  float* q_scale;              /* with q: [M, H / 128]                                    */
  const int32_t* num_rows;     /* nullable [1]                                            */
  int64_t M;
  int64_t ldy, ldr, ldh, ldz, ldgate;
  int32_t H;
  int32_t dtype;               /* MOE_TYPE_*                                              */
  int32_t stream_dtype;        /* dtype or MOE_TYPE_FP32                                  */
  int32_t weight_dtype;        /* dtype or MOE_TYPE_FP32                                  */
  int32_t gate_mode;           /* MOE_GATE_*                                              */
  int32_t post_norm;
  int32_t scale_mode;          /* of q: MOE_SCALES_FP32 or MOE_SCALES_UE8M0               */
  float residual_scale;
  float weight_offset;         /* 0, or 1 for weights kept as the distance from 1         */
  float eps;
} moe_norm_args;

/* H a multiple of 8, 8 <= H <= 16384; row strides multiples of 8 and at least
 * H; pointers 16-byte aligned (q_scale, num_rows and a token gate: 4-byte).
 * 0 <= M < 2^31; eps >= 0 (with eps = 0 a row of zeros gives NaN).  Outputs
 * overlap no input (but h on r, z on y, of the same stride) and not one another. */
moe_status moe_norm_residual(const moe_norm_args* args, moe_stream_t stream);

/* The gradient.  dh is what arrives at h from the stream, dz what arrives at z
 * (each nullable, one is given at least); with R(x) = 1 / sqrt(mean(x^2) + eps):
 *   dH    = dh + R(h) dz w - h R(h)^3 mean(dz w h)           (w = w_pre + offset)
 *   dw_pre[c]  = sum over rows of dz h R(h)
 *   dr    = residual_scale * dH
 *   du    = gate * dH;  dgate = dH u, summed over what the gate is shared by
 *   dy    = du without post_norm, else
 *           R(y) du w - y R(y)^3 mean(du w y)                (w = w_post + offset)
 *   dw_post[c] = sum over rows of du y R(y)
 * h is the forward pass's, as stored (its roots are formed anew); NULL stands
 * for y itself (where h = y: no gate, r or post_norm).  Outputs are nullable.
 * dw_pre, dw_post and a channel gate's dgate are FP32 [H], a token gate's FP32
 * [M], a full one's [M, lddgate] dtype.  accumulate != 0: the three sums over
 * rows are added to what their buffers hold.  Padding rows are not touched and
 * add nothing (a token gate's dgate is not touched there either).  Rows may have
 * whatever magnitude the forward pass takes. */
typedef struct moe_norm_backward_args {
  const void* y;               /* [M, ldy] dtype                                          */
  const void* h;               /* [M, ldh] stream_dtype (with dz; NULL: y)                */
  const void* gate;
  const void* w_post;
  const void* w_pre;
  const void* dh;              /* nullable [M, lddh] stream_dtype                         */
  const void* dz;              /* nullable [M, lddz] dtype                                */
  void* dy;                    /* nullable [M, lddy] dtype; may be dz or y itself         */
  void* dr;                    /* nullable [M, lddr] stream_dtype; may be dh or h itself  */
  void* dgate;                 /* nullable, by gate_mode                                  */
  float* dw_post;              /* nullable [H]                                            */
  float* dw_pre;               /* nullable [H]                                            */
  void* workspace;             /* moe_norm_residual_workspace_size bytes, any contents    */
  const int32_t* num_rows;     /* nullable [1]                                            */
  size_t workspace_bytes;
  int64_t M;
  int64_t ldy, ldh, ldgate, lddh, lddz, lddy, lddr, lddgate;
  int32_t H;
  int32_t dtype, stream_dtype, weight_dtype;
  int32_t gate_mode;
  int32_t post_norm;
  int32_t accumulate;
  float residual_scale;
  float weight_offset;
  float eps;
} moe_norm_backward_args;

/* Device bytes the gradient's sums over rows need (host-only; 0 for sizes it
 * refuses).  Calls that may run at the same time need a workspace each. */
size_t moe_norm_residual_workspace_size(int64_t M, int H);

/* Constraints as above; the workspace 16-byte aligned, and needed only where
 * dw_post, dw_pre or a channel gate's dgate is asked for. */
moe_status moe_norm_residual_backward(const moe_norm_backward_args* args, moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_BLOCK_H */
