/*
 * lc_moe, training operators -- what a program that trains the layer of lc_moe.h needs
 * beside its forward and the grouped FFN's backward (lc_moe_ffn_backward):
 *
 *   lc_moe_forward_saved    where the forward's intermediates lie in its workspace
 *   lc_moe_balance_loss     load-balance and z loss, per-expert counts, and the gradient
 *                           of both losses with respect to the router's logits
 *   lc_moe_gate_backward    gradient of the layer output with respect to every gate
 *   lc_moe_router_backward  gradient of the gates and of losses on the logits, through the
 *                           softmax, with respect to the tokens and the router weight
 *   lc_moe_adamw            one AdamW step over many tensors, states in 32 bits or in 8
 *
 * The pages describe the model's training (LongCat-Flash article, itouyu.top, section
 * "Model scaling and multi-stage training") but give no formula of these; each definition
 * is stated below.  The conventions of lc_moe.h hold here too: device pointers aligned to
 * 16 bytes, host structs, checks before anything is enqueued, no allocation, no host
 * synchronisation, kernel launches only (capturable into a HIP graph), deterministic
 * results, NaN and Inf outside the contract except where a function says otherwise.
 * A workspace may be reused by consecutive calls on one stream; calls that overlap in time
 * (two streams, two captured graphs that are replayed side by side) need one each.
 */
#ifndef LC_MOE_TRAIN_H
#define LC_MOE_TRAIN_H

#include "lc_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Device addresses inside the workspace of lc_moe_forward (host struct). */
typedef struct {
  const float* logits;        /* [T][N+Z] router logits x W_r^T                              */
  const void* ffn_rows;       /* [T*K][d] dtype: output of every FFN pick, one row each;
                                 rows from ffn_offsets[N] on are unwritten                 */
  const int32_t* slot_row;    /* [T][K] row of every pick, -1 for a zero-computation pick    */
  const int32_t* ffn_offsets; /* [N+1] first row of every FFN expert                        */
  const int32_t* perm_token;  /* [T*K] token of every row                                   */
} lc_moe_saved;

/* Fills *saved for this shape and workspace (pure host arithmetic; nothing is enqueued).
 * The arrays hold the values of the last lc_moe_forward / lc_moe_forward_staged on this
 * workspace with this shape, until another call uses the workspace: a program that trains
 * gives each layer a workspace of its own from forward to backward.  After a call of
 * lc_moe_route only `logits` is valid.  (lc_moe_forward_noalloc keeps its intermediates in
 * the library's own array, which has no such view.) */
lc_moe_status lc_moe_forward_saved(const lc_moe_shape* shape, const void* workspace,
                                   size_t workspace_bytes, lc_moe_saved* saved);

/* Coefficients of lc_moe_balance_loss (host struct). */
typedef struct {
  float balance, z;
} lc_moe_balance_coef;

/* Load-balance loss over sequences, router z loss, per-expert counts, and their gradient.
 * The T tokens are cut into num_seqs sequences; sequence s holds the tokens
 * seq_offsets[s] .. seq_offsets[s+1] - 1.  A token counts if it lies in a sequence, its
 * token_mask is nonzero and not all of its logits are -infinity (a single logit of
 * -infinity has probability 0).  With p_t = softmax(logits_t), n_s the tokens of s that
 * count, n their total, S' the number of sequences with n_s > 0, E = N + Z:
 *   load[s][i]  = picks of expert i among the tokens of s that count (picks outside
 *                 0..N+Z-1 are left out; a repeated pick counts each time)
 *   prob[s][i]  = (1 / n_s) sum_t p_t,i                        (0 where n_s = 0)
 *   f[s][i]     = E load[s][i] / (K n_s)
 *   loss[0]     = balance / S' * sum_s sum_i f[s][i] prob[s][i]  (an even load gives
 *                 `balance`); 0 if nothing counts
 *   loss[1]     = z / n * sum_t logsumexp(logits_t)^2
 * The counts are not differentiated, so the gradient of loss[0] + loss[1] is
 *   dlogits_t,i = p_t,i (u_i - sum_j u_j p_t,j) + (2 z / n) logsumexp_t p_t,i,
 *   u_i = balance (f[s][i] - 1) / (S' n_s)
 * (the 1 changes no gradient, since p sums to 1; E load - K n_s is taken in whole numbers,
 * so an even load gives a gradient of exactly 0).  Probabilities, sums and losses are fp32;
 * the sums over tokens are added in a fixed order.
 *   logits       [T][N+Z] fp32         (lc_moe_saved.logits); rows of tokens that the mask or
 *                                      the offsets leave out are not read
 *   topk_idx     [T][K] int32
 *   seq_offsets  [num_seqs+1] int32, ascending, 0 <= seq_offsets[0], last <= T; or NULL with
 *                num_seqs = 1: one sequence of all T tokens.  Sequences may be empty.
 *                Offsets outside 0..T are taken as the nearest of the two; offsets that
 *                descend give unspecified numbers, but nothing out of range is touched.
 *   token_mask   [T] uint8, or NULL: every token
 *   loss         [2] fp32 (out)
 *   load         [num_seqs][N+Z] int32 (out); prob [num_seqs][N+Z] fp32 (out)
 *   dlogits      [T][N+Z] fp32 (out), zero in the rows of tokens that do not count; NULL:
 *                not computed
 * Reads T, N, Z, K of shape (which must pass the usual checks).  1 <= num_seqs <= 65535
 * (else LC_MOE_E_SHAPE). */
size_t lc_moe_balance_workspace_size(const lc_moe_shape* shape, int32_t num_seqs);
lc_moe_status lc_moe_balance_loss(const lc_moe_shape* shape, const lc_moe_balance_coef* coef,
                                  const float* logits, const int32_t* topk_idx,
                                  const int32_t* seq_offsets, int32_t num_seqs,
                                  const uint8_t* token_mask, float* loss, int32_t* load,
                                  float* prob, float* dlogits, void* workspace,
                                  size_t workspace_bytes, hipStream_t stream);

/* Gradient of L = sum_t <dy_t, y_t> with respect to the gates: for an FFN pick (t, k)
 *   dgate[t][k] = <dy_t, ffn_rows[slot_row[t][k]]>,
 * for a zero-computation pick (slot_row < 0) dgate[t][k] = <dy_t, x_t>.  Products and sums
 * are fp32, added in a fixed order.  A row index of num_rows or more reads nothing and
 * gives 0.
 *   x, dy      [T][d] dtype
 *   ffn_rows   [num_rows][d] dtype, 0 <= num_rows <= T*K (else LC_MOE_E_SHAPE); may be NULL if
 *              num_rows = 0
 *   slot_row   [T][K] int32
 *   dgate      [T][K] fp32 (out)
 * Reads T, d, K and dtype of shape. */
lc_moe_status lc_moe_gate_backward(const lc_moe_shape* shape, const void* x, const void* ffn_rows,
                                   int32_t num_rows, const int32_t* slot_row, const void* dy,
                                   float* dgate, hipStream_t stream);

/* Backward of the router: from the gradient of the gates (the selection is held fixed) and
 * the gradient of losses on the logits,
 *   dp_t,i      = sum of dgate[t][k] over the picks k of token t with topk_idx[t][k] = i
 *   dlogits_t,i = p_t,i (dp_t,i - sum_j p_t,j dp_t,j) + dlogits_aux_t,i,  p_t = softmax(logits_t)
 *   dx          = dlogits W_r + dx_add
 *   dw_router   = dlogits^T x
 * with fp32 sums.  For the matrix cores dlogits, W_r and fp32 tokens are cut into parts of 8
 * bits whose products are exact, three of every operand: 24 bits.  dx of a bf16 layer of many
 * tokens is made of two fp16 parts instead, a power of two taken out of every row: 23 bits, of
 * values below 2^-17 of their row's largest down to 2^-39 of it.  dx is rounded once.
 * A pick outside 0..N+Z-1 has no gradient.  A token whose logits are all -infinity has
 * dlogits = dlogits_aux.
 *   x            [T][d] dtype
 *   w_router     [N+Z][d] fp32
 *   logits       [T][N+Z] fp32, topk_idx [T][K] int32, dgate [T][K] fp32: all three, or dgate
 *                NULL (then none is read): no gradient from the gates
 *   dlogits_aux  [T][N+Z] fp32 (lc_moe_balance_loss), or NULL
 *   dx_add       [T][d] dtype, or NULL: added to dx; may be dx itself (the FFN's dx, say)
 *   dx           [T][d] dtype (out), or NULL: not computed
 *   dw_router    [N+Z][d] fp32 (out), or NULL: not computed
 *   dlogits      [T][N+Z] fp32 (out), or NULL; may be dlogits_aux itself
 * Reads T, d, N, Z, K and dtype of shape.  Outputs and inputs may overlap only as said. */
size_t lc_moe_router_backward_workspace_size(const lc_moe_shape* shape);
lc_moe_status lc_moe_router_backward(const lc_moe_shape* shape, const void* x,
                                     const float* w_router, const float* logits,
                                     const int32_t* topk_idx, const float* dgate,
                                     const float* dlogits_aux, const void* dx_add, void* dx,
                                     float* dw_router, float* dlogits, void* workspace,
                                     size_t workspace_bytes, hipStream_t stream);

/* One tensor of an AdamW step (host struct holding device pointers). */
typedef struct {
  void* param;         /* [n] param_dtype (in/out)                                          */
  float* master;       /* [n] fp32 (in/out), or NULL: the weight with all its digits; param is
                          then only written, as its rounding                              */
  const void* grad;    /* [n] grad_dtype                                                    */
  void* m;             /* [n] fp32, or E4M3 codes (uint8) with state_bits = 8 (in/out)       */
  void* v;             /* [n] the same                                                      */
  uint8_t* m_scale;    /* [ceil(n/128)] E8M0 exponents of m's blocks (state_bits = 8)         */
  uint8_t* v_scale;    /* the same of v's                                                   */
  int64_t n;           /* 0 <= n < 2^40                                                     */
  int32_t param_dtype; /* lc_moe_dtype                                                      */
  int32_t grad_dtype;  /* lc_moe_dtype                                                      */
  float weight_decay;
  float lr_scale;      /* the tensor's learning rate is lr * lr_scale                        */
} lc_moe_adamw_tensor;

/* Hyperparameters of an AdamW step (host struct). */
typedef struct {
  float lr, beta1, beta2, eps;
  int32_t state_bits;      /* 32 or 8                                                        */
  int32_t step;            /* number of this step, from 1 on                                 */
  const int32_t* step_dev; /* NULL, or a device word that is read instead of `step` (a step
                              that is captured into a graph and replayed); values below 1
                              are taken as 1                                                */
  const float* grad_scale; /* NULL, or a device word the gradients are multiplied by (loss
                              scale, clipping); if it is not finite the step is left out:
                              nothing changes                                               */
  uint32_t seed;           /* of the random bits (state_bits = 8)                            */
} lc_moe_adamw_hyper;

/* One AdamW step over `count` tensors (host array; read before return).  Per element, in
 * fp32, with t the step number:
 *   g = grad * grad_scale
 *   m = beta1 m + (1 - beta1) g
 *   v = beta2 v + ((1 - beta2) g) g
 *   w = w (1 - lr weight_decay) - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
 * (1 - beta^t and the scalars made of it in fp64, then fp32), w the master if there is one,
 * else param; param is w rounded to nearest even.  A bf16 param without a master forgets
 * updates below half its step: that is the caller's choice.
 *
 * state_bits = 8: m and r = sqrt(v) are kept in blocks of 128 elements in the framework's
 * block-FP8 form (see lc_moe_quantize_activations): E4M3 codes of the values over 2^k, the
 * exponent byte k + 127, k the smallest integer with the block's largest |value| <=
 * 448 * 2^k (0 for a block of zeros, at least -127).  The root halves v's range of exponents,
 * which E4M3 could not span.  Rounded to nearest, a state that moves by less than half a
 * step per update would never move; so the codes are rounded up or down at random with the
 * right mean, from 16 bits each of a hash of (seed, step, place in `tensors`, element), the
 * same bits for the same arguments, and of m and r before their rounding to fp32 (but where m's
 * two terms cancel); and an r above 0 stays above 0, so that no m is ever divided by eps alone.
 * The update itself uses m and v before they are rounded to codes.  A state that becomes infinite
 * (v, for a gradient above 1e19) takes the exponent byte 247 and the largest code, which is
 * infinite again when it is read; its block is lost, other blocks are not.
 * A state starts as zeros: codes 0 and exponent bytes 127.
 *
 * state_bits = 32: m and v are fp32, m_scale and v_scale are not read (may be NULL).
 * Tensors with n = 0 are skipped and their pointers not read.  What a call writes may overlap
 * nothing else of it; gradients may be shared.  count = 0 does nothing; count < 0, n out of range,
 * state_bits other than 8 and 32, step < 1 without step_dev, a beta outside [0, 1), eps < 0 or
 * an eps between 0 and 2^-126 (the quotient's reciprocal takes such numbers as 0):
 * LC_MOE_E_SHAPE; an unknown dtype: LC_MOE_E_DTYPE.  With eps = 0 an element whose v is 0 follows the formula: 0 / 0. */
lc_moe_status lc_moe_adamw(const lc_moe_adamw_tensor* tensors, int32_t count,
                           const lc_moe_adamw_hyper* hyper, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* LC_MOE_TRAIN_H */
