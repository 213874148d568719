/*
 * lc_moe, block operators -- what stands directly around the layer of lc_moe.h in a
 * transformer block:
 *
 *   lc_moe_select            choice of experts from the router's logits: softmax or sigmoid
 *                            scores, a bias that counts for the choice only, groups of
 *                            experts, top-K, renormalised and scaled gates
 *   lc_moe_route_select      the same from the tokens (router logits first)
 *   lc_moe_select_backward   gradient of the gates with respect to the logits
 *   lc_moe_forward_picks     the layer for given picks and gates
 *   lc_moe_block_norm        the norms before and after a block, its gate and the scaled
 *                            residual in one pass, and their gradient
 *   lc_moe_quantize_matrix   a bf16 matrix in block FP8, along its rows, its columns or both
 *   lc_moe_matmul_fp8        product of two such matrices
 *   lc_moe_linear_fp8        product of bf16 rows with a weight kept in block FP8, and its
 *                            gradient: the dense products beside the experts
 *
 * The conventions of lc_moe.h hold here too: device pointers aligned to 16 bytes, checks
 * before anything is enqueued, no allocation, no host synchronisation, kernel launches only
 * (capturable into a HIP graph), deterministic results, NaN and Inf outside the contract
 * except where a function says otherwise.  A workspace may be reused by consecutive calls on
 * one stream; calls that overlap in time (two streams, two captured graphs that are replayed
 * side by side) need one each.  Outputs overlap nothing else of a call except as said.
 */
#ifndef LC_MOE_BLOCK_H
#define LC_MOE_BLOCK_H

#include "lc_moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- choice of experts ------------------------------------------------------------------ */

typedef enum { LC_MOE_SOFTMAX = 0, LC_MOE_SIGMOID = 1 } lc_moe_score;

/* How a router's logits become picks and gates (host struct). */
typedef struct {
  int32_t score;      /* lc_moe_score                                                       */
  int32_t groups;     /* G: the N+Z experts in G equal runs; 1: no groups                   */
  int32_t top_groups; /* M: groups that a token may pick from, 1 <= M <= G                  */
  int32_t group_rank; /* 1 or 2: a group's score is the sum of its that many largest scores */
  int32_t renorm;     /* nonzero: the gates of a token's picks are divided by their sum     */
  float scale;        /* factor of every gate                                               */
} lc_moe_gating;

/* With l the logits of a token and E = N + Z:
 *   s_i = softmax(l)_i or 1 / (1 + e^-l_i);   c_i = s_i + bias_i
 *   group score = sum of the group's group_rank largest c; the top_groups groups of largest
 *   score are kept (equal scores: lower group first)
 *   picks = the K largest c of the kept groups, in descending order (equal c: lower index)
 *   gate_k = scale s_k, or with renorm scale s_k / (sum of the token's picked s)
 * (the rule of lc_moe_route with groups = 1, renorm = 0 and scale = 1, but for its decision,
 * which is fp32's).  The choice is that of scores taken in 64 bits: where fp32 cannot tell two
 * of them apart, a token's scores are computed in fp64.  Gates are fp32; with renorm they are
 * taken from the logits of the picks directly, so that scores too small for fp32 still give
 * the right shares.
 * An expert is switched off for a token if its logit, or for all tokens if its bias, is
 * -infinity (or NaN): it is never picked and adds 0 to its group's score; a group of such
 * experts alone is taken after every other.  A token with fewer experts to pick than K, and a
 * token that token_mask leaves out, gets index -1 and gate 0 in what is left of its K places;
 * lc_moe_forward_picks, lc_moe_permute and the training operators pass over index -1.
 *   logits      [T][N+Z] fp32; rows that the mask leaves out are not read
 *   bias        [N+Z] fp32, or NULL: 0
 *   token_mask  [T] uint8, or NULL: every token
 *   topk_idx    [T][K] int32 (out); topk_gate [T][K] fp32 (out)
 * Reads T, N, Z, K of shape (which must pass the usual checks).  K <= 64, 1 <= G <= 64, G
 * divides N+Z, 1 <= M <= G, group_rank 1 or 2 and at most (N+Z)/G, K <= M (N+Z)/G, score one of
 * lc_moe_score and scale finite, else LC_MOE_E_SHAPE. */
lc_moe_status lc_moe_select(const lc_moe_shape* shape, const lc_moe_gating* gating,
                            const float* logits, const float* bias, const uint8_t* token_mask,
                            int32_t* topk_idx, float* topk_gate, hipStream_t stream);

/* Router logits (as lc_moe_route computes them; left in the workspace, where
 * lc_moe_forward_saved finds them), then lc_moe_select.  The workspace is that of
 * lc_moe_workspace_size. */
lc_moe_status lc_moe_route_select(const lc_moe_shape* shape, const lc_moe_gating* gating,
                                  const void* x, const float* w_router, const float* bias,
                                  const uint8_t* token_mask, int32_t* topk_idx, float* topk_gate,
                                  void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Gradient of the gates with respect to the logits, the choice held fixed.  With dg the
 * gradient of a token's gates, w_k = s_k / sum of the picked s:
 *   renorm:      a_k = scale w_k sum_j w_j (dg_k - dg_j);  dlogits of pick k: a_k (softmax) or
 *                a_k (1 - s_k) (sigmoid); no other logit has a gradient
 *   else:        sigmoid: scale dg_k s_k (1 - s_k) at the picks;
 *                softmax: p_i (dp_i - sum_j p_j dp_j), dp_i = scale sum of dg_k over the picks of i
 * plus dlogits_aux.  An index outside 0..N+Z-1 has no gate and no gradient; an index that
 * repeats within a token counts each time.  A logit of -infinity has s = 0.  lc_moe_router_backward
 * takes dlogits as its dlogits_aux, with dgate NULL, to the tokens and the router weight.
 *   logits       [T][N+Z] fp32, topk_idx [T][K] int32, dgate [T][K] fp32
 *   dlogits_aux  [T][N+Z] fp32, or NULL
 *   dlogits      [T][N+Z] fp32 (out); may be dlogits_aux itself
 * Reads T, N, Z, K of shape and score, renorm and scale of gating; K <= 64. */
lc_moe_status lc_moe_select_backward(const lc_moe_shape* shape, const lc_moe_gating* gating,
                                     const float* logits, const int32_t* topk_idx,
                                     const float* dgate, const float* dlogits_aux, float* dlogits,
                                     hipStream_t stream);

/* lc_moe_forward without its route stage: permute -> grouped FFN -> combine for the picks and
 * gates given (lc_moe_select's, say).  A pick of index outside 0..N+Z-1 must have gate 0 and
 * adds nothing.  weights->w_router and weights->bias are not read.
 *   topk_idx [T][K] int32, topk_gate [T][K] fp32; the rest as lc_moe_forward */
lc_moe_status lc_moe_forward_picks(const lc_moe_shape* shape, const void* x,
                                   const lc_moe_weights* weights, const int32_t* topk_idx,
                                   const float* topk_gate, void* y, int32_t* load,
                                   void* workspace, size_t workspace_bytes, hipStream_t stream);

/* ---- norms around a block ---------------------------------------------------------------- */

typedef enum { LC_MOE_GATE_NONE = 0, LC_MOE_GATE_CHANNEL = 1, LC_MOE_GATE_TOKEN = 2 } lc_moe_gate_kind;

/* Scalars of the norms around a block (host struct). */
typedef struct {
  float residual_scale, block_scale, eps; /* eps >= 2^-126 */
  int32_t gate_kind;                      /* lc_moe_gate_kind */
} lc_moe_norm;

/* The end of one block and the start of the next, in one pass.  For every token, with
 * rms(v) = v / sqrt(mean(v^2) + eps):
 *   u = rms(y) * w_post                 (y itself if w_post is NULL)
 *   h = residual_scale x + block_scale gate u    (gate 1 for LC_MOE_GATE_NONE)
 *   z = rms(h) * w_pre
 * in fp32; h and z are rounded once, z from the h before its rounding.  y NULL: h is
 * residual_scale x (the first norm of a model); w_post and gate are then NULL.
 *   x, y       [T][d] dtype
 *   gate       [d] fp32 (CHANNEL) or [T] fp32 (TOKEN)
 *   w_pre, w_post [d] fp32; w_pre NULL: no z
 *   h          [T][d] dtype (out), or NULL: not written; may be x or y itself
 *   z          [T][d] dtype (out), or NULL: not written; may be x or y itself (not h)
 * 0 <= T < 2^24, 1 <= d <= 16384, d a multiple of 8 (bf16) or 4 (fp32); eps below 2^-126, a scale
 * that is not finite or an unknown gate kind: LC_MOE_E_SHAPE.  The squares of a row must have a
 * sum within fp32's range. */
lc_moe_status lc_moe_block_norm(int32_t T, int32_t d, int32_t dtype, const lc_moe_norm* norm,
                                const void* x, const void* y, const float* gate,
                                const float* w_post, const float* w_pre, void* h, void* z,
                                hipStream_t stream);

/* Its gradient, from the gradients dh and dz of h and z.  With r = 1 / sqrt(mean(h^2) + eps),
 * q = 1 / sqrt(mean(y^2) + eps) and means over a token's d elements:
 *   dH = dh + r (w_pre dz - h r^2 mean(w_pre dz h))
 *   dx = residual_scale dH;      du = block_scale gate dH
 *   dy = q (w_post du - y q^2 mean(w_post du y))       (du if w_post is NULL)
 *   dw_pre = sum_t dz h r;       dw_post = sum_t du y q
 *   dgate = block_scale sum u dH over the tokens (CHANNEL) or a token's elements (TOKEN)
 * in fp32, sums over tokens in a fixed order; r and q are taken from h and y again.
 *   h          [T][d] dtype: the forward's output as stored
 *   dh, dz     [T][d] dtype, either may be NULL: 0 (dz NULL: w_pre may be NULL, dw_pre is zeros)
 *   y, gate, w_post, w_pre   as in the forward; y NULL: dy, dgate, dw_post are NULL
 *   dx         [T][d] dtype (out) or NULL; may be dh or dz itself
 *   dy         [T][d] dtype (out) or NULL; may be y, dh or dz itself (not dx)
 *   dw_pre, dw_post [d] fp32 (out) or NULL; dgate [d] or [T] fp32 (out) or NULL
 * T = 0 writes zeros to the sums.  The workspace holds partial sums. */
size_t lc_moe_block_norm_backward_workspace_size(int32_t T, int32_t d, int32_t dtype);
lc_moe_status lc_moe_block_norm_backward(int32_t T, int32_t d, int32_t dtype, const lc_moe_norm* norm,
                                         const void* h, const void* dh, const void* dz,
                                         const void* y, const float* gate, const float* w_post,
                                         const float* w_pre, void* dx, void* dy, float* dw_pre,
                                         float* dw_post, float* dgate, void* workspace,
                                         size_t workspace_bytes, hipStream_t stream);

/* ---- products in block FP8 --------------------------------------------------------------- */

/* A matrix of R rows and C reduction columns in block FP8 is one buffer of
 * lc_moe_fp8_matrix_size(R, C) bytes (0: out of range):
 *   codes   [R][Cp] E4M3, Cp = C rounded up to 128; columns from C on are 0
 *   scales  at the next multiple of 256: [Cp/128][Rp] E8M0 exponent bytes k + 127, Rp = R rounded
 *           up to 256; the byte of row r lies at (r & ~127) + 4 (r & 31) + (r >> 5 & 3) of its run
 *           (so that a lane of the matrix cores finds those of four row blocks in one word);
 *           bytes of rows from R on are 127; 256 bytes of 127 behind the last run
 * Scales and rounding are those of lc_moe_quantize_activations: 2^k, k the smallest integer with
 * the block's largest |v| <= 448 * 2^k (0 for a block of zeros, at least -127), and the nearest
 * E4M3 value of v / 2^k, ties to the even code.  1 <= R, C < 2^24 and Rp Cp <= 2^37. */
size_t lc_moe_fp8_matrix_size(int32_t rows, int32_t cols);

/* x [rows][cols] bf16 to block FP8.  cols a multiple of 8.
 *   block_rows  1: a scale for each 128 columns of a row (activations, gradients), in `out_t`
 *               for each 128 rows of a column; 128: a scale for each block of 128 x 128 (weights)
 *   out         the matrix [rows][cols], or NULL
 *   out_t       its transpose [cols][rows] (reduction over the rows), or NULL
 * rows = 0 does nothing. */
lc_moe_status lc_moe_quantize_matrix(const void* x, int32_t rows, int32_t cols, int32_t block_rows,
                                     void* out, void* out_t, hipStream_t stream);

/* out = A B^T + add for block-FP8 A [M][K] and B [N][K], out and add [M][N] bf16 (add may be
 * NULL, or out itself); N a multiple of 8.  The products of codes are exact; the FP8 matrix cores
 * add 64 of them and the fp32 accumulator with about 12 bits below the largest addend (see
 * lc_moe_quantize_activations); add is added in fp32 and the sum rounded once.  M = 0 does
 * nothing.  M, N and K are limited as a matrix's sizes are, M and N together too. */
size_t lc_moe_matmul_fp8_workspace_size(int32_t M, int32_t N, int32_t K);
lc_moe_status lc_moe_matmul_fp8(int32_t M, int32_t N, int32_t K, const void* a, const void* b,
                                const void* add, void* out, void* workspace,
                                size_t workspace_bytes, hipStream_t stream);

/* y = Q(x) W^T + add: the tokens quantised in blocks of 1 x 128, W a block-FP8 weight [n][k].
 *   x [T][k] bf16, w the `out` of lc_moe_quantize_matrix(W, n, k, 128, ...), add and y [T][n]
 *   bf16 (add may be NULL, or y itself)
 * k and n multiples of 8; y == x: LC_MOE_E_SHAPE.  Few tokens or a small matrix are quantised and
 * multiplied in one launch; the matrix cores then add 128 products at a time, so that the last
 * bits need not be those of lc_moe_matmul_fp8. */
size_t lc_moe_linear_fp8_workspace_size(int32_t T, int32_t k, int32_t n);
lc_moe_status lc_moe_linear_fp8(int32_t T, int32_t k, int32_t n, const void* x, const void* w,
                                const void* add, void* y, void* workspace, size_t workspace_bytes,
                                hipStream_t stream);

/* Its gradient with FP8 operands:
 *   dx = Q(dy) W + dx_add      dy in blocks of 1 x 128, W's codes transposed (`out_t` of
 *                              lc_moe_quantize_matrix(W, n, k, 128, ...): the same values)
 *   dw = Q'(dy)^T Q'(x)        both in blocks of 128 tokens x 1 column
 *   dy [T][n], x [T][k], dx_add and dx [T][k] (dx_add may be NULL, or dx itself), dw [n][k], bf16
 * dx NULL: not computed (w_t is then not read); dw NULL: not computed (x is then not read; dx as
 * lc_moe_linear_fp8 computes it, so that its last bits may differ).  dx == dy: LC_MOE_E_SHAPE.
 * T = 0 writes zeros to dw. */
size_t lc_moe_linear_fp8_backward_workspace_size(int32_t T, int32_t k, int32_t n);
lc_moe_status lc_moe_linear_fp8_backward(int32_t T, int32_t k, int32_t n, const void* dy,
                                         const void* x, const void* w_t, const void* dx_add,
                                         void* dx, void* dw, void* workspace,
                                         size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* LC_MOE_BLOCK_H */
