/*
 * moe_block.h -- C ABI of what stands around the experts in libmoe.so: routing with other scores
 * than moe_route's (sigmoid, a balance bias, groups), the norms before and after a block with its
 * gate and residual scale, and the experts with 4-bit weights for few tokens.
 *
 * Conventions as in moe.h (status codes, caller-owned device pointers, asynchronous on `stream`,
 * no allocation: scratch is the caller's workspace).  Arrays are aligned as their values' type
 * wants it unless said otherwise (else MOE_ERR_UNSUPPORTED).  Outputs may not overlap inputs
 * unless said otherwise.  Everything is deterministic: sums have a fixed order.
 */
#ifndef MOE_BLOCK_H
#define MOE_BLOCK_H

#include <stddef.h>
#include <stdint.h>

#include "linear_attention.h" /* moe_dtype */
#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ==================================================================== routing by scores
 * "Day-Level Adaptation and LoRA Fine-Tuning of Ultra-Large-Scale Sparse MoE Models", sections
 * 2.1 and 3.3 (routing scores, Top-k selection), with the forms of it that the pages leave open.
 * For every token, over its E logits l:
 *
 *   s_e   = exp(l_e) / sum_i exp(l_i)   or   1 / (1 + exp(-l_e))
 *   c_e   = s_e + b_e                             b: the balance bias, 0 where it is NULL
 *   v_g   = the sum of the `group_best` largest c in group g of E / groups neighbouring experts
 *   topk_idx = the k largest c of the groups_kept groups with the largest v, descending
 *   topk_gate_j = scale * s_(idx j) [ / sum_i s_(idx i) if renormalise ]
 *   prob_partials[b, e] = sum of s_e / sum_i s_i over the tokens 8 b .. 8 b + 7
 *
 * Equal values: the lower index first (experts and groups).  The bias moves the selection alone,
 * not the gates.  Without a bias the experts are compared by their logits.  With one, and where
 * the values of two scores are added for a group, nearly equal values are told apart in
 * more than fp32: what is closer than 2^-40 (or than that times |b|, where that is
 * above 1) may come out in either order.
 *
 * A logit of -inf has the score 0 (NaN counts as -inf).  Where all selected scores are 0 the gates
 * are 0, as are the softmax scores of a row of -inf alone; experts of score 0 are selected, by
 * index, where fewer than k others are left.  A logit of +inf has the sigmoid score 1; it makes
 * the softmax scores of its row NaN.  A bias of -inf or +inf puts an expert last or first, and a
 * group by the values that it is compared by (of +inf and -inf added: last); NaN counts as -inf.
 *
 * logits [T, E], of type `dtype` (a moe_dtype), their rows ld_logits values apart (>= E; 0: one
 * row that all tokens share); select_bias [E] fp32 or NULL; topk_idx [T, k] int32, topk_gate
 * [T, k] fp32; prob_partials [ceil(T/8), E] fp32 (as moe_route's, for moe_aux_loss) or NULL.
 * Supported (else MOE_ERR_UNSUPPORTED): E <= 1024, k <= 32, groups <= 32, T up to 2^24.  groups
 * divides E; 1 <= groups_kept <= groups; group_best is 1 or 2, at most E / groups (not read
 * where groups is 1);
 * k <= groups_kept * E / groups; scale finite (else MOE_ERR_INVALID_ARG). */
enum moe_score {
  MOE_SCORE_SOFTMAX = 0,
  MOE_SCORE_SIGMOID = 1
};

typedef struct moe_route_rule {
  int32_t score;       /* a moe_score */
  int32_t groups;      /* 1: none */
  int32_t groups_kept;
  int32_t group_best;
  int32_t renormalise;
  float scale;
} moe_route_rule;

int moe_route_select(int32_t T, int32_t E, int32_t k, const moe_route_rule* rule, int32_t dtype,
                     const void* logits, int64_t ld_logits, const float* select_bias,
                     int32_t* topk_idx, float* topk_gate, float* prob_partials,
                     moe_stream_t stream);

/* Gradient of <dgate, topk_gate> with respect to the logits, the selection held fixed.
 * dlogits [T, E] dense, of type `dtype`, overwritten (zeros among it), or NULL.  dlogits_topk
 * [T, k] fp32 or NULL: its values at the selected experts alone, which is all of it but for
 * softmax scores that are not renormalised (MOE_ERR_INVALID_ARG there).  One of them is wanted.
 * An expert that a row names twice gets the sum in dlogits (and the parts in dlogits_topk).
 * Entries of topk_idx outside [0, E) are reported as MOE_ERR_BAD_INDEX in *dev_status (may be
 * NULL) and count as not selected. */
int moe_route_select_backward(int32_t T, int32_t E, int32_t k, const moe_route_rule* rule,
                              int32_t dtype, const void* logits, int64_t ld_logits,
                              const int32_t* topk_idx, const float* dgate, void* dlogits,
                              float* dlogits_topk, int32_t* dev_status, moe_stream_t stream);

/* The logits of moe_route alone (the same bits), for moe_route_select.  Workspace:
 * moe_route_workspace_size. */
int moe_route_logits(const moe_problem* p, const moe_bf16* x, const float* w_router,
                     const float* bias, float* logits, void* workspace, size_t workspace_bytes,
                     int32_t* dev_status, moe_stream_t stream);

/* moe_dispatch_route_bwd for gates that moe_route_select made: dx[t] = the sum of the rows of
 * dx_perm of its kept slots + sum_j dlogits_topk[t, j] * w_router[topk_idx[t, j]] (fp32 [T, d]). */
int moe_dispatch_logits_bwd(const moe_problem* p, const moe_bf16* dx_perm,
                            const int32_t* slot_row, const int32_t* topk_idx,
                            const float* dlogits_topk, const float* w_router, float* dx,
                            moe_stream_t stream);

/* ==================================================================== around a block
 * What stands between two blocks of a model (the layer of moe.h, linear attention): the norm after
 * one, its gate and residual scale, the residual sum, and the norm before the next, in one pass
 * ("Fine-Tuning Trillion-Parameter Sparse MoE Models: Challenges and Engineering Practices",
 * section 5, fuses the normalization into the kernels next to it).  For every row, over its D
 * values,
 *
 *   u = w_post * y / sqrt(mean(y^2) + eps)   or   y
 *   z = x + scale * a(gate) * u
 *   n = w_pre * z / sqrt(mean(z^2) + eps)
 *
 * with a the identity or, if gate_sigmoid is not zero, 1 / (1 + exp(-gate)).
 *   x, z [N, D] of type stream_dtype: the residual stream;  y, n [N, D] of type dtype.
 *   gate: a moe_gate says its shape: none, [D] fp32, [N] fp32, or [N, D] of type dtype.
 *   w_post, w_pre [D] fp32, or NULL for ones.  post_norm says whether there is a norm after.
 * y NULL: no block before; z = x, and n is its norm (gate_kind none, post_norm 0).  n NULL: no
 * norm before the next block (w_pre NULL).  z may be NULL where y is NULL, not both z and n.
 * Rows start ld_* values apart (input rows also 0 apart: one row for all); ld_gate is of a gate
 * [N, D].  The stride of a single row means nothing.
 * Supported (else MOE_ERR_UNSUPPORTED): D a multiple of 8, at most 16384; N up to 2^30; types
 * (stream_dtype, dtype) bf16 and bf16, fp32 and bf16, fp32 and fp32; pointers 16-byte aligned (a
 * gate [N] 4-byte), strides multiples of 8.  eps > 0, scale finite.
 * z may be x, and n may be y or a gate [N, D] (same strides and types).
 * All sums are fp32; n is formed from z before z is rounded; z and n are rounded once. */
enum moe_gate {
  MOE_GATE_NONE = 0,
  MOE_GATE_CHANNEL = 1, /* [D]    */
  MOE_GATE_TOKEN = 2,   /* [N]    */
  MOE_GATE_VALUE = 3    /* [N, D] */
};

typedef struct moe_block_in {
  int32_t N, D, stream_dtype, dtype;
  float eps, scale;
  int32_t gate_kind, gate_sigmoid, post_norm;
  const void* x;
  int64_t ld_x;
  const void* y;
  int64_t ld_y;
  const void* gate;
  int64_t ld_gate;
  const float* w_post;
  const float* w_pre;
} moe_block_in;

int moe_block_norm(const moe_block_in* in, void* z, int64_t ld_z, void* n, int64_t ld_n,
                   moe_stream_t stream);

/* Backward: gradients of <dz, z> + <dn, n>.  `in` as the forward read it: z is formed again from
 * it.  dz, dx of type stream_dtype; dn of type dn_dtype (MOE_F32, as layers' backward passes write
 * it, or dtype); dy of type dtype.  dz or dn may be NULL (zero).  dy, dgate, dw_post and dw_pre
 * may each be NULL (not wanted); dgate is shaped and typed as gate.  Without dn, dw_pre is zero.
 * dx may be dz, dy may be y or dn of the same type, a gate's [N, D] gradient may be the gate (each
 * with the same strides).
 * Workspace: for dw_post, dw_pre and the gradient of a gate [D] (else it may be NULL), 16-byte
 * aligned; its size is 0 for sizes that are not supported. */
typedef struct moe_block_grads {
  const void* dz;
  int64_t ld_dz;
  const void* dn;
  int64_t ld_dn;
  int32_t dn_dtype;
  void* dx;
  int64_t ld_dx;
  void* dy;
  int64_t ld_dy;
  void* dgate;
  int64_t ld_dgate;
  float* dw_post;
  float* dw_pre;
} moe_block_grads;

size_t moe_block_norm_backward_workspace_size(int32_t N, int32_t D, int32_t gate_kind);
int moe_block_norm_backward(const moe_block_in* in, const moe_block_grads* grads,
                            void* workspace, size_t workspace_bytes, moe_stream_t stream);

/* ==================================================================== 4-bit experts
 * The experts of moe_expert_ffn for few tokens, with weights of 4 bits: a serving step, whose time
 * is that of reading the weights of the experts which the batch reaches.  A weight is
 *
 *   w = scale * (code - zero),   code 0 .. 15,
 *
 * with one scale (bf16, less than 2^116 in size: larger ones become infinite) and zero (0 .. 15; 8
 * if there are none) for `group` neighbouring weights of a row, and for every token t
 *
 *   h_j  = silu(W_gate[e_j] x_t) * (W_up[e_j] x_t),   e_j = topk_idx[t, j]
 *   y_t  = sum_j topk_gate[t, j] * W_down[e_j] h_j
 *
 * Sums are fp32; each product is exact: x and h are scaled by powers of two, one for a row of x and
 * one for each 64 values of h, and taken as fp16, x in one part (bf16 values that are less than
 * 2^-27 of the largest of their row may lose bits), h in two (to 2^-23 of it); y is rounded once.  A
 * value of x or h that is not finite makes its token's y NaN.  p gives T, d, E, k and F; r has to
 * be 0 (adapters are not part of it) and the capacity is not used: every slot is computed.  Entries
 * of topk_idx outside [0, E) are reported as MOE_ERR_BAD_INDEX in *dev_status (may be NULL) and
 * contribute nothing; a token may name an expert twice.
 * Supported (else MOE_ERR_UNSUPPORTED): p as everywhere (d and F multiples of 64, and up to 2^20
 * here; a matrix of up to 2^40 weights), T * k up to 16384; group 32, 64 or 128, a divisor of d and
 * of F; group and has_zeros the same for all three; packed arrays, x, y and the workspace 16-byte aligned.
 * An expert's weights are read and converted for every 8 of its rows.  Up to about 20 rows to an
 * expert that takes less time than moe_dispatch, moe_expert_ffn and moe_combine with weights in
 * bf16 (8 of 64 experts, 4096 x 1024: 64 tokens 141 us and 293, 256 tokens 379 and 306, 2048 tokens
 * 2689 and 506); beyond, what it saves is memory.
 *
 * moe_w4_pack lays weights [E, rows, cols] out for it, once (cols: what a product sums over).
 * codes [E, rows, cols / 2]: two codes to a byte, the lower four bits first; scales
 * [E, rows, cols / group] bf16; zeros [E, rows, cols / group] bytes (their lower four bits) or
 * NULL.  packed_codes takes as many bytes as codes; packed_scales E * rows * cols / group entries
 * of 2 bytes (4 with zeros); both 16-byte aligned.  rows a multiple of 16, cols of 64. */
typedef struct moe_w4 {
  const void* codes;  /* packed */
  const void* scales; /* packed */
  int32_t group;
  int32_t has_zeros;
} moe_w4;

int moe_w4_pack(int32_t E, int32_t rows, int32_t cols, int32_t group, const uint8_t* codes,
                const moe_bf16* scales, const uint8_t* zeros, void* packed_codes,
                void* packed_scales, moe_stream_t stream);

size_t moe_w4_expert_ffn_workspace_size(const moe_problem* p);
int moe_w4_expert_ffn(const moe_problem* p, const moe_bf16* x, const int32_t* topk_idx,
                      const float* topk_gate, const moe_w4* w_gate, const moe_w4* w_up,
                      const moe_w4* w_down, moe_bf16* y, void* workspace,
                      size_t workspace_bytes, int32_t* dev_status, moe_stream_t stream);

/* Self-test of the waits for copies of weights, which give up after 2 s.  After it, launches of
 * moe_w4_expert_ffn by the calling thread (group 32, no zeros; else MOE_ERR_UNSUPPORTED) wait
 * limit_ms (1..2000) at most, and copy `copy` of warp `warp` of block `block` of the product with
 * w_gate and w_up (down 0) or w_down (1) never arrives whole.  Such a launch ends on its own, reports
 * MOE_ERR_TIMEOUT where there is such a copy, and leaves y undefined.  limit_ms = 0 ends the
 * self-test. */
int moe_selftest_w4_waits(int32_t limit_ms, int32_t down, int32_t block, int32_t warp, int32_t copy);

#ifdef __cplusplus
}
#endif

#endif /* MOE_BLOCK_H */
