/*
 * linear_attention.h -- C ABI of the chunked gated delta-rule linear attention in
 * libmoe.so (the second workload of the hot path).
 *
 * "Fine-Tuning Trillion-Parameter Sparse MoE Models: Challenges and Engineering Practices",
 * section 5 (large fused forward and backward kernels for linear attention: normalization
 * coefficients, gating and decay, intra-chunk query-state interaction and the output; fixed
 * chunks computed with dense intra-chunk products and one small state recurrence between
 * chunks) and "Adapting Ultra-Large MoE Models: Engineering Practices and Optimization
 * Pathways", section 3.2 (state recursion and chunked computation).  The pages give no
 * equations; the operator implemented is the gated delta rule, per sequence b and head h:
 *
 *   q^_t = q_t / ||q_t||,  k^_t = k_t / ||k_t||            (L2 over the key width dk)
 *   S_t  = exp(g_t) S_{t-1} (I - beta_t k^_t k^_t^T) + beta_t v_t k^_t^T     S_t [dv, dk]
 *   o_t  = scale * S_t q^_t
 *
 * Conventions as in moe.h (status codes, caller-owned device pointers, asynchronous on
 * `stream`, no allocation: scratch is the caller's workspace).  Layouts (row-major):
 *   q, k [B, T, H, dk] bf16;  v [B, T, H, dv] bf16;  beta, g [B, T, H] fp32 (beta in [0, 1],
 *   g <= 0 the log decay);  S0 [B, H, dv, dk] fp32 initial state or NULL (zero);
 *   o [B, T, H, dv] bf16;  S_T [B, H, dv, dk] fp32 final state or NULL;
 *   S_chunks [B, H, ceil(T/64), dv, dk] fp32 or NULL: the state at the start of every
 *   64-token chunk (what a backward pass restarts from);  W_chunks [B, H, ceil(T/64), 64, dv]
 *   fp32 or NULL: every chunk's W = U - Y S0^T (its tokens' values corrected by the state at
 *   the chunk start; rows past the sequence zero), which the backward then reads instead of
 *   forming it again.
 * Supported: dk and dv in {64, 128}; any T >= 1 (the last chunk may be partial).  A zero
 * q or k row is treated as a zero vector (no division by zero).  q, k, v, the workspace, the
 * forward's o, W_chunks (and the backward's d_o, S_chunks, W_chunks) must be 16-byte aligned (the kernels move
 * them in 16-byte pieces), else MOE_ERR_UNSUPPORTED.
 *
 * Precision: the state and every accumulation are fp32.  The forward scan's products run on
 * the tensor cores with each fp32 operand carried as two bf16 pieces (hi = bf16(x), mid =
 * bf16(x - hi); three MMAs hi.hi + hi.mid + mid.hi): about 2^-16 relative per product.
 */
#ifndef MOE_LINEAR_ATTENTION_H
#define MOE_LINEAR_ATTENTION_H

#include <stddef.h>
#include <stdint.h>

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Workspace bytes of moe_gdr_forward (the per-chunk factors: about
 * 4 * (3 dk + dv + 65) bytes per token and head), 0 for non-positive sizes. */
size_t moe_gdr_workspace_size(int32_t B, int32_t T, int32_t H, int32_t dk, int32_t dv);

/* Forward of the gated delta rule over all B x H sequences (two launches: the per-chunk
 * factors of every chunk in parallel, then the scan over chunks in slices of 16 value rows
 * of the state, on the tensor cores).  The scan's waits on its own tensor-core work are
 * bounded; one that runs out ends the scan early and records MOE_ERR_TIMEOUT for
 * moe_gdr_device_status. */
int moe_gdr_forward(int32_t B, int32_t T, int32_t H, int32_t dk, int32_t dv, const moe_bf16* q,
                    const moe_bf16* k, const moe_bf16* v, const float* beta, const float* g,
                    const float* S0, float scale, moe_bf16* o, float* S_T, float* S_chunks,
                    float* W_chunks, void* workspace, size_t workspace_bytes,
                    moe_stream_t stream);

/* Device-side status of the linear-attention kernels: waits for `stream`, writes the first
 * error a kernel recorded since the previous call (MOE_OK if none; MOE_ERR_TIMEOUT when a
 * bounded wait ran out, the outputs of that launch then being incomplete) to *status and
 * clears it.  Returns MOE_ERR_INVALID_ARG for a NULL status, MOE_ERR_CUDA if the stream or
 * the copy failed. */
int moe_gdr_device_status(int32_t* status, moe_stream_t stream);

/* Backward: gradients of <d_o, o> + <dS_T, S_T> with respect to q, k, v, beta, g and S0
 * (three launches: the per-chunk factors rebuilt, a backward scan over chunks for the state
 * gradient in slices of 16 value rows on the tensor cores (bounded waits as in the forward,
 * reported through moe_gdr_device_status), then every chunk's local backward in
 * parallel).
 * S_chunks: the forward's chunk-start states (required); W_chunks: the forward's W_chunks, or
 * NULL (then formed again from S_chunks).  d_o [B, T, H, dv] bf16; dS_T
 * [B, H, dv, dk] fp32 or NULL (zero).  Outputs fp32, overwritten: dq, d_k [B, T, H, dk],
 * d_v [B, T, H, dv], dbeta, dg [B, T, H], dS0 [B, H, dv, dk] (may be NULL).  Deterministic:
 * every reduction runs in a fixed order. */
size_t moe_gdr_backward_workspace_size(int32_t B, int32_t T, int32_t H, int32_t dk,
                                       int32_t dv);
int moe_gdr_backward(int32_t B, int32_t T, int32_t H, int32_t dk, int32_t dv, const moe_bf16* q,
                     const moe_bf16* k, const moe_bf16* v, const float* beta, const float* g,
                     float scale, const moe_bf16* d_o, const float* dS_T, const float* S_chunks,
                     const float* W_chunks,
                     float* dq, float* d_k, float* d_v, float* dbeta, float* dg, float* dS0,
                     void* workspace, size_t workspace_bytes, moe_stream_t stream);

/* ---------------------------------------------------------------- queries and keys
 * Root-mean-square norm of every query and key head with the rotation by the token's position
 * in the same pass ("Fine-Tuning Trillion-Parameter Sparse MoE Models: Challenges and
 * Engineering Practices", section 5, fuses the normalization coefficients into the
 * linear-attention kernels): what stands between the projections and moe_gdr_forward.  For
 * every token t and head h, over the head's D values,
 *
 *   n = w * x / sqrt(mean(x^2) + eps)
 *   (y_a, y_b) = (n_a cos th_i - n_b sin th_i,  n_b cos th_i + n_a sin th_i),
 *   th_i = positions[t] * inv_freq[i],   0 <= i < rotary_dim / 2,
 *
 * where pair i is (a, b) = (i, i + rotary_dim / 2), or (2 i, 2 i + 1) if `interleaved` is not
 * zero; values from rotary_dim on are normed only.  th_i is formed in 64 bits and reduced to a
 * fraction of a turn before its sine and cosine are taken in fp32, so far positions lose
 * nothing.
 *
 * Supported (else MOE_ERR_UNSUPPORTED): D a multiple of 8, at most 256; rotary_dim a multiple
 * of 16, at most D, 0 for no rotation (positions and inv_freq may then be NULL); at most 4096
 * heads in a group and 2^30 tokens; pointers 16-byte aligned (positions and inv_freq as their types
 * want it); strides multiples of 8 values.  eps > 0.  Heads are addressed by strides (in values), so
 * q and k can be parts of one fused projection row; token t's head h starts at
 * t * token_stride + h * head_stride.  Input strides may be 0 (broadcast); rows of an output
 * must not overlap (MOE_ERR_INVALID_ARG).  y may be x, with the same strides, and dx may be x
 * or dy (of the same type, with the same strides); other overlaps of inputs and outputs give
 * undefined values. */
enum moe_dtype {
  MOE_BF16 = 0,
  MOE_F32 = 1
};

typedef struct moe_qk_rows {
  const void* x;                          /* [N, heads, D] by strides */
  int64_t x_token_stride, x_head_stride;
  void* y;                                /* [N, heads, D] by strides */
  int64_t y_token_stride, y_head_stride;
  const float* weight;                    /* [D], or [heads, D] if weight_per_head; NULL: ones */
  int32_t weight_per_head;
  int32_t heads;
} moe_qk_rows;

typedef struct moe_qk_grads {
  const void* x;                          /* the forward's input */
  int64_t x_token_stride, x_head_stride;
  const void* dy;                         /* gradient of y, of type dy_dtype */
  int64_t dy_token_stride, dy_head_stride;
  void* dx;                               /* overwritten, of x's type */
  int64_t dx_token_stride, dx_head_stride;
  const float* weight;
  float* dweight;                         /* overwritten, shaped as weight; NULL: not wanted */
  int32_t weight_per_head;
  int32_t heads;
} moe_qk_grads;

/* q and k: the two groups of heads, which share the positions (one launch); k may be NULL.
 * positions [N] int32 (any sign), inv_freq [rotary_dim / 2] fp64, both on the device.  dtype:
 * the type of x and y (a moe_dtype). */
int moe_qk_norm_rope(int32_t N, int32_t D, int32_t rotary_dim, int32_t interleaved,
                     int32_t dtype, float eps, const int32_t* positions, const double* inv_freq,
                     const moe_qk_rows* q, const moe_qk_rows* k, moe_stream_t stream);

/* Backward: dx and the weight gradients of <dy, y> (two launches; one if no weight gradient is
 * wanted).  The norm is formed again from x.  dy_dtype: MOE_F32 (what moe_gdr_backward writes)
 * or dtype.  Deterministic: every reduction runs in a fixed order.  The size is 0 where D or the
 * numbers of rows or heads are not supported. */
size_t moe_qk_norm_rope_backward_workspace_size(int32_t N, int32_t D, int32_t q_heads,
                                                int32_t k_heads);
int moe_qk_norm_rope_backward(int32_t N, int32_t D, int32_t rotary_dim, int32_t interleaved,
                              int32_t dtype, int32_t dy_dtype, float eps,
                              const int32_t* positions, const double* inv_freq,
                              const moe_qk_grads* q, const moe_qk_grads* k, void* workspace,
                              size_t workspace_bytes, moe_stream_t stream);

/* ---------------------------------------------------------------- one token
 * One step of the gated delta rule for B requests, each of one token: the state of request b
 * is row slot[b] of S [n_slots, H, dv, dk] fp32, updated in place,
 *
 *   S <- exp(g) S (I - beta k^ k^T) + beta v k^T,   o = scale * S q^,
 *
 * with q, k [B, H, dk], v [B, H, dv], o [B, H, dv] bf16 and beta, g [B, H] fp32 (types, norms
 * and zero rows as in moe_gdr_forward, whose S_T is a state to go on from).  slot [B] int32, or
 * NULL: request b has row b (then B <= n_slots).  slot[b] = -1 marks a padding row: it is
 * skipped and its o left as it was.  Any other value outside [0, n_slots) and every later
 * request with an earlier one's slot is skipped the same way and reported as MOE_ERR_BAD_INDEX
 * in *dev_status (may be NULL).  The products are plain fp32; deterministic.  q, k, v, o and S
 * must be 16-byte aligned (the rest as their types want it), dk and dv in {64, 128},
 * B * H up to 2^24 and, with slot, B up to 65535 (a request's slot is compared with all before
 * it), else MOE_ERR_UNSUPPORTED. */
int moe_gdr_step(int32_t B, int32_t H, int32_t dk, int32_t dv, const moe_bf16* q,
                 const moe_bf16* k, const moe_bf16* v, const float* beta, const float* g,
                 const int32_t* slot, int32_t n_slots, float scale, float* S, moe_bf16* o,
                 int32_t* dev_status, moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_LINEAR_ATTENTION_H */
