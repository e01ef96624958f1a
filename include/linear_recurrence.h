/*
 * linear_recurrence.h -- C ABI of the gated linear recurrence in libmoe.so: the element-wise
 * relative of the gated delta rule (linear_attention.h), with the same convention for the
 * decay.
 *
 * "Adapting Ultra-Large MoE Models: Engineering Practices and Optimization Pathways", section
 * 3.2 (state recursion and chunked computation), and "Fine-Tuning Trillion-Parameter Sparse MoE
 * Models: Challenges and Engineering Practices", section 5 (gating and decay coefficients; a
 * small state recurrence between chunks).  For every sequence and channel,
 *
 *   h_t = exp(g_t) h_{t-1} + x_t                         MOE_GLR_ADD
 *   h_t = exp(g_t) h_{t-1} + (1 - exp(g_t)) x_t          MOE_GLR_MIX
 *
 * with g_t <= 0 the log decay (-inf forgets the state) and h_0 the sequence's initial state.
 *
 * Conventions as in moe.h (status codes, caller-owned device pointers, asynchronous on
 * `stream`, no allocation; these entry points need no workspace).  Layouts:
 *   g, x, h and their gradients: N rows of D channels, type `dtype` (a moe_dtype).  g and x may
 *   be columns of a wider matrix: their rows start ld_g and ld_x values apart (>= D, or 0 for
 *   one row that all N share in an input without gradients); h and dh are dense.
 *   The rows hold n_seq packed sequences: sequence s has rows [seq_off[s], seq_off[s+1]),
 *   seq_off [n_seq + 1] int32 on the device with seq_off[0] = 0, non-decreasing, at most N;
 *   rows from seq_off[n_seq] on are padding, neither read nor written.  A sequence may be
 *   empty.  seq_off NULL: n_seq sequences of N / n_seq rows each.  A seq_off that breaks these
 *   rules is reported as MOE_ERR_BAD_INDEX in *dev_status (may be NULL); the outputs are then
 *   unspecified (nothing outside them is touched).
 *   h0, h_T, dh_T, dh0 [n_seq, D] fp32: the state before a sequence's first row and after its
 *   last, and their gradients; each may be NULL (zero, or not wanted).  h_T may be h0: the
 *   states are then updated in place.  An empty sequence hands its h0 to h_T.
 * D up to 2^20, N up to 2^30 and n_seq up to 2^24, every array aligned as its values' type wants
 * it (else MOE_ERR_UNSUPPORTED); where the rows of all `dtype` tensors begin on 16-byte
 * boundaries they are copied by TMA, which is faster.  Apart from h_T over h0, outputs may not
 * overlap inputs.
 *
 * Waits inside the kernels are bounded; one that runs out ends that launch early, its outputs then
 * being incomplete, and is reported as MOE_ERR_TIMEOUT in *dev_status.  Nothing of it is under way
 * any more when it has ended.
 *
 * Precision: states, products and sums are fp32; h, dg and dx are rounded once.  The scans form
 * exp(g) as 2^(g log2(e)), whose rounded product costs |g| 2^-24 of it, and take less than 2^-126
 * as zero; the step calls the library's exponential, so the two round differently.  Sequences do
 * not see each other: infinities or NaN in one leave the others alone.  An infinity makes all
 * that follows in its sequence and channel infinite or NaN, but not always the one that the
 * formula gives: where the decays of up to 64 rows multiply to less than 2^-149 the scans'
 * product is zero, and zero times an infinity is NaN.  Deterministic: the work is cut by sizes
 * (and by what the GPU has room for) alone and every combination has a fixed order.
 */
#ifndef MOE_LINEAR_RECURRENCE_H
#define MOE_LINEAR_RECURRENCE_H

#include <stddef.h>
#include <stdint.h>

#include "linear_attention.h"
#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

enum moe_glr_mode {
  MOE_GLR_ADD = 0,
  MOE_GLR_MIX = 1
};

/* Forward.  h_chunks [ceil(N/64), D] fp32 or NULL: the state before row 64 c (what the backward
 * restarts from); not written for rows 64 c that are padding, zero where one begins a sequence. */
int moe_glr_forward(int32_t N, int32_t D, int32_t n_seq, const int32_t* seq_off, int32_t mode,
                    int32_t dtype, const void* g, int64_t ld_g, const void* x, int64_t ld_x,
                    const float* h0, void* h, float* h_T, float* h_chunks, int32_t* dev_status,
                    moe_stream_t stream);

/* Backward: gradients of <dh, h> + <dh_T, h_T>.  h0: as the forward read it (a copy, where h_T
 * went over it).  h_chunks: the forward's (required); h_{t-1} is formed again from it in fp32.  dg
 * and dx have the strides of g and x (ld >= D).  No output may overlap an input. */
int moe_glr_backward(int32_t N, int32_t D, int32_t n_seq, const int32_t* seq_off, int32_t mode,
                     int32_t dtype, const void* g, int64_t ld_g, const void* x, int64_t ld_x,
                     const float* h0, const float* h_chunks, const void* dh, const float* dh_T,
                     void* dg, void* dx, float* dh0, int32_t* dev_status, moe_stream_t stream);

/* One token for each of B requests: the state of request b is row slot[b] of state
 * [n_slots, D] fp32, updated in place; its h [B, D] is also written in `dtype`.  g, x: B rows,
 * ld_g and ld_x apart.  slot as in moe_gdr_step: NULL for b itself, -1 for a padding row
 * (skipped, its h left as it was), anything else out of range and later requests with an earlier
 * one's slot skipped and reported as MOE_ERR_BAD_INDEX.  B up to 65535 (else
 * MOE_ERR_UNSUPPORTED). */
int moe_glr_step(int32_t B, int32_t D, int32_t mode, int32_t dtype, const void* g, int64_t ld_g,
                 const void* x, int64_t ld_x, const int32_t* slot, int32_t n_slots, float* state,
                 void* h, int32_t* dev_status, moe_stream_t stream);

/* Self-test of those waits.  After it, launches of moe_glr_forward and moe_glr_backward by the
 * calling thread wait limit_ms (1..2000) at most, and warp `warp` (0..9) of the blocks of rank `rank`
 * in their clusters leaves at step `step` as if a wait of its own had run out; every such launch ends
 * on its own and reports MOE_ERR_TIMEOUT.  limit_ms = 0 ends the self-test. */
int moe_selftest_recurrence_waits(int32_t limit_ms, int32_t rank, int32_t warp, int32_t step);

#ifdef __cplusplus
}
#endif

#endif /* MOE_LINEAR_RECURRENCE_H */
