/*
 * ssm_recurrent.h -- C ABI of the recurrent-layer operators that stand next to
 * the scans of ssm_scan.h, in the same library:
 *
 *   ssm_gated_scan_fwd / _fwd_varlen / _bwd / _bwd_varlen, ssm_gated_state_update
 *       the gated linear recurrence: one float32 state per channel, a decay
 *       gate and an input gate per channel and token
 *   ssm_qk_norm_rotate_fwd / _bwd
 *       the norm of queries and keys for each head with the position rotation
 *       in the same pass (for ssm_ssd_fwd, whose recurrence is masked linear
 *       attention: its C are the queries, its B the keys)
 *   ssm_causal_conv1d_bwd
 *       the gradients of ssm_causal_conv1d_fwd
 *
 * The conventions are those of ssm_scan.h: device pointers on the current HIP
 * device, contiguous row-major tensors (token strides where an argument gives
 * one), "act" tensors of the element type `dtype`, everything else float32;
 * arithmetic and states in float32, bf16 results rounded to nearest even; the
 * caller owns every buffer, the library allocates nothing and never
 * synchronises; argument errors return a negative ssm_status_t before anything
 * is enqueued, with a message in ssm_last_error().  Alignment: act tensors to
 * their element size, float32 and int32 tensors to 4 bytes, workspaces to 256
 * bytes.  Outputs may not overlap inputs, each other or the workspace unless a
 * function says so.  A workspace holds nothing between calls, but two calls
 * that may run at the same time need one each.
 */
#ifndef SSM_RECURRENT_H
#define SSM_RECURRENT_H

#include "ssm_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Tokens between the states that the forward hands to the backward. */
#define SSM_GATED_CHUNK 16

/*
 * Gated linear recurrence over whole sequences.  Per sequence b and channel d,
 * with a state h (float32), sigma the logistic function:
 *   a_t = exp(A[d] * sigma(rgate[b,t,d] + rgate_bias[d]))
 *   h   = a_t * h + m_t * sigma(igate[b,t,d] + igate_bias[d]) * x[b,t,d]
 *   out[b,t,d] = z ? h * z*sigma(z) : h
 * with m_t = sqrt(1 - a_t^2) when normalize is 1 (the state keeps the inputs'
 * variance whatever the gate) and m_t = 1 when it is 0.
 *   x, rgate, igate, z, out : (batch, seqlen, dim) act; z may be NULL
 *   A                 : (dim) float32, A <= 0: the log of the smallest decay.
 *                       (A > 0, up to 88, grows; with normalize its m_t is 0.
 *                       A state that passes float32's range is infinite or
 *                       NaN from there on.)
 *   rgate_bias, igate_bias : (dim) float32 or NULL (= 0)
 *   initial_state     : (batch, dim) float32 or NULL (= zeros)
 *   last_state        : (batch, dim) float32 or NULL; h after the last token.
 *                       May be the initial_state buffer (resume in place).
 *   chunk_states      : (batch, ceil(seqlen / SSM_GATED_CHUNK), dim) float32
 *                       or NULL; receives the state before every
 *                       SSM_GATED_CHUNK-th token, for ssm_gated_scan_bwd
 *   batch, dim >= 1; seqlen >= 0 (0 only copies the initial state);
 *   dim <= 2^22; batch <= 65535; batch * ceil(seqlen / 128) * ceil(dim / 64)
 *   < 2^31 (SSM_ERR_SHAPE beyond).
 *   workspace         : at least ssm_gated_scan_fwd_workspace_bytes(...) bytes
 * Bitwise reproducible run to run on one device.
 * An infinite state or input gives an infinite state from there on (NaN where
 * infinities of both signs meet; where a decay rounds to 0, below about
 * 2^-126, infinite or NaN).
 */
int ssm_gated_scan_fwd(const void* x, const void* rgate, const void* igate, const float* A,
                       const float* rgate_bias, const float* igate_bias, int normalize,
                       const void* z, void* out, float* last_state, const float* initial_state,
                       float* chunk_states, int64_t batch, int64_t seqlen, int64_t dim, int dtype,
                       void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Workspace size of the call above (0 when none is needed, or for invalid sizes). */
size_t ssm_gated_scan_fwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim, int dtype);

/*
 * The same over packed variable-length sequences.
 *   x, rgate, igate, z, out : (total_len, dim) act, the sequences one after
 *                      another
 *   cu_seqlens       : (nseq + 1) int32 DEVICE array of token offsets with
 *                      0 = cu[0] <= ... <= cu[nseq] <= total_len (empty
 *                      sequences are allowed).  Rows behind cu[nseq] are
 *                      padding: their contents never reach a result, and
 *                      outputs keep what they held there.  The offsets are not
 *                      checked: ones that break the rule give unspecified
 *                      values, but every access stays inside the buffers.
 *   initial_state, last_state : (nseq, dim) float32 or NULL.  last_state may
 *                      not overlap initial_state.
 *   chunk_states     : (ceil(total_len / SSM_GATED_CHUNK), dim) float32 or
 *                      NULL; receives the state that enters token
 *                      SSM_GATED_CHUNK c from the one before it (zero for
 *                      c = 0)
 *   1 <= nseq < 2^24; total_len >= 0.
 * Nothing passes from one sequence into another, a NaN or an infinity neither.
 * Many sequences of a few tokens each, equally long ones too, are quicker here
 * than as rows of ssm_gated_scan_fwd (512 of 4 tokens and 2048 channels: 26
 * and 189 us).
 */
int ssm_gated_scan_fwd_varlen(const void* x, const void* rgate, const void* igate, const float* A,
                              const float* rgate_bias, const float* igate_bias, int normalize,
                              const void* z, void* out, float* last_state,
                              const float* initial_state, float* chunk_states,
                              const int32_t* cu_seqlens, int64_t nseq, int64_t total_len,
                              int64_t dim, int dtype, void* workspace, size_t workspace_bytes,
                              hipStream_t stream);

size_t ssm_gated_scan_fwd_varlen_workspace_bytes(int64_t nseq, int64_t total_len, int64_t dim,
                                                 int dtype);

/*
 * Gradients of ssm_gated_scan_fwd for the scalar loss = sum(dout * out) +
 * sum(dlast_state * last_state), with respect to every input.  The states are
 * not kept but walked again from chunk_states.
 *   inputs as ssm_gated_scan_fwd, plus
 *     chunk_states : what the forward left for the same inputs, or NULL: then
 *                    they are computed here first (three more reads of
 *                    activations)
 *     dout         : (batch, seqlen, dim) act
 *     dlast_state  : (batch, dim) float32 or NULL (= 0)
 *   outputs (all overwritten, none accumulated into):
 *     dx, drgate, digate : (batch, seqlen, dim) act
 *     dz           : (batch, seqlen, dim) act; required when z is given, NULL
 *                    otherwise
 *     dA           : (dim) float32
 *     drgate_bias, digate_bias : (dim) float32 or NULL
 *     dinitial_state : (batch, dim) float32 or NULL
 * Where 1 - a_t^2 is below 2^-126 (normalize, and a gate closed that far, or
 * A >= 0) the gradients take m_t as 0, and the term that divides by m_t too,
 * its limit for a closing gate.  A decay of 0 (A = -infinity) has no slope.
 * An infinite dout or dlast_state gives infinite gradients at the tokens before
 * it, as infinite states do behind it.  Where a state is infinite, drgate and
 * dz (and the sums over such tokens) are not finite; dx, digate and
 * dinitial_state do not depend on the states.
 * Sums over tokens and sequences are formed in a fixed order from float32
 * partials: bitwise reproducible run to run on one device.
 */
int ssm_gated_scan_bwd(const void* x, const void* rgate, const void* igate, const float* A,
                       const float* rgate_bias, const float* igate_bias, int normalize,
                       const void* z, const float* initial_state, const float* chunk_states,
                       const void* dout, const float* dlast_state, void* dx, void* drgate,
                       void* digate, void* dz, float* dA, float* drgate_bias, float* digate_bias,
                       float* dinitial_state, int64_t batch, int64_t seqlen, int64_t dim, int dtype,
                       void* workspace, size_t workspace_bytes, hipStream_t stream);

/* with_chunk_states: 1 when the call gets chunk_states, 0 when it does not. */
size_t ssm_gated_scan_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim, int dtype,
                                          int with_chunk_states);

/* Gradients of ssm_gated_scan_fwd_varlen; layouts as there, dlast_state and
 * dinitial_state (nseq, dim).  Rows of dx, drgate, digate and dz behind
 * cu[nseq] keep what they held. */
int ssm_gated_scan_bwd_varlen(const void* x, const void* rgate, const void* igate, const float* A,
                              const float* rgate_bias, const float* igate_bias, int normalize,
                              const void* z, const float* initial_state,
                              const float* chunk_states, const void* dout,
                              const float* dlast_state, void* dx, void* drgate, void* digate,
                              void* dz, float* dA, float* drgate_bias, float* digate_bias,
                              float* dinitial_state, const int32_t* cu_seqlens, int64_t nseq,
                              int64_t total_len, int64_t dim, int dtype, void* workspace,
                              size_t workspace_bytes, hipStream_t stream);

size_t ssm_gated_scan_bwd_varlen_workspace_bytes(int64_t nseq, int64_t total_len, int64_t dim,
                                                 int dtype, int with_chunk_states);

/*
 * One decoding step of the gated recurrence for `batch` sequences:
 *   state : (batch, dim) float32, read and overwritten in place
 *   x, rgate, igate, z, out : (batch, dim) act; z may be NULL
 * Equivalent to ssm_gated_scan_fwd with seqlen = 1 and initial_state =
 * last_state = state.  batch * dim < 2^31 - 2048 (SSM_ERR_SHAPE otherwise).
 */
int ssm_gated_state_update(float* state, const void* x, const void* rgate, const void* igate,
                           const float* A, const float* rgate_bias, const float* igate_bias,
                           int normalize, const void* z, void* out, int64_t batch, int64_t dim,
                           int dtype, hipStream_t stream);

/*
 * Norm of queries and keys for each head, with the position rotation in the
 * same pass.  For every token and head, with v the head's row of `headdim`
 * values and w its weight:
 *   n = v / sqrt(mean(v^2) + eps) * w
 *   out = n with its first rotary_dim values turned in pairs (p, q) by the
 *   angle theta_i = position * inv_freq[i], i < rotary_dim / 2:
 *     out[p] = n[p] cos - n[q] sin,  out[q] = n[p] sin + n[q] cos
 *   pairs: (i, i + rotary_dim/2) with interleaved = 0, (2i, 2i+1) with 1
 *   q               : (batch, seqlen, nheads_q, headdim) act, a token's heads
 *                     together, tokens q_token_stride values apart (at least
 *                     nheads_q * headdim, at most 2^30: rows of a fused
 *                     projection are read where they are); batch rows follow each other at seqlen
 *                     token strides.  k likewise with nheads_k.
 *   q_out, k_out    : (batch, seqlen, heads, headdim) act, contiguous.  q_out
 *                     may be q (and k_out k) where its rows are contiguous.
 *   q_weight, k_weight : (headdim) float32 or NULL (= 1)
 *   inv_freq        : (rotary_dim / 2) float32; NULL when rotary_dim is 0
 *   positions       : (batch, seqlen) int32 DEVICE array or NULL (= the token's
 *                     index in its sequence)
 *   nheads_q >= 1; nheads_k >= 0 (0: k, k_weight and k_out NULL); headdim even,
 *   2..256; rotary_dim even, 0..headdim; eps >= 0; batch * seqlen < 2^31;
 *   at most 65536 heads each.
 * mean(v^2) + eps is a float32: rows where it is below 2^-126 (eps = 0 alone
 * allows it) or where a sum of squares overflows give unspecified values.
 * The angle is formed and reduced in two parts of float64, so no position loses
 * anything; its sine and cosine are float32 (within 2^-23).
 */
int ssm_qk_norm_rotate_fwd(const void* q, const void* k, const float* q_weight,
                           const float* k_weight, const float* inv_freq, const int32_t* positions,
                           float eps, int interleaved, void* q_out, void* k_out, int64_t batch,
                           int64_t seqlen, int64_t nheads_q, int64_t nheads_k, int64_t headdim,
                           int64_t rotary_dim, int64_t q_token_stride, int64_t k_token_stride,
                           int dtype, hipStream_t stream);

/*
 * Its gradients for the loss sum(dq_out * q_out) + sum(dk_out * k_out).
 *   dq_out, dk_out  : (batch, seqlen, heads, headdim) act, contiguous
 *   dq, dk          : (batch, seqlen, heads, headdim) act, contiguous
 *   dq_weight, dk_weight : (headdim) float32 or NULL (not wanted); summed over
 *                     tokens and heads in a fixed order
 * workspace: at least ssm_qk_norm_rotate_bwd_workspace_bytes(...) bytes.
 */
int ssm_qk_norm_rotate_bwd(const void* q, const void* k, const float* q_weight,
                           const float* k_weight, const float* inv_freq, const int32_t* positions,
                           float eps, int interleaved, const void* dq_out, const void* dk_out,
                           void* dq, void* dk, float* dq_weight, float* dk_weight, int64_t batch,
                           int64_t seqlen, int64_t nheads_q, int64_t nheads_k, int64_t headdim,
                           int64_t rotary_dim, int64_t q_token_stride, int64_t k_token_stride,
                           int dtype, void* workspace, size_t workspace_bytes, hipStream_t stream);

size_t ssm_qk_norm_rotate_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t nheads_q,
                                              int64_t nheads_k, int64_t headdim);

/*
 * Gradients of ssm_causal_conv1d_fwd for the loss sum(dout * out) +
 * sum(dfinal_conv_state * final_conv_state); the convolution before the SiLU
 * is computed again.
 *   inputs as ssm_causal_conv1d_fwd, plus
 *     dout              : (batch, seqlen, dim) act
 *     dfinal_conv_state : (batch, dim, width-1) act or NULL (= 0)
 *   outputs (all overwritten):
 *     dx                : (batch, seqlen, dim) act
 *     dweight           : (dim, width) float32;  dbias : (dim) float32 or NULL
 *     dinitial_conv_state : (batch, dim, width-1) act or NULL
 *   2 <= width <= 4; batch, dim >= 1; seqlen >= 0; dim <= 2^22, the other
 *   limits as the forward.
 * Sums over tokens and sequences in a fixed order.
 */
int ssm_causal_conv1d_bwd(const void* x, const float* weight, const float* bias,
                          const void* initial_conv_state, const void* dout,
                          const void* dfinal_conv_state, void* dx, float* dweight, float* dbias,
                          void* dinitial_conv_state, int64_t batch, int64_t seqlen, int64_t dim,
                          int64_t width, int silu, int dtype, void* workspace,
                          size_t workspace_bytes, hipStream_t stream);

size_t ssm_causal_conv1d_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim,
                                             int64_t width);

#ifdef __cplusplus
}
#endif
#endif /* SSM_RECURRENT_H */
