/*
 * ssm_layer.h -- C ABI of the delta-rule layer's operators, in the same library
 * as ssm_scan.h and ssm_recurrent.h:
 *
 *   ssm_delta_rule_fwd / _fwd_varlen / _bwd / _bwd_varlen, ssm_delta_state_update
 *       the gated delta rule: a float32 matrix state per head, from which every
 *       token erases what its key reads before it writes its value there
 *   ssm_layer_norm_fwd / _bwd
 *       the norm in front of a layer, with the residual sum in the same pass
 *
 * A layer calls ssm_layer_norm_fwd, its projections, ssm_causal_conv1d_fwd,
 * ssm_qk_norm_rotate_fwd (rotary_dim 0 and weights 1/sqrt(headdim) give keys of
 * unit norm) and ssm_delta_rule_fwd.
 *
 * The conventions are those of ssm_scan.h: device pointers on the current HIP
 * device, row-major tensors (contiguous where no stride is given), "act"
 * tensors of the element type `dtype`, everything else float32; the state and
 * every sum that a state, an output or a gradient goes through are held to
 * float32's precision, bf16 results rounded to nearest even; the caller owns every buffer, the
 * library allocates nothing and never synchronises; argument errors return a
 * negative ssm_status_t before anything is enqueued, with a message in
 * ssm_last_error().  Alignment: act tensors to their element size, float32 and
 * int32 tensors to 4 bytes, workspaces to 256 bytes.  Outputs may not overlap
 * inputs, each other or the workspace unless a function says so.  A workspace
 * holds nothing between calls, but two calls that may run at the same time
 * need one each.
 */
#ifndef SSM_LAYER_H
#define SSM_LAYER_H

#include "ssm_scan.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Tokens between the states that the forward hands to the backward. */
#define SSM_DELTA_CHUNK 64

/*
 * Gated delta rule over whole sequences.  Per sequence b and value head h, with
 * a float32 state S of headdim_k rows and headdim_v columns and the key head
 * j = h / (nheads_v / nheads_k):
 *   S   <- e^{g[b,t,h]} S
 *   u    = beta[b,t,h] (v[b,t,h,:] - S^T k[b,t,j,:])
 *   S   <- S + k[b,t,j,:] u^T
 *   out[b,t,h,:] = scale S^T q[b,t,j,:]
 *   q, k            : (batch, seqlen, nheads_k, headdim_k) act; a token's heads
 *                     together, tokens q_token_stride (k_token_stride) values
 *                     apart (at least nheads_k * headdim_k, at most 2^22: rows
 *                     of a fused projection are read where they are); batch
 *                     rows follow each other at seqlen token strides
 *   v               : (batch, seqlen, nheads_v, headdim_v) act, tokens
 *                     v_token_stride values apart, likewise
 *   beta            : (batch, seqlen, nheads_v) float32
 *   g               : (batch, seqlen, nheads_v) float32, the log of the decay,
 *                     or NULL (= 0, no decay).  g <= 0; -infinity forgets all.
 *                     (g > 0 grows the state: sums of g over a chunk of 64
 *                     tokens up to 80.)
 *   out             : (batch, seqlen, nheads_v, headdim_v) act, contiguous
 *   initial_state   : (batch, nheads_v, headdim_k, headdim_v) float32 or NULL
 *                     (= zeros)
 *   last_state      : the same shape or NULL; S after the last token.  May be
 *                     the initial_state buffer (resume in place).
 *   chunk_states    : (batch, ceil(seqlen / SSM_DELTA_CHUNK), nheads_v,
 *                     headdim_k + SSM_DELTA_CHUNK, headdim_v) float32 or NULL;
 *                     receives for every chunk of SSM_DELTA_CHUNK tokens the
 *                     state before it (headdim_k rows), then v - S^T k of its
 *                     tokens (zeros behind the last one), for
 *                     ssm_delta_rule_bwd
 *   1 <= headdim_k, headdim_v <= 256; nheads_v a multiple of nheads_k, at most
 *   65535; 1 <= batch <= 65535; seqlen >= 0 (0 only copies the initial state);
 *   batch * seqlen < 2^31; batch * ceil(seqlen / SSM_DELTA_CHUNK) * nheads_v and
 *   batch * nheads_v * ceil(headdim_v / 16) < 2^22 (SSM_ERR_SHAPE beyond).
 *   workspace       : at least ssm_delta_rule_fwd_workspace_bytes(...) bytes
 * The recurrence is stable while 0 <= beta |k|^2 <= 2; beyond, states grow as
 * the formulas say and their rounding errors with them.
 * Float32's precision is that of values above 2^-108 (3e-33); of smaller ones,
 * here and in the gradients, what lies below 2^-126 or so is lost.
 * A value that is not finite (or beyond the largest bf16 value, 3.38e38) leaves
 * its own token's outputs and those behind it in its sequence and head
 * unspecified, and the chunk_states behind its token; nothing else is touched.
 * Bitwise reproducible run to run on one device.
 */
int ssm_delta_rule_fwd(const void* q, const void* k, const void* v, const float* beta,
                       const float* g, float scale, void* out, float* last_state,
                       const float* initial_state, float* chunk_states, int64_t batch,
                       int64_t seqlen, int64_t nheads_k, int64_t nheads_v, int64_t headdim_k,
                       int64_t headdim_v, int64_t q_token_stride, int64_t k_token_stride,
                       int64_t v_token_stride, int dtype, void* workspace, size_t workspace_bytes,
                       hipStream_t stream);

/* Workspace size of the call above (0 when none is needed, or for invalid sizes). */
size_t ssm_delta_rule_fwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t nheads_k,
                                          int64_t nheads_v, int64_t headdim_k, int64_t headdim_v,
                                          int dtype);

/*
 * The same over packed variable-length sequences.
 *   q, k, v, beta, g, out : as above without the batch dimension, (total_len,
 *                      ...), the sequences one after another
 *   cu_seqlens       : (nseq + 1) int32 DEVICE array of token offsets with
 *                      0 = cu[0] <= ... <= cu[nseq] <= total_len (empty
 *                      sequences are allowed).  Rows behind cu[nseq] are
 *                      padding: their contents never reach a result, and
 *                      outputs keep what they held there.  The offsets are not
 *                      checked: ones that break the rule give unspecified
 *                      values, but every access stays inside the buffers.
 *   initial_state, last_state : (nseq, nheads_v, headdim_k, headdim_v) float32
 *                      or NULL.  last_state may be the initial_state buffer.
 *   chunk_states     : (total_len / SSM_DELTA_CHUNK + nseq, nheads_v,
 *                      headdim_k + SSM_DELTA_CHUNK, headdim_v) float32 or NULL
 *                      (the division rounds down); receives what belongs to
 *                      chunk c of sequence s at cu[s] / SSM_DELTA_CHUNK + s + c.
 *                      Places that no chunk has keep what they held.
 *   1 <= nseq < 2^20; 0 <= total_len < 2^31; (total_len / SSM_DELTA_CHUNK +
 *   nseq) * nheads_v and nseq * nheads_v * ceil(headdim_v / 16) < 2^22.
 * Nothing passes from one sequence into another, a NaN or an infinity neither.
 */
int ssm_delta_rule_fwd_varlen(const void* q, const void* k, const void* v, const float* beta,
                              const float* g, float scale, void* out, float* last_state,
                              const float* initial_state, float* chunk_states,
                              const int32_t* cu_seqlens, int64_t nseq, int64_t total_len,
                              int64_t nheads_k, int64_t nheads_v, int64_t headdim_k,
                              int64_t headdim_v, int64_t q_token_stride, int64_t k_token_stride,
                              int64_t v_token_stride, int dtype, void* workspace,
                              size_t workspace_bytes, hipStream_t stream);

size_t ssm_delta_rule_fwd_varlen_workspace_bytes(int64_t nseq, int64_t total_len, int64_t nheads_k,
                                                 int64_t nheads_v, int64_t headdim_k,
                                                 int64_t headdim_v, int dtype);

/*
 * Gradients of ssm_delta_rule_fwd for the scalar loss = sum(dout * out) +
 * sum(dlast_state * last_state), with respect to every input.
 *   inputs as ssm_delta_rule_fwd, plus
 *     chunk_states : what the forward left for the same inputs, or NULL: then
 *                    they are computed here first
 *     dout         : (batch, seqlen, nheads_v, headdim_v) act, contiguous
 *     dlast_state  : the shape of last_state, float32, or NULL (= 0)
 *   outputs (all overwritten, none accumulated into):
 *     dq, dk       : (batch, seqlen, nheads_k, headdim_k) act, contiguous; the
 *                    value heads of a key head summed before the rounding
 *     dv           : (batch, seqlen, nheads_v, headdim_v) act, contiguous
 *     dbeta        : (batch, seqlen, nheads_v) float32
 *     dg           : the same or NULL (not wanted)
 *     dinitial_state : the shape of initial_state, float32, or NULL
 * A value that is not finite leaves all gradients of its sequence and head (of
 * the key head: of dq and dk) unspecified, and no others.
 * Sums are formed in a fixed order: bitwise reproducible run to run on one
 * device.  A decay that rounds to 0 (g below about -104) has no slope: dg is 0.
 */
int ssm_delta_rule_bwd(const void* q, const void* k, const void* v, const float* beta,
                       const float* g, float scale, const float* initial_state,
                       const float* chunk_states, const void* dout, const float* dlast_state,
                       void* dq, void* dk, void* dv, float* dbeta, float* dg,
                       float* dinitial_state, int64_t batch, int64_t seqlen, int64_t nheads_k,
                       int64_t nheads_v, int64_t headdim_k, int64_t headdim_v,
                       int64_t q_token_stride, int64_t k_token_stride, int64_t v_token_stride,
                       int dtype, void* workspace, size_t workspace_bytes, hipStream_t stream);

/* with_chunk_states: 1 when the call gets chunk_states, 0 when it does not. */
size_t ssm_delta_rule_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t nheads_k,
                                          int64_t nheads_v, int64_t headdim_k, int64_t headdim_v,
                                          int dtype, int with_chunk_states);

/* Gradients of ssm_delta_rule_fwd_varlen; layouts as there, dlast_state and
 * dinitial_state (nseq, ...).  Rows of the per-token gradients behind cu[nseq]
 * keep what they held. */
int ssm_delta_rule_bwd_varlen(const void* q, const void* k, const void* v, const float* beta,
                              const float* g, float scale, const float* initial_state,
                              const float* chunk_states, const void* dout,
                              const float* dlast_state, void* dq, void* dk, void* dv, float* dbeta,
                              float* dg, float* dinitial_state, const int32_t* cu_seqlens,
                              int64_t nseq, int64_t total_len, int64_t nheads_k, int64_t nheads_v,
                              int64_t headdim_k, int64_t headdim_v, int64_t q_token_stride,
                              int64_t k_token_stride, int64_t v_token_stride, int dtype,
                              void* workspace, size_t workspace_bytes, hipStream_t stream);

size_t ssm_delta_rule_bwd_varlen_workspace_bytes(int64_t nseq, int64_t total_len, int64_t nheads_k,
                                                 int64_t nheads_v, int64_t headdim_k,
                                                 int64_t headdim_v, int dtype,
                                                 int with_chunk_states);

/*
 * One decoding step of the delta rule for `batch` sequences:
 *   state : (batch, nheads_v, headdim_k, headdim_v) float32, read and
 *           overwritten in place
 *   q, k  : (batch, nheads_k, headdim_k) act, sequences q_stride (k_stride)
 *           values apart;  v : (batch, nheads_v, headdim_v) act, v_stride apart
 *   beta  : (batch, nheads_v) float32;  g : the same or NULL
 *   out   : (batch, nheads_v, headdim_v) act, contiguous
 * Equivalent to ssm_delta_rule_fwd with seqlen = 1 and initial_state =
 * last_state = state, with sums in float32 in another order.  Here a value that
 * is not finite stays in its own head.  batch * nheads_v *
 * ceil(headdim_v / 32) < 2^24.
 */
int ssm_delta_state_update(float* state, const void* q, const void* k, const void* v,
                           const float* beta, const float* g, float scale, void* out,
                           int64_t batch, int64_t nheads_k, int64_t nheads_v, int64_t headdim_k,
                           int64_t headdim_v, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                           int dtype, hipStream_t stream);

/*
 * Layer norm over the rows of a residual stream:
 *   s = residual ? x + residual, rounded to act : x
 *   out = (s - mean(s)) / sqrt(var(s) + eps) * weight + bias,  per row, var the
 *   mean square around the mean
 *   x, residual     : (rows, dim) act, rows x_row_stride (residual_row_stride)
 *                     values apart (at least dim, at most 2^30); residual may be
 *                     NULL
 *   weight, bias    : (dim) float32 or NULL (= 1, = 0)
 *   out             : (rows, dim) act, contiguous; may be x or residual where
 *                     that is contiguous
 *   residual_out    : (rows, dim) act, contiguous, or NULL (the sum is not
 *                     wanted); receives s; needs residual.  May be x or residual
 *                     where that is contiguous.
 *   0 <= rows < 2^31; 1 <= dim <= 16384; eps >= 0 (rows whose var + eps is below
 *   2^-126 give unspecified values, and rows with values 2^57 or more apart,
 *   whose squares' sum may pass float32's range).
 * A row that holds a NaN or an infinity is NaN, and no other one.
 */
int ssm_layer_norm_fwd(const void* x, const void* residual, const float* weight, const float* bias,
                       float eps, void* out, void* residual_out, int64_t rows, int64_t dim,
                       int64_t x_row_stride, int64_t residual_row_stride, int dtype,
                       hipStream_t stream);

/*
 * Its gradients for the loss sum(dout * out) + sum(dresidual * s), from s (what
 * residual_out received, or x): mean and variance are computed again.
 *   s               : (rows, dim) act, rows s_row_stride values apart
 *   dout            : (rows, dim) act, contiguous
 *   dresidual       : (rows, dim) act, contiguous, or NULL (= 0)
 *   dx              : (rows, dim) act, contiguous: the gradient of x and of
 *                     residual alike.  May be dout or dresidual.
 *   dweight, dbias  : (dim) float32 or NULL (not wanted); summed over the rows
 *                     in a fixed order
 * workspace: at least ssm_layer_norm_bwd_workspace_bytes(...) bytes.
 */
int ssm_layer_norm_bwd(const void* s, const float* weight, float eps, const void* dout,
                       const void* dresidual, void* dx, float* dweight, float* dbias, int64_t rows,
                       int64_t dim, int64_t s_row_stride, int dtype, void* workspace,
                       size_t workspace_bytes, hipStream_t stream);

size_t ssm_layer_norm_bwd_workspace_bytes(int64_t rows, int64_t dim, int dtype);

#ifdef __cplusplus
}
#endif
#endif /* SSM_LAYER_H */
