/*
 * mamba_mi355x_lm.h -- C ABI of the token-model operators of libmamba_mi355x.so:
 * what a model of tokens needs around the scan of mamba_mi355x.h.
 *
 *   mamba_embed_fwd / _bwd          token ids -> scaled rows of a table, and the table's gradient
 *   mamba_gated_scan_fwd / _bwd     a gated linear recurrence over whole sequences, and its gradients
 *   mamba_gated_state_update        one token of that recurrence
 *   mamba_sample                    logits -> the next token
 *
 * The conventions are those of mamba_mi355x.h: device pointers to contiguous
 * row-major arrays, each 16-byte aligned; I/O tensors of the type io_dtype
 * (rounded to nearest even on output); fp32 arithmetic, states and sums;
 * arguments checked on the host before anything is enqueued; work enqueued on
 * `stream`; nothing allocated.  Every result is formed in a fixed order:
 * repeated calls give identical bits.  "Nullable" pointers may be NULL.
 */
#ifndef MAMBA_MI355X_LM_H
#define MAMBA_MI355X_LM_H

#include "mamba_mi355x.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Tokens between two states that mamba_gated_scan_fwd saves for the backward. */
#define MAMBA_GATED_STATE_CHUNK 8

/*
 * Gated linear recurrence.  Per batch row and channel d, with sigma the logistic
 * function and kappa_d = c * softplus(lam_d):
 *     l_t = -kappa_d * sigma(gate_a_t),   a_t = e^{l_t},   s_t = sqrt(1 - a_t^2)
 *     h_t = a_t * h_{t-1} + s_t * sigma(gate_x_t) * u_t
 *     out_t = h_t * SiLU(z_t)             (z NULL: out_t = h_t)
 * A nonzero reset_t starts a new sequence at token t: a_t = 0 and s_t = 1 there,
 * and l_t does not enter.
 *   u, gate_a, gate_x, z, out : (batch, seqlen, dim)  I/O type, z nullable
 *   lam                       : (dim)                 float
 *   c                         : decay rate, finite and > 0 (host value)
 *   reset                     : (batch, seqlen)       bytes, nullable
 *   h0, last_state            : (batch, dim)          float, nullable
 *   states                    : (batch, ceil(seqlen / 8), dim) float, nullable:
 *                               the state entering every 8th token (the first is
 *                               h0 or zero), for mamba_gated_scan_bwd
 *   workspace                 : mamba_gated_scan_fwd_workspace_size() bytes of
 *                               scratch (may be NULL when that is 0)
 * Limits: 0 <= batch <= 65535, 0 <= seqlen <= 2^40, 0 <= dim <= 4194304, and
 * batch * ceil(dim / 64) * ceil(seqlen / 56) < 2^31; a c out of range is
 * MAMBA_ERR_OPTION.  seqlen == 0 writes only last_state (= h0 or zero).
 * Where a sequence is split over workgroups they hand their states over in
 * bounded waits as mamba_scan_fwd's chunks do: mamba_stream_status reports one
 * that gave up, and what follows it is NaN.
 */
size_t mamba_gated_scan_fwd_workspace_size(int64_t batch, int64_t seqlen, int64_t dim, int io_dtype);
int mamba_gated_scan_fwd(int64_t batch, int64_t seqlen, int64_t dim, int io_dtype, const void* u, const void* gate_a,
                         const void* gate_x, const float* lam, float c, const void* z, const uint8_t* reset,
                         const float* h0, void* out, float* last_state, float* states, void* workspace,
                         size_t workspace_bytes, void* stream);

/*
 * Gradients of sum(dout * out) + sum(dlast_state * last_state) with respect to
 * every input of mamba_gated_scan_fwd.
 *   u ... h0        : exactly as for the forward
 *   states          : what the forward saved from the same inputs; NULL: computed
 *                     again here (one more pass over u, gate_a, gate_x)
 *   dout            : (batch, seqlen, dim) I/O type
 *   dlast_state     : (batch, dim) float, nullable (zero)
 * Outputs, all overwritten:
 *   du, dgate_a, dgate_x : (batch, seqlen, dim) I/O type
 *   dz              : (batch, seqlen, dim) I/O type, nullable; written when z is given
 *   dlam            : (dim) float
 *   dh0             : (batch, dim) float, nullable; defined also when h0 is NULL
 * Where 1 - a_t^2 is 0 in fp32 (kappa or the gate underflows), the gradient's
 * l_t / s_t is taken as its limit 0.  seqlen == 0 writes dlam = 0 and dh0 =
 * dlast_state (or 0).
 */
size_t mamba_gated_scan_bwd_workspace_size(int64_t batch, int64_t seqlen, int64_t dim, int io_dtype);
int mamba_gated_scan_bwd(int64_t batch, int64_t seqlen, int64_t dim, int io_dtype, const void* u, const void* gate_a,
                         const void* gate_x, const float* lam, float c, const void* z, const uint8_t* reset,
                         const float* h0, const float* states, const void* dout, const float* dlast_state, void* du,
                         void* dgate_a, void* dgate_x, float* dlam, void* dz, float* dh0, void* workspace,
                         size_t workspace_bytes, void* stream);

/*
 * One token of the recurrence for every (batch row, channel), in place on state.
 *   state                     : (batch, dim) float, read and overwritten
 *   u, gate_a, gate_x, z, out : (batch, dim) I/O type, z nullable
 *   lam, c                    : as for mamba_gated_scan_fwd
 *   reset                     : (batch) bytes, nullable
 */
int mamba_gated_state_update(int64_t batch, int64_t dim, int io_dtype, float* state, const void* u,
                             const void* gate_a, const void* gate_x, const float* lam, float c, const void* z,
                             const uint8_t* reset, void* out, void* stream);

/*
 * Embedding lookup: out_i = scale * weight[ids_i].
 *   ids    : (count) int64.  A negative id is padding: its row is zero.  An id of
 *            vocab or more reads nothing: its row is NaN.
 *   weight : (vocab, dim) I/O type;  out : (count, dim) I/O type
 *   scale  : finite host value (else MAMBA_ERR_OPTION)
 * Limits: 0 <= count <= 2^31 - 1, 0 <= vocab <= 2^31 - 1, 0 <= dim <= 4194304.
 */
int mamba_embed_fwd(int64_t count, int64_t vocab, int64_t dim, int io_dtype, const int64_t* ids, const void* weight,
                    float scale, void* out, void* stream);

/*
 * The table's gradient: dweight_v = scale * sum of dout_i over the i with ids_i == v,
 * added in the order of i in fp32 within fixed spans of the id-sorted rows, and
 * rounded once; rows that no id names are zero.  Ids outside [0, vocab) add nothing.
 *   dout : (count, dim) I/O type;  dweight : (vocab, dim) I/O type, overwritten
 *   workspace : mamba_embed_bwd_workspace_size() bytes of scratch
 */
size_t mamba_embed_bwd_workspace_size(int64_t count, int64_t vocab, int64_t dim, int io_dtype);
int mamba_embed_bwd(int64_t count, int64_t vocab, int64_t dim, int io_dtype, const int64_t* ids, const void* dout,
                    float scale, void* dweight, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Draws one token per row of logits.  Per row, with x the logits (a NaN counts as
 * -inf: masked), m their largest and w_i = e^{(x_i - m) / temperature} (1 where
 * x_i = m, also where m is infinite):
 *   top_k  the k largest logits stay (equal ones: lower index first)
 *   top_p  of these, in falling order (equal ones: lower index first), those stay
 *          whose predecessors' w sum to less than top_p of the sum of all that top_k left
 *   min_p  of these, those stay with w_i >= min_p
 *   token  = argmax of w_i / noise_i over what stays with w_i > 0, the lowest index of equal ones
 *   logprob = ln(w_token / sum of w over what stays)
 * With independent Exp(1) noise the token has the distribution w / sum(w) over
 * what stays.  The noise of what does not stay may hold anything.  A noise value of 0 always
 * wins; a negative or NaN one never does, unless none else stays.
 *   logits  : (rows, vocab) I/O type;  noise : (rows, vocab) float
 *   temperature, top_p, min_p : (rows) float, top_k : (rows) int32, all nullable.
 *     temperature NULL: 1; <= 0 or NaN: greedy (k = 1).  top_k NULL or <= 0: off.
 *     top_p NULL, >= 1 or NaN: off; <= 0 keeps the largest only.  min_p NULL,
 *     <= 0 or NaN: off; >= 1 keeps what equals the largest.
 *   tokens  : (rows) int64; -1 for a row whose logits are all -inf or NaN
 *   logprob : (rows) float, nullable; -inf for such a row
 * Limits: 0 <= rows <= 2^20, 1 <= vocab <= 2^20.
 */
int mamba_sample(int64_t rows, int64_t vocab, int io_dtype, const void* logits, const float* noise,
                 const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                 int64_t* tokens, float* logprob, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MAMBA_MI355X_LM_H */
