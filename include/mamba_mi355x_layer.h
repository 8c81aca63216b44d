/*
 * mamba_mi355x_layer.h -- C ABI of the layer operators of libmamba_mi355x.so: what
 * stands around the scans of mamba_mi355x.h and mamba_mi355x_lm.h inside a layer, and
 * what checks the tokens that a smaller model drafted.
 *
 *   mamba_conv_fwd / _bwd / _update       the short causal convolution before a scan:
 *                                         sequences, gradients, one token
 *   mamba_conv_ssm_update                 one token through convolution, selection and
 *                                         state update
 *   mamba_residual_norm_fwd / _bwd        the norm behind a block with its gate and
 *                                         residual scale, and the norm before the next
 *   mamba_draft_verify                    drafted tokens against the target's probabilities
 *
 * The conventions are those of mamba_mi355x.h: device pointers to contiguous
 * row-major arrays, each 16-byte aligned; I/O tensors of the type io_dtype
 * (rounded to nearest even on output); fp32 arithmetic and sums; arguments
 * checked on the host before anything is enqueued; work enqueued on `stream`;
 * nothing allocated.  Every result is formed in a fixed order: repeated calls give
 * identical bits.  "Nullable" pointers may be NULL.  Outputs must not overlap
 * inputs, except where a function says that they may.
 */
#ifndef MAMBA_MI355X_LAYER_H
#define MAMBA_MI355X_LAYER_H

#include "mamba_mi355x.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Short causal convolution.  Per batch row and channel, with W = width taps:
 *     c_t = bias + sum_{j=0}^{W-1} weight_j * x_{t-(W-1)+j},   out_t = SiLU(c_t)   (silu 0: out_t = c_t)
 * where x at negative positions is the carried window: window row j is the input at
 * position j - (W-1).  A nonzero reset_t starts a new sequence at token t: no tap of t
 * or of what follows reaches an input before t.
 *   x, out       : (batch, seqlen, dim)     I/O type
 *   weight       : (dim, width)             float
 *   bias         : (dim)                    float, nullable (zero)
 *   window       : (batch, width - 1, dim)  I/O type, nullable (zero)
 *   reset        : (batch, seqlen)          bytes, nullable
 *   lengths      : (batch)                  int32, nullable: row b holds lengths[b] tokens
 *                  (below 0 counts as 0, above seqlen as seqlen); what of x lies behind
 *                  them is not read, and out is zero there
 *   last_window  : (batch, width - 1, dim)  I/O type, nullable: the last width - 1 inputs
 *                  of the row, the carried window's among them where it is shorter, zero
 *                  where a reset cut them off: the window with which the row goes on
 * Limits: 0 <= batch <= 65535, 0 <= seqlen <= 2^40, 0 <= dim <= 4194304, 2 <= width <= 4
 * (else MAMBA_ERR_UNSUPPORTED), and batch * ceil(dim / 2) * (ceil(seqlen / 32) + 1) < 2^31.
 * An output that is the very buffer of an input is refused (MAMBA_ERR_OPTION): last_window is
 * not written over window.
 * seqlen == 0 writes only last_window (= window or zero), and needs no x, weight and out.
 */
int mamba_conv_fwd(int64_t batch, int64_t seqlen, int64_t dim, int64_t width, int io_dtype, const void* x,
                   const float* weight, const float* bias, const void* window, const uint8_t* reset,
                   const int32_t* lengths, int silu, void* out, void* last_window, void* stream);

/*
 * Gradients of sum(dout * out) + sum(dlast_window * last_window) with respect to every
 * input of mamba_conv_fwd (called without lengths).
 *   x ... silu   : exactly as for the forward
 *   dout         : (batch, seqlen, dim)     I/O type
 *   dlast_window : (batch, width - 1, dim)  I/O type, nullable (zero)
 * Outputs, all overwritten:
 *   dx           : (batch, seqlen, dim)     I/O type
 *   dweight      : (dim, width)             float
 *   dbias        : (dim)                    float, nullable
 *   dwindow      : (batch, width - 1, dim)  I/O type, nullable; defined also when window is NULL
 *   workspace    : mamba_conv_bwd_workspace_size() bytes of scratch
 * Limits as for the forward.  seqlen == 0 writes dweight = dbias = 0 and dwindow = dlast_window (or 0), and
 * needs no x, weight, dout and dx.
 */
size_t mamba_conv_bwd_workspace_size(int64_t batch, int64_t seqlen, int64_t dim, int64_t width, int io_dtype);
int mamba_conv_bwd(int64_t batch, int64_t seqlen, int64_t dim, int64_t width, int io_dtype, const void* x,
                   const float* weight, const float* bias, const void* window, const uint8_t* reset, int silu,
                   const void* dout, const void* dlast_window, void* dx, float* dweight, float* dbias, void* dwindow,
                   void* workspace, size_t workspace_bytes, void* stream);

/*
 * One token of the convolution for every batch row, in place on the windows.
 *   window       : (nslots, width - 1, dim) I/O type, read and moved on by one token
 *   x, out       : (batch, dim)             I/O type; out may be x's buffer
 *   slots        : (batch) int32, nullable: row b has window slots[b] (NULL: window b, and
 *                  nslots >= batch).  A negative number, or one of nslots or more, marks an
 *                  idle row: nothing of it is read, its out and every window stay as they
 *                  were.  A window named by two rows is written by both in no order.
 *   weight, bias, silu : as for mamba_conv_fwd
 * Limits: 0 <= batch <= 65535, 0 <= dim <= 4194304, batch * ceil(dim / 2) < 2^30, 0 <= nslots < 2^31, width as there.
 */
int mamba_conv_update(int64_t batch, int64_t dim, int64_t width, int io_dtype, int64_t nslots, void* window,
                      const void* x, const float* weight, const float* bias, const int32_t* slots, int silu, void* out,
                      void* stream);

/*
 * One token of a layer from its input projection on: the convolution with SiLU, the selection
 * projections and the state update, for every batch row, in place on states and windows:
 *     xc = SiLU(conv(x)),   (r, B, C) = xc W_x^T,   dt = softplus(r W_dt^T + dt_bias),
 *     h = e^{dt A} h + (e^{dt A} - 1)/A B xc,   out = (C . h + Dskip xc) SiLU(z)
 * What mamba_conv_update, mamba_selection_fwd and mamba_state_update give one after the other, with
 * xc, r, B, C and dt in fp32 between them instead of the I/O type.
 *   state        : (nslots, dim, dstate)     float
 *   window       : (nslots, width - 1, dim)  I/O type
 *   x, z, out    : (batch, dim)              I/O type, z nullable (no gate); out may be the
 *                  buffer of x or z
 *   conv_weight, conv_bias : (dim, width), (dim) float, conv_bias nullable
 *   W_x          : (dt_rank + 2 * dstate, dim)  I/O type
 *   W_dt         : (dim, dt_rank)            I/O type
 *   dt_bias, Dskip : (dim) float, nullable;  A : (dim, dstate) float
 *   slots, nslots : as for mamba_conv_update, for state and window alike
 *   workspace    : mamba_conv_ssm_update_workspace_size() bytes of scratch
 * Limits: 0 <= batch <= 65535, 0 <= dim <= 4194304, dstate in {1, 2, 4, 8, 16}, 1 <= dt_rank <= 512,
 * 2 <= width <= 4, 0 <= nslots < 2^31, and ceil(batch / 16) * dim < 2^28.
 */
size_t mamba_conv_ssm_update_workspace_size(int64_t batch, int64_t dim, int64_t dstate, int64_t dt_rank, int io_dtype);
int mamba_conv_ssm_update(int64_t batch, int64_t dim, int64_t dstate, int64_t dt_rank, int64_t width, int io_dtype,
                          int64_t nslots, float* state, void* window, const void* x, const float* conv_weight,
                          const float* conv_bias, const void* W_x, const void* W_dt, const float* dt_bias,
                          const float* A, const float* Dskip, const void* z, const int32_t* slots, void* out,
                          void* workspace, size_t workspace_bytes, void* stream);

/*
 * The norm behind a block with its gate, the residual sum, and the norm before the next block.
 * Per row, with rms(v) = sqrt(mean(v^2) + eps):
 *     gate_first != 0:  p = post_weight * v / rms(v), v = x * SiLU(gate)
 *     gate_first == 0:  p = post_weight * x / rms(x) * SiLU(gate)
 *     residual_out = residual + alpha * scale * p
 *     out = pre_weight * r / rms(r), r = residual_out before it is rounded
 *   x, gate, out : (rows, dim) I/O type, gate nullable (no gate)
 *   residual, residual_out : (rows, dim) of the type res_dtype: io_dtype or MAMBA_IO_F32, both
 *                  nullable (residual: zero; residual_out: not written)
 *   post_weight  : (dim) float, nullable: no norm behind the block (p = x [SiLU(gate)])
 *   scale        : (dim) float, nullable (1)
 *   pre_weight   : (dim) float, nullable: no norm behind the sum; out is then not written
 *                  and may be NULL
 *   alpha        : finite host value;  eps : finite and > 0   (else MAMBA_ERR_OPTION)
 * An output may be the very buffer of an input of its shape and type.
 * Limits: 0 <= rows < 2^31, 1 <= dim <= 16384 (0 allowed when rows is 0), and rows times 64 (up to 768
 * elements), 192 (up to 1536), 512 (up to 4096) or 1024 (beyond) below 2^31.  Squares are summed in
 * fp32: a row whose squares sum past 3.4e38 normalises to zero.
 */
int mamba_residual_norm_fwd(int64_t rows, int64_t dim, int io_dtype, int res_dtype, const void* x, const void* gate,
                            int gate_first, const float* post_weight, const float* scale, const void* residual,
                            const float* pre_weight, float alpha, float eps, void* residual_out, void* out,
                            void* stream);

/*
 * Gradients of sum(dout * out) + sum(dresidual_out * residual_out) with respect to every input of
 * mamba_residual_norm_fwd, which are all that is needed of it.
 *   x ... eps    : exactly as for the forward
 *   dout         : (rows, dim) I/O type; given exactly where pre_weight is
 *   dresidual_out: (rows, dim) of the type res_dtype, nullable (zero)
 * Outputs, all overwritten:
 *   dx           : (rows, dim) I/O type
 *   dgate        : (rows, dim) I/O type, nullable; written when gate is given
 *   dresidual    : (rows, dim) of the type res_dtype, nullable; defined also when residual is NULL
 *   dpost_weight, dscale, dpre_weight : (dim) float, nullable; written when post_weight, scale,
 *                  pre_weight are given
 *   workspace    : mamba_residual_norm_bwd_workspace_size() bytes of scratch
 * dx, dgate and dresidual may be the very buffers of inputs of their shape and type.
 */
size_t mamba_residual_norm_bwd_workspace_size(int64_t rows, int64_t dim, int io_dtype);
int mamba_residual_norm_bwd(int64_t rows, int64_t dim, int io_dtype, int res_dtype, const void* x, const void* gate,
                            int gate_first, const float* post_weight, const float* scale, const void* residual,
                            const float* pre_weight, float alpha, float eps, const void* dout,
                            const void* dresidual_out, void* dx, void* dgate, void* dresidual, float* dpost_weight,
                            float* dscale, float* dpre_weight, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Verification of drafted tokens.  Per row, with n = counts[row] drafts d_k of probability q_k and
 * the target's probabilities p_k (p_k: after the first k drafts), draft k is kept where
 *     uniform_k * q_k(d_k) < p_k(d_k)      (one fp32 product)
 * and all before it are kept.  With a kept, one token more is drawn, the argmax of w_i / noise_i
 * over the i with w_i > 0, the lowest index of equal ones, where
 *     w = max(p_a - q_a, 0) if draft a was refused, or p_a if that is zero everywhere;
 *     w = p_a if all n were kept.
 * With uniforms from [0, 1) and Exp(1) noise, independent, the tokens are distributed as if drawn
 * from the target one by one.  A draft that is no token of the vocabulary is refused, and so is
 * one whose p or q is NaN; an i where w comes out NaN is not drawn.  A noise value of 0 always
 * wins; a negative or NaN one loses against every other.
 *   target    : (rows, drafts + 1, vocab) I/O type;  draft : (rows, drafts, vocab) I/O type
 *   drafted   : (rows, drafts) int64;  uniform : (rows, drafts) float;  noise : (rows, vocab) float
 *   counts    : (rows) int32, nullable (drafts; below 0 counts as 0, above drafts as drafts)
 *   tokens    : (rows, drafts + 1) int64: the kept drafts, the drawn token, then -1; the drawn
 *               token is -1 where no p_a is above 0
 *   accepted  : (rows) int32: the number of kept drafts
 *   workspace : mamba_draft_verify_workspace_size() bytes of scratch (may be NULL when that is 0)
 * Limits: 0 <= rows <= 2^20, 0 <= drafts <= 4096, 1 <= vocab <= 2^20.
 */
size_t mamba_draft_verify_workspace_size(int64_t rows, int64_t drafts, int64_t vocab, int io_dtype);
int mamba_draft_verify(int64_t rows, int64_t drafts, int64_t vocab, int io_dtype, const void* target,
                       const void* draft, const int64_t* drafted, const float* uniform, const float* noise,
                       const int32_t* counts, int64_t* tokens, int32_t* accepted, void* workspace,
                       size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MAMBA_MI355X_LAYER_H */
