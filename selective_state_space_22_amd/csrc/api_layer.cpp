// api_layer.cpp -- the C ABI declared in include/mamba_mi355x_layer.h.
//
// As in api.cpp, every entry point validates its arguments on the host before
// it touches the HIP runtime, then enqueues kernels on the caller's stream.
#include <cmath>

#include "../../include/mamba_mi355x_layer.h"
#include "api_check.h"
#include "layer_internal.h"

using s6::fail;
using s6::kMaxBatch;
using s6::kMaxDim;
using s6::PtrCheck;

namespace {

constexpr int64_t kMaxSlots = 0x7fffffff;
constexpr int64_t kMaxRank = 512;
constexpr int64_t kMaxVerify = int64_t(1) << 20;
constexpr int64_t kMaxDrafts = 4096;

bool dtype_ok(int io) { return io == MAMBA_IO_F32 || io == MAMBA_IO_BF16; }

int check_conv(const char* where, int64_t batch, int64_t seqlen, int64_t dim, int64_t width, int io) {
  if (!dtype_ok(io)) return fail(MAMBA_ERR_DTYPE, where, "io_dtype");
  if (batch < 0 || seqlen < 0 || dim < 0) return fail(MAMBA_ERR_DIM, where, "negative size");
  if (batch > kMaxBatch) return fail(MAMBA_ERR_DIM, where, "batch > 65535");
  if (dim > kMaxDim) return fail(MAMBA_ERR_DIM, where, "dim > 4194304");
  if (seqlen > (int64_t(1) << 40)) return fail(MAMBA_ERR_DIM, where, "seqlen > 2^40");
  if (width < 2 || width > 4) return fail(MAMBA_ERR_UNSUPPORTED, where, "width");
  if (!s6::conv_fits(batch, seqlen, dim)) return fail(MAMBA_ERR_DIM, where, "tensor too large");
  return MAMBA_OK;
}

int check_slots(const char* where, int64_t batch, int64_t nslots, const int32_t* slots) {
  if (nslots < 0 || nslots > kMaxSlots) return fail(MAMBA_ERR_DIM, where, "nslots");
  if (!slots && nslots < batch) return fail(MAMBA_ERR_DIM, where, "nslots < batch without slots");
  return MAMBA_OK;
}

// An output that is an input's buffer would be read by one thread behind another's write.
template <int M, int N>
bool is_one_of(const void* const (&outs)[M], const void* const (&ins)[N]) {
  for (const void* o : outs)
    for (const void* i : ins)
      if (o && o == i) return true;
  return false;
}

int check_ssm(const char* where, int64_t batch, int64_t dim, int64_t dstate, int64_t dt_rank, int io) {
  if (!dtype_ok(io)) return fail(MAMBA_ERR_DTYPE, where, "io_dtype");
  if (batch < 0 || dim < 0) return fail(MAMBA_ERR_DIM, where, "negative size");
  if (batch > kMaxBatch) return fail(MAMBA_ERR_DIM, where, "batch > 65535");
  if (dim > kMaxDim) return fail(MAMBA_ERR_DIM, where, "dim > 4194304");
  if (!s6::dstate_supported(dstate)) return fail(MAMBA_ERR_UNSUPPORTED, where, "dstate");
  if (dt_rank < 1 || dt_rank > kMaxRank) return fail(MAMBA_ERR_DIM, where, "dt_rank");
  if ((batch + 15) / 16 * dim >= (int64_t(1) << 28)) return fail(MAMBA_ERR_DIM, where, "tensor too large");
  return MAMBA_OK;
}

int check_norm(const char* where, int64_t rows, int64_t dim, int io) {
  if (!dtype_ok(io)) return fail(MAMBA_ERR_DTYPE, where, "io_dtype");
  if (rows < 0 || dim < 0 || (dim == 0 && rows > 0)) return fail(MAMBA_ERR_DIM, where, "size");
  if (dim > s6::kMaxNormDim) return fail(MAMBA_ERR_DIM, where, "dim > 16384");
  if (rows > 0x7fffffff || !s6::norm_fits(rows, dim)) return fail(MAMBA_ERR_DIM, where, "rows");
  return MAMBA_OK;
}

int check_norm_call(const char* where, int64_t rows, int64_t dim, int io, int res, float alpha, float eps) {
  const int st = check_norm(where, rows, dim, io);
  if (st != MAMBA_OK) return st;
  if (res != MAMBA_IO_F32 && res != io) return fail(MAMBA_ERR_DTYPE, where, "res_dtype");
  if (!std::isfinite(alpha)) return fail(MAMBA_ERR_OPTION, where, "alpha");
  if (!std::isfinite(eps) || !(eps > 0.0f)) return fail(MAMBA_ERR_OPTION, where, "eps");
  return MAMBA_OK;
}

int check_verify(const char* where, int64_t rows, int64_t drafts, int64_t vocab, int io) {
  if (!dtype_ok(io)) return fail(MAMBA_ERR_DTYPE, where, "io_dtype");
  if (rows < 0 || rows > kMaxVerify) return fail(MAMBA_ERR_DIM, where, "rows");
  if (drafts < 0 || drafts > kMaxDrafts) return fail(MAMBA_ERR_DIM, where, "drafts");
  if (vocab < 1 || vocab > kMaxVerify) return fail(MAMBA_ERR_DIM, where, "vocab");
  return MAMBA_OK;
}

s6::NormArgs norm_args(int64_t rows, int64_t dim, const void* x, const void* gate, int gate_first, const float* post,
                       const float* scale, const void* residual, const float* pre, float alpha, float eps) {
  s6::NormArgs a{};
  a.x = x;
  a.gate = gate;
  a.post = post;
  a.scale = scale;
  a.residual = residual;
  a.pre = pre;
  a.rows = rows;
  a.D = dim;
  a.alpha = alpha;
  a.eps = eps;
  a.gate_first = gate_first != 0;
  return a;
}

}  // namespace

extern "C" {

int mamba_conv_fwd(int64_t batch, int64_t seqlen, int64_t dim, int64_t width, int io_dtype, const void* x,
                   const float* weight, const float* bias, const void* window, const uint8_t* reset,
                   const int32_t* lengths, int silu, void* out, void* last_window, void* stream) {
  const char* where = "mamba_conv_fwd";
  const int st = check_conv(where, batch, seqlen, dim, width, io_dtype);
  if (st != MAMBA_OK) return st;
  const bool tokens = batch > 0 && seqlen > 0 && dim > 0;
  PtrCheck pc{where};
  pc.req(x, tokens, "x");
  pc.req(weight, tokens, "weight");
  pc.req(out, tokens, "out");
  pc.opt(bias, "bias");
  pc.opt(window, "window");
  pc.opt(reset, "reset");
  pc.opt(lengths, "lengths");
  pc.opt(last_window, "last_window");
  if (pc.status != MAMBA_OK) return pc.status;
  if (batch == 0 || dim == 0 || (seqlen == 0 && !last_window)) return MAMBA_OK;
  if (is_one_of({out, last_window}, {x, window})) return fail(MAMBA_ERR_OPTION, where, "an output is an input's buffer");
  const s6::ConvArgs a{x, weight, bias, window, reset, lengths, out, last_window, batch, seqlen, dim, (int32_t)width,
                       silu != 0};
  const hipError_t e = s6::launch_conv_fwd(a, io_dtype, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(MAMBA_ERR_HIP, where, hipGetErrorString(e));
  return MAMBA_OK;
}

size_t mamba_conv_bwd_workspace_size(int64_t batch, int64_t seqlen, int64_t dim, int64_t width, int io_dtype) {
  if (check_conv("mamba_conv_bwd_workspace_size", batch, seqlen, dim, width, io_dtype) != MAMBA_OK) return 0;
  return s6::conv_bwd_ws_bytes(batch, seqlen, dim, width);
}

int mamba_conv_bwd(int64_t batch, int64_t seqlen, int64_t dim, int64_t width, int io_dtype, const void* x,
                   const float* weight, const float* bias, const void* window, const uint8_t* reset, int silu,
                   const void* dout, const void* dlast_window, void* dx, float* dweight, float* dbias, void* dwindow,
                   void* workspace, size_t workspace_bytes, void* stream) {
  const char* where = "mamba_conv_bwd";
  const int st = check_conv(where, batch, seqlen, dim, width, io_dtype);
  if (st != MAMBA_OK) return st;
  const bool tokens = batch > 0 && seqlen > 0 && dim > 0;
  PtrCheck pc{where};
  pc.req(x, tokens, "x");
  pc.req(weight, tokens, "weight");
  pc.req(dout, tokens, "dout");
  pc.req(dx, tokens, "dx");
  pc.req(dweight, dim > 0, "dweight");
  pc.opt(bias, "bias");
  pc.opt(window, "window");
  pc.opt(reset, "reset");
  pc.opt(dlast_window, "dlast_window");
  pc.opt(dbias, "dbias");
  pc.opt(dwindow, "dwindow");
  pc.opt(workspace, "workspace");
  if (pc.status != MAMBA_OK) return pc.status;
  if (dim == 0) return MAMBA_OK;
  const size_t need = s6::conv_bwd_ws_bytes(batch, seqlen, dim, width);
  if (need > 0 && (!workspace || workspace_bytes < need)) return fail(MAMBA_ERR_WORKSPACE, where, "workspace");
  if (is_one_of({dx, dwindow}, {x, window, dout, dlast_window}))
    return fail(MAMBA_ERR_OPTION, where, "an output is an input's buffer");
  s6::ConvBwdArgs a{};
  a.f = s6::ConvArgs{x, weight, bias, window, reset, nullptr, nullptr, nullptr, batch, seqlen, dim, (int32_t)width,
                     silu != 0};
  a.dout = dout;
  a.dlast = dlast_window;
  a.dx = dx;
  a.dweight = dweight;
  a.dbias = dbias;
  a.dwindow = dwindow;
  const hipError_t e = s6::launch_conv_bwd(a, io_dtype, workspace, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(MAMBA_ERR_HIP, where, hipGetErrorString(e));
  return MAMBA_OK;
}

int mamba_conv_update(int64_t batch, int64_t dim, int64_t width, int io_dtype, int64_t nslots, void* window,
                      const void* x, const float* weight, const float* bias, const int32_t* slots, int silu, void* out,
                      void* stream) {
  const char* where = "mamba_conv_update";
  int st = check_conv(where, batch, 1, dim, width, io_dtype);
  if (st == MAMBA_OK) st = check_slots(where, batch, nslots, slots);
  if (st != MAMBA_OK) return st;
  const bool any = batch > 0 && dim > 0;
  PtrCheck pc{where};
  pc.req(window, any && nslots > 0, "window");
  pc.req(x, any, "x");
  pc.req(weight, any, "weight");
  pc.req(out, any, "out");
  pc.opt(bias, "bias");
  pc.opt(slots, "slots");
  if (pc.status != MAMBA_OK) return pc.status;
  if (!any) return MAMBA_OK;
  const s6::ConvStepArgs a{window, x, weight, bias, slots, out, batch, dim, nslots, (int32_t)width, silu != 0};
  const hipError_t e = s6::launch_conv_step(a, io_dtype, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(MAMBA_ERR_HIP, where, hipGetErrorString(e));
  return MAMBA_OK;
}

size_t mamba_conv_ssm_update_workspace_size(int64_t batch, int64_t dim, int64_t dstate, int64_t dt_rank, int io_dtype) {
  if (check_ssm("mamba_conv_ssm_update_workspace_size", batch, dim, dstate, dt_rank, io_dtype) != MAMBA_OK) return 0;
  return s6::ssm_step_ws_bytes(batch, dim, dstate, dt_rank);
}

int mamba_conv_ssm_update(int64_t batch, int64_t dim, int64_t dstate, int64_t dt_rank, int64_t width, int io_dtype,
                          int64_t nslots, float* state, void* window, const void* x, const float* conv_weight,
                          const float* conv_bias, const void* W_x, const void* W_dt, const float* dt_bias,
                          const float* A, const float* Dskip, const void* z, const int32_t* slots, void* out,
                          void* workspace, size_t workspace_bytes, void* stream) {
  const char* where = "mamba_conv_ssm_update";
  int st = check_ssm(where, batch, dim, dstate, dt_rank, io_dtype);
  if (st != MAMBA_OK) return st;
  if (width < 2 || width > 4) return fail(MAMBA_ERR_UNSUPPORTED, where, "width");
  st = check_slots(where, batch, nslots, slots);
  if (st != MAMBA_OK) return st;
  const bool any = batch > 0 && dim > 0;
  PtrCheck pc{where};
  pc.req(state, any && nslots > 0, "state");
  pc.req(window, any && nslots > 0, "window");
  pc.req(x, any, "x");
  pc.req(conv_weight, any, "conv_weight");
  pc.req(W_x, any, "W_x");
  pc.req(W_dt, any, "W_dt");
  pc.req(A, any, "A");
  pc.req(out, any, "out");
  pc.opt(conv_bias, "conv_bias");
  pc.opt(dt_bias, "dt_bias");
  pc.opt(Dskip, "Dskip");
  pc.opt(z, "z");
  pc.opt(slots, "slots");
  pc.opt(workspace, "workspace");
  if (pc.status != MAMBA_OK) return pc.status;
  if (!any) return MAMBA_OK;
  const size_t need = s6::ssm_step_ws_bytes(batch, dim, dstate, dt_rank);
  if (!workspace || workspace_bytes < need) return fail(MAMBA_ERR_WORKSPACE, where, "workspace");
  const s6::SsmStepArgs a{state, window, x,     conv_weight, conv_bias, W_x, W_dt,   dt_bias, A,
                          Dskip, z,      slots, out,         batch,     dim, dstate, dt_rank, nslots,
                          (int32_t)width};
  const hipError_t e = s6::launch_ssm_step(a, io_dtype, workspace, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(MAMBA_ERR_HIP, where, hipGetErrorString(e));
  return MAMBA_OK;
}

int mamba_residual_norm_fwd(int64_t rows, int64_t dim, int io_dtype, int res_dtype, const void* x, const void* gate,
                            int gate_first, const float* post_weight, const float* scale, const void* residual,
                            const float* pre_weight, float alpha, float eps, void* residual_out, void* out,
                            void* stream) {
  const char* where = "mamba_residual_norm_fwd";
  const int st = check_norm_call(where, rows, dim, io_dtype, res_dtype, alpha, eps);
  if (st != MAMBA_OK) return st;
  const bool any = rows > 0;
  PtrCheck pc{where};
  pc.req(x, any, "x");
  pc.req(out, any && pre_weight, "out");
  pc.opt(gate, "gate");
  pc.opt(post_weight, "post_weight");
  pc.opt(scale, "scale");
  pc.opt(residual, "residual");
  pc.opt(pre_weight, "pre_weight");
  pc.opt(residual_out, "residual_out");
  if (pc.status != MAMBA_OK) return pc.status;
  if (!any || (!pre_weight && !residual_out)) return MAMBA_OK;
  s6::NormArgs a = norm_args(rows, dim, x, gate, gate_first, post_weight, scale, residual, pre_weight, alpha, eps);
  a.residual_out = residual_out;
  a.out = out;
  const hipError_t e = s6::launch_norm_fwd(a, io_dtype, res_dtype, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(MAMBA_ERR_HIP, where, hipGetErrorString(e));
  return MAMBA_OK;
}

size_t mamba_residual_norm_bwd_workspace_size(int64_t rows, int64_t dim, int io_dtype) {
  if (check_norm("mamba_residual_norm_bwd_workspace_size", rows, dim, io_dtype) != MAMBA_OK) return 0;
  return s6::norm_bwd_ws_bytes(rows, dim);
}

int mamba_residual_norm_bwd(int64_t rows, int64_t dim, int io_dtype, int res_dtype, const void* x, const void* gate,
                            int gate_first, const float* post_weight, const float* scale, const void* residual,
                            const float* pre_weight, float alpha, float eps, const void* dout,
                            const void* dresidual_out, void* dx, void* dgate, void* dresidual, float* dpost_weight,
                            float* dscale, float* dpre_weight, void* workspace, size_t workspace_bytes, void* stream) {
  const char* where = "mamba_residual_norm_bwd";
  const int st = check_norm_call(where, rows, dim, io_dtype, res_dtype, alpha, eps);
  if (st != MAMBA_OK) return st;
  const bool any = rows > 0;
  PtrCheck pc{where};
  pc.req(x, any, "x");
  pc.req(dout, any && pre_weight, "dout");
  pc.req(dx, any, "dx");
  pc.opt(gate, "gate");
  pc.opt(post_weight, "post_weight");
  pc.opt(scale, "scale");
  pc.opt(residual, "residual");
  pc.opt(pre_weight, "pre_weight");
  pc.opt(dresidual_out, "dresidual_out");
  pc.opt(dgate, "dgate");
  pc.opt(dresidual, "dresidual");
  pc.opt(dpost_weight, "dpost_weight");
  pc.opt(dscale, "dscale");
  pc.opt(dpre_weight, "dpre_weight");
  pc.opt(workspace, "workspace");
  if (pc.status != MAMBA_OK) return pc.status;
  if (dim == 0) return MAMBA_OK;
  const size_t need = s6::norm_bwd_ws_bytes(rows, dim);
  if (need > 0 && (!workspace || workspace_bytes < need)) return fail(MAMBA_ERR_WORKSPACE, where, "workspace");
  s6::NormBwdArgs b{};
  b.f = norm_args(rows, dim, x, gate, gate_first, post_weight, scale, residual, pre_weight, alpha, eps);
  b.dout = pre_weight ? dout : nullptr;
  b.dres_out = dresidual_out;
  b.dx = dx;
  b.dgate = gate ? dgate : nullptr;
  b.dresidual = dresidual;
  b.dpost = post_weight ? dpost_weight : nullptr;
  b.dscale = scale ? dscale : nullptr;
  b.dpre = pre_weight ? dpre_weight : nullptr;
  const hipError_t e = s6::launch_norm_bwd(b, io_dtype, res_dtype, workspace, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(MAMBA_ERR_HIP, where, hipGetErrorString(e));
  return MAMBA_OK;
}

size_t mamba_draft_verify_workspace_size(int64_t rows, int64_t drafts, int64_t vocab, int io_dtype) {
  if (check_verify("mamba_draft_verify_workspace_size", rows, drafts, vocab, io_dtype) != MAMBA_OK) return 0;
  return s6::verify_ws_bytes(rows, vocab);
}

int mamba_draft_verify(int64_t rows, int64_t drafts, int64_t vocab, int io_dtype, const void* target,
                       const void* draft, const int64_t* drafted, const float* uniform, const float* noise,
                       const int32_t* counts, int64_t* tokens, int32_t* accepted, void* workspace,
                       size_t workspace_bytes, void* stream) {
  const char* where = "mamba_draft_verify";
  const int st = check_verify(where, rows, drafts, vocab, io_dtype);
  if (st != MAMBA_OK) return st;
  const bool any = rows > 0;
  PtrCheck pc{where};
  pc.req(target, any, "target");
  pc.req(draft, any && drafts > 0, "draft");
  pc.req(drafted, any && drafts > 0, "drafted");
  pc.req(uniform, any && drafts > 0, "uniform");
  pc.req(noise, any, "noise");
  pc.req(tokens, any, "tokens");
  pc.req(accepted, any, "accepted");
  pc.opt(counts, "counts");
  pc.opt(workspace, "workspace");
  if (pc.status != MAMBA_OK) return pc.status;
  if (!any) return MAMBA_OK;
  const size_t need = s6::verify_ws_bytes(rows, vocab);
  if (need > 0 && (!workspace || workspace_bytes < need)) return fail(MAMBA_ERR_WORKSPACE, where, "workspace");
  const s6::VerifyArgs a{target, draft, drafted, uniform, noise, counts, tokens, accepted, rows, drafts, vocab};
  const hipError_t e = s6::launch_verify(a, io_dtype, workspace, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(MAMBA_ERR_HIP, where, hipGetErrorString(e));
  return MAMBA_OK;
}

}  // extern "C"
