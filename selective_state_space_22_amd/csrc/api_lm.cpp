// api_lm.cpp -- the C ABI declared in include/mamba_mi355x_lm.h.
//
// As in api.cpp, every entry point validates its arguments on the host before
// it touches the HIP runtime, then enqueues kernels on the caller's stream.
#include <cmath>

#include "../../include/mamba_mi355x_lm.h"
#include "api_check.h"
#include "lm_internal.h"

using s6::fail;
using s6::kMaxBatch;
using s6::kMaxDim;
using s6::PtrCheck;

static_assert(MAMBA_GATED_STATE_CHUNK == s6::kGatedStateChunk, "header and kernels agree");

namespace {

constexpr int64_t kMaxCount = 0x7fffffff;
constexpr int64_t kMaxSampleRows = int64_t(1) << 20;
constexpr int64_t kMaxSampleVocab = int64_t(1) << 20;

bool dtype_ok(int io) { return io == MAMBA_IO_F32 || io == MAMBA_IO_BF16; }

int check_gated(const char* where, int64_t batch, int64_t seqlen, int64_t dim, int io) {
  if (!dtype_ok(io)) return fail(MAMBA_ERR_DTYPE, where, "io_dtype");
  if (batch < 0 || seqlen < 0 || dim < 0) return fail(MAMBA_ERR_DIM, where, "negative size");
  if (batch > kMaxBatch) return fail(MAMBA_ERR_DIM, where, "batch > 65535");
  if (dim > kMaxDim) return fail(MAMBA_ERR_DIM, where, "dim > 4194304");
  if (seqlen > (int64_t(1) << 40)) return fail(MAMBA_ERR_DIM, where, "seqlen > 2^40");
  if ((double)batch * (double)seqlen * (double)dim > 1.0e18 || !s6::gated_fits(batch, seqlen, dim))
    return fail(MAMBA_ERR_DIM, where, "tensor too large");
  return MAMBA_OK;
}

int check_rate(const char* where, float c) {
  return std::isfinite(c) && c > 0.0f ? MAMBA_OK : fail(MAMBA_ERR_OPTION, where, "c");
}

int check_embed(const char* where, int64_t count, int64_t vocab, int64_t dim, int io) {
  if (!dtype_ok(io)) return fail(MAMBA_ERR_DTYPE, where, "io_dtype");
  if (count < 0 || vocab < 0 || dim < 0) return fail(MAMBA_ERR_DIM, where, "negative size");
  if (count > kMaxCount || vocab > kMaxCount) return fail(MAMBA_ERR_DIM, where, "count or vocab > 2^31 - 1");
  if (dim > kMaxDim) return fail(MAMBA_ERR_DIM, where, "dim > 4194304");
  return MAMBA_OK;
}

int check_sample(const char* where, int64_t rows, int64_t vocab, int io) {
  if (!dtype_ok(io)) return fail(MAMBA_ERR_DTYPE, where, "io_dtype");
  if (rows < 0 || rows > kMaxSampleRows) return fail(MAMBA_ERR_DIM, where, "rows");
  if (vocab < 1 || vocab > kMaxSampleVocab) return fail(MAMBA_ERR_DIM, where, "vocab");
  return MAMBA_OK;
}

s6::GatedArgs gated_args(int64_t batch, int64_t L, int64_t D, const void* u, const void* ra, const void* rx,
                         const float* lam, float c, const void* z, const uint8_t* reset, const float* h0) {
  s6::GatedArgs a{};
  a.u = u;
  a.ra = ra;
  a.rx = rx;
  a.lam = lam;
  a.z = z;
  a.reset = reset;
  a.h0 = h0;
  a.batch = batch;
  a.L = L;
  a.D = D;
  a.c = c;
  return a;
}

}  // namespace

extern "C" {

size_t mamba_gated_scan_fwd_workspace_size(int64_t batch, int64_t seqlen, int64_t dim, int io_dtype) {
  if (check_gated("mamba_gated_scan_fwd_workspace_size", batch, seqlen, dim, io_dtype) != MAMBA_OK) return 0;
  return s6::gated_fwd_ws_bytes(batch, seqlen, dim, io_dtype);
}

int mamba_gated_scan_fwd(int64_t batch, int64_t seqlen, int64_t dim, int io_dtype, const void* u, const void* gate_a,
                         const void* gate_x, const float* lam, float c, const void* z, const uint8_t* reset,
                         const float* h0, void* out, float* last_state, float* states, void* workspace,
                         size_t workspace_bytes, void* stream) {
  const char* where = "mamba_gated_scan_fwd";
  int st = check_gated(where, batch, seqlen, dim, io_dtype);
  if (st == MAMBA_OK) st = check_rate(where, c);
  if (st != MAMBA_OK) return st;
  const bool tokens = batch > 0 && seqlen > 0 && dim > 0;
  PtrCheck pc{where};
  pc.req(u, tokens, "u");
  pc.req(gate_a, tokens, "gate_a");
  pc.req(gate_x, tokens, "gate_x");
  pc.req(lam, tokens, "lam");
  pc.req(out, tokens, "out");
  pc.opt(z, "z");
  pc.opt(reset, "reset");
  pc.opt(h0, "h0");
  pc.opt(last_state, "last_state");
  pc.opt(states, "states");
  pc.opt(workspace, "workspace");
  if (pc.status != MAMBA_OK) return pc.status;
  if (batch == 0 || dim == 0) return MAMBA_OK;
  const size_t need = s6::gated_fwd_ws_bytes(batch, seqlen, dim, io_dtype);
  if (need > 0 && (!workspace || workspace_bytes < need)) return fail(MAMBA_ERR_WORKSPACE, where, "workspace");
  s6::GatedArgs a = gated_args(batch, seqlen, dim, u, gate_a, gate_x, lam, c, z, reset, h0);
  a.out = out;
  a.last = last_state;
  a.states = states;
  const hipError_t e = s6::launch_gated_fwd(a, io_dtype, workspace, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(MAMBA_ERR_HIP, where, hipGetErrorString(e));
  return MAMBA_OK;
}

size_t mamba_gated_scan_bwd_workspace_size(int64_t batch, int64_t seqlen, int64_t dim, int io_dtype) {
  if (check_gated("mamba_gated_scan_bwd_workspace_size", batch, seqlen, dim, io_dtype) != MAMBA_OK) return 0;
  return s6::gated_bwd_ws_bytes(batch, seqlen, dim, io_dtype);
}

int mamba_gated_scan_bwd(int64_t batch, int64_t seqlen, int64_t dim, int io_dtype, const void* u, const void* gate_a,
                         const void* gate_x, const float* lam, float c, const void* z, const uint8_t* reset,
                         const float* h0, const float* states, const void* dout, const float* dlast_state, void* du,
                         void* dgate_a, void* dgate_x, float* dlam, void* dz, float* dh0, void* workspace,
                         size_t workspace_bytes, void* stream) {
  const char* where = "mamba_gated_scan_bwd";
  int st = check_gated(where, batch, seqlen, dim, io_dtype);
  if (st == MAMBA_OK) st = check_rate(where, c);
  if (st != MAMBA_OK) return st;
  const bool tokens = batch > 0 && seqlen > 0 && dim > 0;
  PtrCheck pc{where};
  pc.req(u, tokens, "u");
  pc.req(gate_a, tokens, "gate_a");
  pc.req(gate_x, tokens, "gate_x");
  pc.req(lam, tokens, "lam");
  pc.req(dout, tokens, "dout");
  pc.req(du, tokens, "du");
  pc.req(dgate_a, tokens, "dgate_a");
  pc.req(dgate_x, tokens, "dgate_x");
  pc.req(dlam, dim > 0, "dlam");
  pc.opt(z, "z");
  pc.opt(reset, "reset");
  pc.opt(h0, "h0");
  pc.opt(states, "states");
  pc.opt(dlast_state, "dlast_state");
  pc.opt(dz, "dz");
  pc.opt(dh0, "dh0");
  pc.opt(workspace, "workspace");
  if (pc.status != MAMBA_OK) return pc.status;
  if (dim == 0) return MAMBA_OK;
  const size_t need = s6::gated_bwd_ws_bytes(batch, seqlen, dim, io_dtype);
  if (need > 0 && (!workspace || workspace_bytes < need)) return fail(MAMBA_ERR_WORKSPACE, where, "workspace");
  s6::GatedBwdArgs a{};
  a.f = gated_args(batch, seqlen, dim, u, gate_a, gate_x, lam, c, z, reset, h0);
  a.f.states = const_cast<float*>(states);
  a.dout = dout;
  a.dlast = dlast_state;
  a.du = du;
  a.dra = dgate_a;
  a.drx = dgate_x;
  a.dlam = dlam;
  a.dz = z ? dz : nullptr;
  a.dh0 = dh0;
  const hipError_t e = s6::launch_gated_bwd(a, io_dtype, workspace, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(MAMBA_ERR_HIP, where, hipGetErrorString(e));
  return MAMBA_OK;
}

int mamba_gated_state_update(int64_t batch, int64_t dim, int io_dtype, float* state, const void* u,
                             const void* gate_a, const void* gate_x, const float* lam, float c, const void* z,
                             const uint8_t* reset, void* out, void* stream) {
  const char* where = "mamba_gated_state_update";
  int st = check_gated(where, batch, 1, dim, io_dtype);
  if (st == MAMBA_OK) st = check_rate(where, c);
  if (st != MAMBA_OK) return st;
  const bool any = batch > 0 && dim > 0;
  PtrCheck pc{where};
  pc.req(state, any, "state");
  pc.req(u, any, "u");
  pc.req(gate_a, any, "gate_a");
  pc.req(gate_x, any, "gate_x");
  pc.req(lam, any, "lam");
  pc.req(out, any, "out");
  pc.opt(z, "z");
  pc.opt(reset, "reset");
  if (pc.status != MAMBA_OK) return pc.status;
  if (!any) return MAMBA_OK;
  const s6::GatedStepArgs a{state, u, gate_a, gate_x, lam, z, reset, out, batch, dim, c};
  const hipError_t e = s6::launch_gated_step(a, io_dtype, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(MAMBA_ERR_HIP, where, hipGetErrorString(e));
  return MAMBA_OK;
}

int mamba_embed_fwd(int64_t count, int64_t vocab, int64_t dim, int io_dtype, const int64_t* ids, const void* weight,
                    float scale, void* out, void* stream) {
  const char* where = "mamba_embed_fwd";
  const int st = check_embed(where, count, vocab, dim, io_dtype);
  if (st != MAMBA_OK) return st;
  if (!std::isfinite(scale)) return fail(MAMBA_ERR_OPTION, where, "scale");
  const bool any = count > 0 && dim > 0;
  PtrCheck pc{where};
  pc.req(ids, any, "ids");
  pc.req(weight, any && vocab > 0, "weight");
  pc.req(out, any, "out");
  if (pc.status != MAMBA_OK) return pc.status;
  if (!any) return MAMBA_OK;
  const hipError_t e = s6::launch_embed_fwd(count, vocab, dim, io_dtype, ids, weight, scale, out,
                                            static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(MAMBA_ERR_HIP, where, hipGetErrorString(e));
  return MAMBA_OK;
}

size_t mamba_embed_bwd_workspace_size(int64_t count, int64_t vocab, int64_t dim, int io_dtype) {
  if (check_embed("mamba_embed_bwd_workspace_size", count, vocab, dim, io_dtype) != MAMBA_OK) return 0;
  return s6::embed_bwd_ws_bytes(count, vocab, dim, io_dtype);
}

int mamba_embed_bwd(int64_t count, int64_t vocab, int64_t dim, int io_dtype, const int64_t* ids, const void* dout,
                    float scale, void* dweight, void* workspace, size_t workspace_bytes, void* stream) {
  const char* where = "mamba_embed_bwd";
  const int st = check_embed(where, count, vocab, dim, io_dtype);
  if (st != MAMBA_OK) return st;
  if (!std::isfinite(scale)) return fail(MAMBA_ERR_OPTION, where, "scale");
  const bool table = vocab > 0 && dim > 0;
  PtrCheck pc{where};
  pc.req(ids, table && count > 0, "ids");
  pc.req(dout, table && count > 0, "dout");
  pc.req(dweight, table, "dweight");
  pc.opt(workspace, "workspace");
  if (pc.status != MAMBA_OK) return pc.status;
  if (!table) return MAMBA_OK;
  const size_t need = s6::embed_bwd_ws_bytes(count, vocab, dim, io_dtype);
  if (need > 0 && (!workspace || workspace_bytes < need)) return fail(MAMBA_ERR_WORKSPACE, where, "workspace");
  const hipError_t e = s6::launch_embed_bwd(count, vocab, dim, io_dtype, ids, dout, scale, dweight, workspace,
                                            static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(MAMBA_ERR_HIP, where, hipGetErrorString(e));
  return MAMBA_OK;
}

int mamba_sample(int64_t rows, int64_t vocab, int io_dtype, const void* logits, const float* noise,
                 const float* temperature, const int32_t* top_k, const float* top_p, const float* min_p,
                 int64_t* tokens, float* logprob, void* stream) {
  const char* where = "mamba_sample";
  const int st = check_sample(where, rows, vocab, io_dtype);
  if (st != MAMBA_OK) return st;
  const bool any = rows > 0;
  PtrCheck pc{where};
  pc.req(logits, any, "logits");
  pc.req(noise, any, "noise");
  pc.req(tokens, any, "tokens");
  pc.opt(temperature, "temperature");
  pc.opt(top_k, "top_k");
  pc.opt(top_p, "top_p");
  pc.opt(min_p, "min_p");
  pc.opt(logprob, "logprob");
  if (pc.status != MAMBA_OK) return pc.status;
  if (!any) return MAMBA_OK;
  const s6::SampleArgs a{logits, noise, temperature, top_k, top_p, min_p, tokens, logprob, rows, vocab};
  const hipError_t e = s6::launch_sample(a, io_dtype, static_cast<hipStream_t>(stream));
  if (e != hipSuccess) return fail(MAMBA_ERR_HIP, where, hipGetErrorString(e));
  return MAMBA_OK;
}

}  // extern "C"
