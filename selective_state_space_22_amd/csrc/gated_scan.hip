// gated_scan.hip -- the gated linear recurrence of include/mamba_mi355x_lm.h:
// forward over sequences, backward, and the one-token step.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "gated_device.h"
#include "lm_internal.h"

namespace s6 {
namespace {

// One lane per (batch row, channel), token after token.
template <typename IO>
__global__ __launch_bounds__(64) void gated_fwd_lane_kernel(GatedArgs g) {
  const int64_t d = (int64_t)blockIdx.x * 64 + threadIdx.x;
  const int64_t bt = blockIdx.y;
  if (d >= g.D) return;
  const float kappa = g.L > 0 ? g.c * softplus(g.lam[d]) : 0.0f;
  float h = g.h0 ? g.h0[bt * g.D + d] : 0.0f;
  const int64_t nst = (g.L + kGatedStateChunk - 1) / kGatedStateChunk;
  for (int64_t t = 0; t < g.L; ++t) {
    if (g.states && t % kGatedStateChunk == 0) g.states[(bt * nst + t / kGatedStateChunk) * g.D + d] = h;
    const size_t i = (size_t)(bt * g.L + t) * g.D + d;
    float a, b;
    const bool reset = g.reset && g.reset[bt * g.L + t] != 0;
    gated_token(load_io((const IO*)g.ra, i), load_io((const IO*)g.rx, i), load_io((const IO*)g.u, i), kappa, reset, a,
                b);
    h = reset ? b : __builtin_fmaf(a, h, b);
    if (g.out) store_io((IO*)g.out, i, g.z ? h * silu(load_io((const IO*)g.z, i)) : h);
  }
  if (g.last) g.last[bt * g.D + d] = h;
}

// The reverse: each 64-token chunk is scanned forward again from its saved state
// into LDS, then backward.  pl: (batch, D) partial sums of dlam.
template <typename IO>
__global__ __launch_bounds__(64) void gated_bwd_lane_kernel(GatedBwdArgs g, float* pl) {
  __shared__ float hs[kGatedStateChunk][64];
  const GatedArgs& f = g.f;
  const int64_t d = (int64_t)blockIdx.x * 64 + threadIdx.x;
  const int64_t bt = blockIdx.y;
  if (d >= f.D) return;
  const float kappa = f.L > 0 ? f.c * softplus(f.lam[d]) : 0.0f;
  const int64_t nst = (f.L + kGatedStateChunk - 1) / kGatedStateChunk;
  float carry = g.dlast ? g.dlast[bt * f.D + d] : 0.0f;  // a_{t+1} G_{t+1}, or the gradient at the end
  float sum = 0.0f;
  for (int64_t c = nst - 1; c >= 0; --c) {
    const int64_t t0 = c * kGatedStateChunk;
    const int n = (int)(f.L - t0 < kGatedStateChunk ? f.L - t0 : kGatedStateChunk);
    float h = f.states[(bt * nst + c) * f.D + d];
    for (int k = 0; k < n; ++k) {
      const size_t i = (size_t)(bt * f.L + t0 + k) * f.D + d;
      float a, b;
      hs[k][threadIdx.x] = h;  // the state before token k
      const bool reset = f.reset && f.reset[bt * f.L + t0 + k] != 0;
      gated_token(load_io((const IO*)f.ra, i), load_io((const IO*)f.rx, i), load_io((const IO*)f.u, i), kappa, reset,
                  a, b);
      h = reset ? b : __builtin_fmaf(a, h, b);
    }
    for (int k = n - 1; k >= 0; --k) {
      const size_t i = (size_t)(bt * f.L + t0 + k) * f.D + d;
      const float u = load_io((const IO*)f.u, i);
      const bool reset = f.reset && f.reset[bt * f.L + t0 + k] != 0;
      const GatedGrad w = gated_grad(load_io((const IO*)f.ra, i), load_io((const IO*)f.rx, i), kappa, reset);
      const float hp = reset ? 0.0f : hs[k][threadIdx.x];
      const float x = w.sx * u;
      const float hk = __builtin_fmaf(w.a, hp, w.s * x);
      float dy = load_io((const IO*)g.dout, i);
      if (f.z) {
        float sz, dsz;
        silu_pair(load_io((const IO*)f.z, i), sz, dsz);
        if (g.dz) store_io((IO*)g.dz, i, dy * hk * dsz);
        dy *= sz;
      }
      const float G = dy + carry;
      const float Gs = G * w.s;
      const float e = G * __builtin_fmaf(w.a * hp, w.l, -w.q * x);
      store_io((IO*)g.du, i, Gs * w.sx);
      store_io((IO*)g.drx, i, Gs * x * w.ox);
      store_io((IO*)g.dra, i, e * w.oa);
      sum += e;
      carry = reset ? 0.0f : w.a * G;
    }
  }
  if (g.dh0) g.dh0[bt * f.D + d] = carry;
  pl[bt * f.D + d] = sum;
}

// dlam_d = (c sigma(lam) / kappa) sum of the partial sums, in order.
__global__ __launch_bounds__(64) void gated_dlam_kernel(const float* pl, const float* lam, float* dlam, int64_t n,
                                                        int64_t D) {
  const int64_t d = (int64_t)blockIdx.x * 64 + threadIdx.x;
  if (d >= D) return;
  float s = 0.0f;
  for (int64_t i = 0; i < n; ++i) s += pl[i * D + d];
  dlam[d] = n > 0 ? s * dlam_factor(lam[d]) : 0.0f;
}

template <typename IO>
__global__ __launch_bounds__(256) void gated_step_kernel(GatedStepArgs g) {
  const int64_t d = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t bt = blockIdx.y;
  if (d >= g.D) return;
  const size_t i = (size_t)bt * g.D + d;
  const bool reset = g.reset && g.reset[bt] != 0;
  float a, b;
  gated_token(load_io((const IO*)g.ra, i), load_io((const IO*)g.rx, i), load_io((const IO*)g.u, i),
              g.c * softplus(g.lam[d]), reset, a, b);
  const float h = reset ? b : __builtin_fmaf(a, g.state[i], b);
  g.state[i] = h;
  store_io((IO*)g.out, i, g.z ? h * silu(load_io((const IO*)g.z, i)) : h);
}

size_t al256(size_t v) { return (v + 255) / 256 * 256; }

size_t states_bytes(int64_t batch, int64_t L, int64_t D) {
  return al256((size_t)batch * ((L + kGatedStateChunk - 1) / kGatedStateChunk) * D * 4);
}

}  // namespace

size_t gated_fwd_ws_bytes(int64_t, int64_t, int64_t, int) { return 0; }

hipError_t launch_gated_fwd(const GatedArgs& a, int io, void*, hipStream_t st) {
  const dim3 grid((unsigned)((a.D + 63) / 64), (unsigned)a.batch);
  if (io == kIoBF16) hipLaunchKernelGGL(gated_fwd_lane_kernel<uint16_t>, grid, dim3(64), 0, st, a);
  else hipLaunchKernelGGL(gated_fwd_lane_kernel<float>, grid, dim3(64), 0, st, a);
  return hipGetLastError();
}

size_t gated_bwd_ws_bytes(int64_t batch, int64_t L, int64_t D, int) {
  if (batch == 0 || D == 0) return 0;
  return states_bytes(batch, L, D) + al256((size_t)batch * D * 4);
}

hipError_t launch_gated_bwd(const GatedBwdArgs& a, int io, void* ws, hipStream_t st) {
  GatedBwdArgs g = a;
  const GatedArgs& f = a.f;
  float* pl = nullptr;
  if (f.batch > 0) {
    float* states = static_cast<float*>(ws);
    pl = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + states_bytes(f.batch, f.L, f.D));
    if (!f.states && f.L > 0) {
      GatedArgs s = f;
      s.out = nullptr;
      s.last = nullptr;
      s.z = nullptr;
      s.states = states;
      const hipError_t e = launch_gated_fwd(s, io, nullptr, st);
      if (e != hipSuccess) return e;
      g.f.states = states;
    }
    const dim3 grid((unsigned)((f.D + 63) / 64), (unsigned)f.batch);
    if (io == kIoBF16) hipLaunchKernelGGL(gated_bwd_lane_kernel<uint16_t>, grid, dim3(64), 0, st, g, pl);
    else hipLaunchKernelGGL(gated_bwd_lane_kernel<float>, grid, dim3(64), 0, st, g, pl);
  }
  hipLaunchKernelGGL(gated_dlam_kernel, dim3((unsigned)((f.D + 63) / 64)), dim3(64), 0, st, pl, f.lam, a.dlam,
                     f.L > 0 ? f.batch : 0, f.D);
  return hipGetLastError();
}

hipError_t launch_gated_step(const GatedStepArgs& a, int io, hipStream_t st) {
  const dim3 grid((unsigned)((a.D + 255) / 256), (unsigned)a.batch);
  if (io == kIoBF16) hipLaunchKernelGGL(gated_step_kernel<uint16_t>, grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL(gated_step_kernel<float>, grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace s6
