// norm.hip -- the norms behind and before a block with its gate and residual scale, forward and backward,
// on gfx950.
//
// Per row of D elements, with rms(v) = sqrt(mean(v^2) + eps) and s = SiLU(gate) (1 without a gate):
//     gate first:   v = x s,  p = post v / rms(v)          gate after:  v = x,  p = s post v / rms(v)
//     r' = residual + alpha scale p,   out = pre r' / rms(r')
// (post NULL: no norm there, p = x s).  Backward, with k = 1 / rms(v), K = 1 / rms(r'), n = v k:
//     dn' = dout pre,   dr = dr' + K (dn' - r' K^2 mean(dn' r')),   dresidual = dr,
//     dp = dr alpha scale,   e = dp post [s],   dv = k (e - n mean(e n)),
//     gate first: dx = dv s, dgate = dv x s'        after: dx = dv, dgate = dp post n s'
//     dpre = sum dout r' K,   dscale = alpha sum dr p,   dpost = sum dp [s] n.
// A few dozen operations per element: memory bounds it.  A row stays in the registers of its threads (a wave
// up to 4096 elements, a workgroup beyond that or where there are few rows), so every tensor is read once and
// written once; the backward recomputes p and r' from the inputs instead of reading saved ones.  Sums of
// squares and products are fp32.
#include <type_traits>

#include "layer_device.h"
#include "layer_internal.h"

namespace s6 {
namespace {

constexpr int E = 8;  // elements per thread and chunk

// Sum over the NT threads of a row, the same value in all of them.  Rows of more than a wave meet at
// workgroup barriers: every thread of the workgroup takes part.
template <int NT, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float (*lds)[K]) {
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) v[k] += __shfl_xor(v[k], m, 64);
  if constexpr (NT > 64) {
    __syncthreads();  // the last sum has been read
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) lds[threadIdx.x >> 6][k] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      v[k] = 0.0f;
#pragma unroll
      for (int w = 0; w < NT / 64; ++w) v[k] += lds[threadIdx.x / NT * (NT / 64) + w][k];
    }
  }
}

// EVEN: D is a multiple of E, chunks are whole or absent.
template <typename T, bool EVEN>
__device__ __forceinline__ raw_t<T, E> chunk_in(const T* row, int64_t e0, int64_t D) {
  if (e0 + E <= D) return load_raw<T, E, true>(row + e0, E);
  if (!EVEN && e0 < D) return load_raw<T, E, false>(row + e0, (int)(D - e0));
  return raw_t<T, E>(0u);
}
template <typename T, bool EVEN>
__device__ __forceinline__ void chunk_out(T* row, int64_t e0, int64_t D, const float (&f)[E]) {
  if (e0 + E <= D) store_raw<T, E, true>(row + e0, narrow<T, E>(f), E);
  else if (!EVEN && e0 < D) store_raw<T, E, false>(row + e0, narrow<T, E>(f), (int)(D - e0));
}
template <bool EVEN>
__device__ __forceinline__ void weights_in(const float* w, int64_t e0, int64_t D, float (&f)[E]) {
  widen<float, E>(chunk_in<float, EVEN>(w, e0, D), f);
}

// Rows per workgroup.
constexpr int rows_of(int nt) { return nt > 128 ? 1 : 256 / nt; }

template <typename IO, typename RES, int NT, int NV, bool EVEN>
__global__ __launch_bounds__(NT* rows_of(NT)) void norm_fwd_kernel(NormArgs a) {
  constexpr int RPB = rows_of(NT);
  __shared__ float lds[NT / 64 * RPB][1];
  const int lane = threadIdx.x % NT;
  const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / NT;
  // a row behind the last reads as one of no elements
  const int64_t D = row < a.rows ? a.D : 0, at = row * D;
  const float inv = 1.0f / (float)a.D;
  raw_t<IO, E> xr[NV], gr[NV];
  raw_t<RES, E> rr[NV];
#pragma unroll
  for (int c = 0; c < NV; ++c) xr[c] = chunk_in<IO, EVEN>(static_cast<const IO*>(a.x) + at, (c * NT + lane) * E, D);
  if (a.gate)
#pragma unroll
    for (int c = 0; c < NV; ++c)
      gr[c] = chunk_in<IO, EVEN>(static_cast<const IO*>(a.gate) + at, (c * NT + lane) * E, D);
  if (a.residual)
#pragma unroll
    for (int c = 0; c < NV; ++c)
      rr[c] = chunk_in<RES, EVEN>(static_cast<const RES*>(a.residual) + at, (c * NT + lane) * E, D);
  float v[NV][E];
  float sum[1] = {0.0f};
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    widen<IO, E>(xr[c], v[c]);
    if (a.gate && a.gate_first) {
      float g[E];
      widen<IO, E>(gr[c], g);
#pragma unroll
      for (int i = 0; i < E; ++i) v[c][i] *= silu(g[i]);
    }
#pragma unroll
    for (int i = 0; i < E; ++i) sum[0] = __builtin_fmaf(v[c][i], v[c][i], sum[0]);
  }
  float k = 1.0f;
  if (a.post) {
    row_sum<NT, 1>(sum, lds);
    k = rsqrtf(__builtin_fmaf(sum[0], inv, a.eps));
  }
  sum[0] = 0.0f;
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    const int64_t e0 = (c * NT + lane) * E;
    float w[E];
    if (a.post) {
      weights_in<EVEN>(a.post, e0, D, w);
#pragma unroll
      for (int i = 0; i < E; ++i) v[c][i] *= k * w[i];
    }
    if (a.gate && !a.gate_first) {
      float g[E];
      widen<IO, E>(gr[c], g);
#pragma unroll
      for (int i = 0; i < E; ++i) v[c][i] *= silu(g[i]);
    }
    if (a.scale) {
      weights_in<EVEN>(a.scale, e0, D, w);
#pragma unroll
      for (int i = 0; i < E; ++i) v[c][i] *= w[i];
    }
    if (a.residual) {
      widen<RES, E>(rr[c], w);
#pragma unroll
      for (int i = 0; i < E; ++i) v[c][i] = __builtin_fmaf(a.alpha, v[c][i], w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i) v[c][i] *= a.alpha;
    }
    if (a.residual_out) chunk_out<RES, EVEN>(static_cast<RES*>(a.residual_out) + at, e0, D, v[c]);
#pragma unroll
    for (int i = 0; i < E; ++i) sum[0] = __builtin_fmaf(v[c][i], v[c][i], sum[0]);
  }
  if (!a.pre) return;
  row_sum<NT, 1>(sum, lds);
  k = rsqrtf(__builtin_fmaf(sum[0], inv, a.eps));
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    const int64_t e0 = (c * NT + lane) * E;
    float w[E];
    weights_in<EVEN>(a.pre, e0, D, w);
#pragma unroll
    for (int i = 0; i < E; ++i) w[i] *= v[c][i] * k;
    chunk_out<IO, EVEN>(static_cast<IO*>(a.out) + at, e0, D, w);
  }
}

// Rows blockIdx.x, + gridDim.x, ... of RPB each; the sums over them go to part (gridDim.x, 3, D):
// dpost, dscale (without alpha), dpre.
template <typename IO, typename RES, int NT, int NV, bool EVEN>
__global__ __launch_bounds__(NT* rows_of(NT)) void norm_bwd_kernel(NormBwdArgs b, float* part) {
  constexpr int RPB = rows_of(NT);
  __shared__ float lds[NT / 64 * RPB][2];
  const NormArgs& a = b.f;
  const int lane = threadIdx.x % NT, slot = threadIdx.x / NT;
  const float inv = 1.0f / (float)a.D;
  float spost[NV][E], sscale[NV][E], spre[NV][E];
#pragma unroll
  for (int c = 0; c < NV; ++c)
#pragma unroll
    for (int i = 0; i < E; ++i) spost[c][i] = sscale[c][i] = spre[c][i] = 0.0f;
  for (int64_t first = (int64_t)blockIdx.x * RPB; first < a.rows; first += (int64_t)gridDim.x * RPB) {
    // a row behind the last reads as one of no elements: all threads pass the same barriers
    const int64_t row = first + slot, D = row < a.rows ? a.D : 0, at = row * D;
    raw_t<IO, E> xr[NV], gr[NV], dor[NV];
    raw_t<RES, E> rr[NV], drr[NV];
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int64_t e0 = (c * NT + lane) * E;
      xr[c] = chunk_in<IO, EVEN>(static_cast<const IO*>(a.x) + at, e0, D);
      if (a.gate) gr[c] = chunk_in<IO, EVEN>(static_cast<const IO*>(a.gate) + at, e0, D);
      if (a.residual) rr[c] = chunk_in<RES, EVEN>(static_cast<const RES*>(a.residual) + at, e0, D);
      if (b.dout) dor[c] = chunk_in<IO, EVEN>(static_cast<const IO*>(b.dout) + at, e0, D);
      if (b.dres_out) drr[c] = chunk_in<RES, EVEN>(static_cast<const RES*>(b.dres_out) + at, e0, D);
    }
    // n = v / rms(v)
    float n[NV][E], s1[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      widen<IO, E>(xr[c], n[c]);
      if (a.gate && a.gate_first) {
        float g[E];
        widen<IO, E>(gr[c], g);
#pragma unroll
        for (int i = 0; i < E; ++i) n[c][i] *= silu(g[i]);
      }
#pragma unroll
      for (int i = 0; i < E; ++i) s1[0] = __builtin_fmaf(n[c][i], n[c][i], s1[0]);
    }
    float k = 1.0f;
    if (a.post) {
      row_sum<NT, 1>(s1, reinterpret_cast<float(*)[1]>(lds));
      k = rsqrtf(__builtin_fmaf(s1[0], inv, a.eps));
    }
    // p, r', and the sums of the second norm
    float r[NV][E], s2[2] = {0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int64_t e0 = (c * NT + lane) * E;
      float w[E];
#pragma unroll
      for (int i = 0; i < E; ++i) {
        n[c][i] *= k;
        r[c][i] = n[c][i];
      }
      if (a.post) {
        weights_in<EVEN>(a.post, e0, D, w);
#pragma unroll
        for (int i = 0; i < E; ++i) r[c][i] *= w[i];
      }
      if (a.gate && !a.gate_first) {
        widen<IO, E>(gr[c], w);
#pragma unroll
        for (int i = 0; i < E; ++i) r[c][i] *= silu(w[i]);
      }
      if (a.scale) {
        weights_in<EVEN>(a.scale, e0, D, w);
#pragma unroll
        for (int i = 0; i < E; ++i) r[c][i] *= w[i];
      }
      if (a.residual) {
        widen<RES, E>(rr[c], w);
#pragma unroll
        for (int i = 0; i < E; ++i) r[c][i] = __builtin_fmaf(a.alpha, r[c][i], w[i]);
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i) r[c][i] *= a.alpha;
      }
      if (b.dout) {
        float d[E];
        weights_in<EVEN>(a.pre, e0, D, w);
        widen<IO, E>(dor[c], d);
#pragma unroll
        for (int i = 0; i < E; ++i) {
          s2[0] = __builtin_fmaf(r[c][i], r[c][i], s2[0]);
          s2[1] = __builtin_fmaf(d[i] * w[i], r[c][i], s2[1]);
        }
      }
    }
    float K = 0.0f, kk = 0.0f;
    if (b.dout) {
      row_sum<NT, 2>(s2, lds);
      K = rsqrtf(__builtin_fmaf(s2[0], inv, a.eps));
      kk = K * K * (s2[1] * inv);
    }
    // dr (kept in r), the sums over rows, e (kept in place of nothing that is still needed) and mean(e n)
    float e[NV][E];
    s1[0] = 0.0f;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int64_t e0 = (c * NT + lane) * E;
      float dr[E], w[E], t[E];
#pragma unroll
      for (int i = 0; i < E; ++i) dr[i] = 0.0f;
      if (b.dres_out) widen<RES, E>(drr[c], dr);
      if (b.dout) {
        widen<IO, E>(dor[c], t);
        weights_in<EVEN>(a.pre, e0, D, w);
#pragma unroll
        for (int i = 0; i < E; ++i) {
          spre[c][i] = __builtin_fmaf(t[i], r[c][i] * K, spre[c][i]);
          dr[i] = __builtin_fmaf(K, __builtin_fmaf(-kk, r[c][i], t[i] * w[i]), dr[i]);
        }
      }
      if (b.dresidual) chunk_out<RES, EVEN>(static_cast<RES*>(b.dresidual) + at, e0, D, dr);
      // s: the gate behind the norm; t: p / s / post = n
      float s[E], post[E];
#pragma unroll
      for (int i = 0; i < E; ++i) s[i] = post[i] = 1.0f;
      if (a.gate && !a.gate_first) {
        widen<IO, E>(gr[c], s);
#pragma unroll
        for (int i = 0; i < E; ++i) s[i] = silu(s[i]);
      }
      if (a.post) weights_in<EVEN>(a.post, e0, D, post);
      if (a.scale) {
        weights_in<EVEN>(a.scale, e0, D, w);
#pragma unroll
        for (int i = 0; i < E; ++i) sscale[c][i] = __builtin_fmaf(dr[i], n[c][i] * post[i] * s[i], sscale[c][i]);
      } else {
#pragma unroll
        for (int i = 0; i < E; ++i) w[i] = 1.0f;
      }
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float dp = dr[i] * (a.alpha * w[i]);
        spost[c][i] = __builtin_fmaf(dp * s[i], n[c][i], spost[c][i]);
        r[c][i] = dp * post[i];
        e[c][i] = r[c][i] * s[i];
        s1[0] = __builtin_fmaf(e[c][i], n[c][i], s1[0]);
      }
    }
    float m = 0.0f;
    if (a.post) {
      row_sum<NT, 1>(s1, reinterpret_cast<float(*)[1]>(lds));
      m = s1[0] * inv;
    }
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int64_t e0 = (c * NT + lane) * E;
      float dx[E], dg[E], x[E], g[E];
#pragma unroll
      for (int i = 0; i < E; ++i) dx[i] = k * __builtin_fmaf(-n[c][i], m, e[c][i]);
      if (a.gate) {
        widen<IO, E>(gr[c], g);
        if (a.gate_first) {
          widen<IO, E>(xr[c], x);
#pragma unroll
          for (int i = 0; i < E; ++i) {
            dg[i] = dx[i] * x[i] * silu_slope(g[i]);
            dx[i] *= silu(g[i]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < E; ++i) dg[i] = r[c][i] * n[c][i] * silu_slope(g[i]);
        }
        if (b.dgate) chunk_out<IO, EVEN>(static_cast<IO*>(b.dgate) + at, e0, D, dg);
      }
      chunk_out<IO, EVEN>(static_cast<IO*>(b.dx) + at, e0, D, dx);
    }
  }
  // the sums of the workgroup's row slots, in their order
  const int64_t D = a.D;
  float* out = part + (int64_t)blockIdx.x * 3 * D;
  if constexpr (RPB == 1) {
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int64_t e0 = (c * NT + lane) * E;
      chunk_out<float, EVEN>(out, e0, D, spost[c]);
      chunk_out<float, EVEN>(out + D, e0, D, sscale[c]);
      chunk_out<float, EVEN>(out + 2 * D, e0, D, spre[c]);
    }
  } else {
    __shared__ float acc[3][NT * NV * E];
    for (int s = 0; s < RPB; ++s) {
      __syncthreads();
      if (slot != s) continue;
#pragma unroll
      for (int c = 0; c < NV; ++c)
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const int e = (c * E + i) * NT + lane;  // lanes side by side: no bank conflicts
          acc[0][e] = s ? acc[0][e] + spost[c][i] : spost[c][i];
          acc[1][e] = s ? acc[1][e] + sscale[c][i] : sscale[c][i];
          acc[2][e] = s ? acc[2][e] + spre[c][i] : spre[c][i];
          if (s == RPB - 1) {
            spost[c][i] = acc[0][e];
            sscale[c][i] = acc[1][e];
            spre[c][i] = acc[2][e];
          }
        }
    }
    if (slot == RPB - 1)
#pragma unroll
      for (int c = 0; c < NV; ++c) {
        const int64_t e0 = (c * NT + lane) * E;
        chunk_out<float, EVEN>(out, e0, D, spost[c]);
        chunk_out<float, EVEN>(out + D, e0, D, sscale[c]);
        chunk_out<float, EVEN>(out + 2 * D, e0, D, spre[c]);
      }
  }
}

__global__ __launch_bounds__(1024) void norm_sum_kernel(const float* part, int64_t rows, int64_t D, float alpha,
                                                        float* dpost, float* dscale, float* dpre) {
  const int64_t col = (int64_t)blockIdx.x * 32 + (threadIdx.x & 31);
  const float v = column_sum(part, rows, 3 * D, col);
  if (threadIdx.x >= 32 || col >= 3 * D) return;
  if (col < D) {
    if (dpost) dpost[col] = v;
  } else if (col < 2 * D) {
    if (dscale) dscale[col - D] = alpha * v;
  } else if (dpre) {
    dpre[col - 2 * D] = v;
  }
}

template <typename IO, typename RES, int NT, int NV>
void fwd_at(const NormArgs& a, hipStream_t s) {
  constexpr int RPB = rows_of(NT);
  const dim3 grid((unsigned)((a.rows + RPB - 1) / RPB)), block(NT * RPB);
  if (a.D % E == 0) hipLaunchKernelGGL((norm_fwd_kernel<IO, RES, NT, NV, true>), grid, block, 0, s, a);
  else hipLaunchKernelGGL((norm_fwd_kernel<IO, RES, NT, NV, false>), grid, block, 0, s, a);
}

// A wave per row, or a workgroup where rows are long or too few to fill the chip with waves.
template <typename IO, typename RES>
hipError_t fwd_types(const NormArgs& a, hipStream_t s) {
  const int64_t D = a.D;
  if (D <= 512) fwd_at<IO, RES, 64, 1>(a, s);
  else if (D <= 4096 && a.rows >= 2048) {
    if (D <= 1024) fwd_at<IO, RES, 64, 2>(a, s);
    else if (D <= 1536) fwd_at<IO, RES, 64, 3>(a, s);
    else if (D <= 2560) fwd_at<IO, RES, 64, 5>(a, s);
    else fwd_at<IO, RES, 64, 8>(a, s);
  } else if (D <= 2048) fwd_at<IO, RES, 256, 1>(a, s);
  else if (D <= 4096) fwd_at<IO, RES, 256, 2>(a, s);
  else if (D <= 8192) fwd_at<IO, RES, 256, 4>(a, s);
  else fwd_at<IO, RES, 512, 4>(a, s);
  return hipGetLastError();
}

// The backward holds about 90 registers per chunk and thread, so a thread has one chunk of the row as long as
// a workgroup's threads suffice.
template <typename F>
void bwd_shape(int64_t D, F f) {
#define S6_NORM_SHAPE(nt, nv) f(std::integral_constant<int, nt>(), std::integral_constant<int, nv>())
  if (D <= 512) S6_NORM_SHAPE(64, 1);
  else if (D <= 1024) S6_NORM_SHAPE(128, 1);
  else if (D <= 1536) S6_NORM_SHAPE(192, 1);
  else if (D <= 2048) S6_NORM_SHAPE(256, 1);
  else if (D <= 2560) S6_NORM_SHAPE(320, 1);
  else if (D <= 4096) S6_NORM_SHAPE(512, 1);
  else if (D <= 8192) S6_NORM_SHAPE(512, 2);
  else S6_NORM_SHAPE(1024, 2);
#undef S6_NORM_SHAPE
}

int64_t bwd_blocks(int64_t rows, int64_t D) {
  int64_t n = 0;
  bwd_shape(D, [&](auto nt, auto) { n = (rows + rows_of(nt) - 1) / rows_of(nt); });
  return n < 768 ? n : 768;
}

template <typename IO, typename RES>
hipError_t bwd_types(const NormBwdArgs& b, float* part, hipStream_t s) {
  bwd_shape(b.f.D, [&](auto nt, auto nv) {
    constexpr int NT = decltype(nt)::value, NV = decltype(nv)::value;
    const dim3 grid((unsigned)bwd_blocks(b.f.rows, b.f.D)), block(NT * rows_of(NT));
    if (b.f.D % E == 0) hipLaunchKernelGGL((norm_bwd_kernel<IO, RES, NT, NV, true>), grid, block, 0, s, b, part);
    else hipLaunchKernelGGL((norm_bwd_kernel<IO, RES, NT, NV, false>), grid, block, 0, s, b, part);
  });
  return hipGetLastError();
}

}  // namespace

bool norm_fits(int64_t rows, int64_t D) {
  return rows * (D <= 512 ? 64 : (D <= 8192 ? 256 : 512)) < (int64_t(1) << 32) - 1024;
}

hipError_t launch_norm_fwd(const NormArgs& a, int io, int res, hipStream_t s) {
  if (io == kIoBF16) return res == kIoBF16 ? fwd_types<uint16_t, uint16_t>(a, s) : fwd_types<uint16_t, float>(a, s);
  return fwd_types<float, float>(a, s);
}

size_t norm_bwd_ws_bytes(int64_t rows, int64_t D) { return (size_t)bwd_blocks(rows, D) * 3 * (size_t)D * sizeof(float); }

hipError_t launch_norm_bwd(const NormBwdArgs& b, int io, int res, void* workspace, hipStream_t s) {
  float* part = static_cast<float*>(workspace);
  const int64_t D = b.f.D;
  hipError_t e = hipSuccess;
  if (b.f.rows > 0) {
    if (io == kIoBF16)
      e = res == kIoBF16 ? bwd_types<uint16_t, uint16_t>(b, part, s) : bwd_types<uint16_t, float>(b, part, s);
    else
      e = bwd_types<float, float>(b, part, s);
  }
  if (e != hipSuccess || !(b.dpost || b.dscale || b.dpre)) return e;
  hipLaunchKernelGGL(norm_sum_kernel, dim3((unsigned)((3 * D + 31) / 32)), dim3(1024), 0, s, part,
                     b.f.rows > 0 ? bwd_blocks(b.f.rows, D) : 0, D, b.f.alpha, b.dpost, b.dscale, b.dpre);
  return hipGetLastError();
}

}  // namespace s6
