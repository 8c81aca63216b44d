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
// A few dozen operations per element: memory bounds it.  A row stays in the registers of its threads (part of a
// wave up to 128 elements, a wave up to 768, a workgroup beyond), so every tensor is read once and written once; the
// backward recomputes p and r' from the inputs instead of reading saved ones.  Sums of squares and products are
// fp32.  Measured (a streaming copy reaches 6.1 TB/s):
//   forward 16384 x 2560 bf16, fp32 residual    115 to 121 us, 587 MB: 5.0 TB/s; bound by memory
//   forward 16384 x 768 bf16    25 to 30 us, 126 MB: 4.6 TB/s;   4611 x 1101 fp32  16 us, 81 MB: 5.1 TB/s
//   gradients 16384 x 768 bf16  41 us, 201 MB: 4.9 TB/s;         4611 x 1101 fp32  27 us, 122 MB: 4.5 TB/s
//   sum over the workgroups' parts 5 us;  one row 1 x 2560 2.6 us: the launch and two sums' latency
#include <type_traits>

#include "layer_device.h"
#include "layer_internal.h"

namespace s6 {
namespace {

constexpr int E = 4;  // elements per thread and chunk: 16 bytes of fp32, 8 of bf16

// Sum over NT lanes of a wave (16, 32 or 64), the same value in all of them: within rows of 16 lanes by lane
// swaps, then the rows.
template <int NT>
__device__ __forceinline__ float lane_sum(float v) {
#define S6_DPP_ADD(ctrl) \
  v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), ctrl, 0xf, 0xf, false))
  S6_DPP_ADD(0xB1);   // lane ^ 1
  S6_DPP_ADD(0x4E);   // lane ^ 2
  S6_DPP_ADD(0x141);  // mirrored in 8
  S6_DPP_ADD(0x140);  // mirrored in 16
#undef S6_DPP_ADD
  if constexpr (NT == 16) return v;
  if constexpr (NT == 32) return v + __shfl_xor(v, 16, 64);
  const int i = __float_as_int(v);
  return (__int_as_float(__builtin_amdgcn_readlane(i, 0)) + __int_as_float(__builtin_amdgcn_readlane(i, 16))) +
         (__int_as_float(__builtin_amdgcn_readlane(i, 32)) + __int_as_float(__builtin_amdgcn_readlane(i, 48)));
}

// Sum over the NT threads of a row, the same value in all of them.  Rows of more than a wave meet at
// workgroup barriers: every thread of the workgroup takes part.
template <int NT, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float (*lds)[K]) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = lane_sum<(NT < 64 ? NT : 64)>(v[k]);
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

// How rows that E does not divide are read.
enum Rest {
  kEven,   // E divides D: chunks are whole or absent
  kShare,  // D >= E: the last chunk begins earlier and shares elements with the one before; both write them, with the
           // same values, and the sums over the row leave the shared ones out once
  kParts,  // the last chunk has fewer elements (rows shorter than a chunk; outputs that are inputs, where a shared
           // element could be read after it was written).  Its waves hold the row up: 4611 x 1101 fp32 with its
           // gradients 54 us, shared 45
};
// First element of the chunk that begins at e0 < D.
template <int REST>
__device__ __forceinline__ int64_t begin_of(int64_t e0, int64_t D) {
  return REST == kShare && e0 + E > D ? D - E : e0;
}
template <typename T, int REST>
__device__ __forceinline__ raw_t<T, E> chunk_in(const T* row, int64_t e0, int64_t D) {
  if (REST == kShare) {
    if (e0 < D) return load_raw<T, E, true>(row + begin_of<REST>(e0, D), E);
  } else {
    if (e0 + E <= D) return load_raw<T, E, true>(row + e0, E);
    if (REST == kParts && e0 < D) return load_raw<T, E, false>(row + e0, (int)(D - e0));
  }
  return raw_t<T, E>(0u);
}
template <typename T, int REST>
__device__ __forceinline__ void chunk_out(T* row, int64_t e0, int64_t D, const float (&f)[E]) {
  if (REST == kShare) {
    if (e0 < D) store_raw<T, E, true>(row + begin_of<REST>(e0, D), narrow<T, E>(f), E);
  } else {
    if (e0 + E <= D) store_raw<T, E, true>(row + e0, narrow<T, E>(f), E);
    else if (REST == kParts && e0 < D) store_raw<T, E, false>(row + e0, narrow<T, E>(f), (int)(D - e0));
  }
}
template <int REST>
__device__ __forceinline__ void weights_in(const float* w, int64_t e0, int64_t D, float (&f)[E]) {
  widen<float, E>(chunk_in<float, REST>(w, e0, D), f);
}
// sum + a b where element i of the chunk at e0 counts in the row's sums, else sum.
template <int REST>
__device__ __forceinline__ float count(float a, float b, float sum, int64_t e0, int i, int64_t D) {
  const float v = __builtin_fmaf(a, b, sum);
  return REST == kShare && e0 + E > D && i < (int)(e0 + E - D) ? sum : v;
}

// Rows per workgroup.
constexpr int rows_of(int nt) { return nt > 128 ? 1 : 256 / nt; }

template <typename IO, typename RES, int NT, int NV, int REST>
__global__ __launch_bounds__(NT* rows_of(NT)) void norm_fwd_kernel(NormArgs a) {
  constexpr int RPB = rows_of(NT);
  __shared__ float lds[NT * RPB / 64][1];
  const int lane = threadIdx.x % NT;
  const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / NT;
  // a row behind the last reads as one of no elements
  const int64_t D = row < a.rows ? a.D : 0, at = row * D;
  const float inv = 1.0f / (float)a.D;
  raw_t<IO, E> xr[NV], gr[NV];
  raw_t<RES, E> rr[NV];
#pragma unroll
  for (int c = 0; c < NV; ++c) xr[c] = chunk_in<IO, REST>(static_cast<const IO*>(a.x) + at, (c * NT + lane) * E, D);
  if (a.gate)
#pragma unroll
    for (int c = 0; c < NV; ++c)
      gr[c] = chunk_in<IO, REST>(static_cast<const IO*>(a.gate) + at, (c * NT + lane) * E, D);
  if (a.residual)
#pragma unroll
    for (int c = 0; c < NV; ++c)
      rr[c] = chunk_in<RES, REST>(static_cast<const RES*>(a.residual) + at, (c * NT + lane) * E, D);
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
    for (int i = 0; i < E; ++i) sum[0] = count<REST>(v[c][i], v[c][i], sum[0], (c * NT + lane) * E, i, D);
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
      weights_in<REST>(a.post, e0, D, w);
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
      weights_in<REST>(a.scale, e0, D, w);
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
    if (a.residual_out) chunk_out<RES, REST>(static_cast<RES*>(a.residual_out) + at, e0, D, v[c]);
#pragma unroll
    for (int i = 0; i < E; ++i) sum[0] = count<REST>(v[c][i], v[c][i], sum[0], (c * NT + lane) * E, i, D);
  }
  if (!a.pre) return;
  row_sum<NT, 1>(sum, lds);
  k = rsqrtf(__builtin_fmaf(sum[0], inv, a.eps));
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    const int64_t e0 = (c * NT + lane) * E;
    float w[E];
    weights_in<REST>(a.pre, e0, D, w);
#pragma unroll
    for (int i = 0; i < E; ++i) w[i] *= v[c][i] * k;
    chunk_out<IO, REST>(static_cast<IO*>(a.out) + at, e0, D, w);
  }
}

// Rows blockIdx.x, + gridDim.x, ... of RPB each; the sums over them go to part (gridDim.x, 3, D):
// dpost, dscale (without alpha), dpre.
template <typename IO, typename RES, int NT, int NV, int REST>
__global__ __launch_bounds__(NT* rows_of(NT)) void norm_bwd_kernel(NormBwdArgs b, float* part) {
  constexpr int RPB = rows_of(NT);
  __shared__ float lds[NT * RPB / 64][2];
  const NormArgs& a = b.f;
  const int lane = threadIdx.x % NT, slot = threadIdx.x / NT;
  const float inv = 1.0f / (float)a.D;
  const bool first_gate = a.gate && a.gate_first, after_gate = a.gate && !a.gate_first;
  // The weights stay in registers over the rows (absent ones as 1): post, alpha scale, pre.
  float post[NV][E], asc[NV][E], pre[NV][E];
  float spost[NV][E], sscale[NV][E], spre[NV][E];
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    const int64_t e0 = (c * NT + lane) * E;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      post[c][i] = asc[c][i] = pre[c][i] = 1.0f;
      spost[c][i] = sscale[c][i] = spre[c][i] = 0.0f;
    }
    if (a.post) weights_in<REST>(a.post, e0, a.D, post[c]);
    if (a.scale) weights_in<REST>(a.scale, e0, a.D, asc[c]);
    if (a.pre) weights_in<REST>(a.pre, e0, a.D, pre[c]);
#pragma unroll
    for (int i = 0; i < E; ++i) asc[c][i] *= a.alpha;
  }
  for (int64_t first = (int64_t)blockIdx.x * RPB; first < a.rows; first += (int64_t)gridDim.x * RPB) {
    // a row behind the last reads as one of no elements: all threads pass the same barriers
    const int64_t row = first + slot, D = row < a.rows ? a.D : 0, at = row * a.D;
    raw_t<IO, E> xr[NV], gr[NV], dor[NV];
    raw_t<RES, E> rr[NV], drr[NV];
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int64_t e0 = (c * NT + lane) * E;
      xr[c] = chunk_in<IO, REST>(static_cast<const IO*>(a.x) + at, e0, D);
      gr[c] = dor[c] = raw_t<IO, E>(0u);
      rr[c] = drr[c] = raw_t<RES, E>(0u);
      if (a.gate) gr[c] = chunk_in<IO, REST>(static_cast<const IO*>(a.gate) + at, e0, D);
      if (a.residual) rr[c] = chunk_in<RES, REST>(static_cast<const RES*>(a.residual) + at, e0, D);
      if (b.dout) dor[c] = chunk_in<IO, REST>(static_cast<const IO*>(b.dout) + at, e0, D);
      if (b.dres_out) drr[c] = chunk_in<RES, REST>(static_cast<const RES*>(b.dres_out) + at, e0, D);
    }
    // n = v / rms(v); s = SiLU(gate) and its slope sigma + s (1 - sigma)
    float n[NV][E], s[NV][E], slope[NV][E], s1[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      widen<IO, E>(xr[c], n[c]);
      if (a.gate) {
        widen<IO, E>(gr[c], s[c]);
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const float sg = sigmoid(s[c][i]);
          s[c][i] *= sg;
          slope[c][i] = __builtin_fmaf(s[c][i], 1.0f - sg, sg);
        }
        if (first_gate)
#pragma unroll
          for (int i = 0; i < E; ++i) n[c][i] *= s[c][i];
      }
#pragma unroll
      for (int i = 0; i < E; ++i) s1[0] = count<REST>(n[c][i], n[c][i], s1[0], (c * NT + lane) * E, i, D);
    }
    float k = 1.0f;
    if (a.post) {
      row_sum<NT, 1>(s1, reinterpret_cast<float(*)[1]>(lds));
      k = rsqrtf(__builtin_fmaf(s1[0], inv, a.eps));
    }
    // what n is multiplied by to give p
    auto factor = [&](int c, float (&f)[E]) {
#pragma unroll
      for (int i = 0; i < E; ++i) f[i] = post[c][i];
      if (after_gate)
#pragma unroll
        for (int i = 0; i < E; ++i) f[i] *= s[c][i];
    };
    // r', and the sums of the second norm
    float r[NV][E], s2[2] = {0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      float f[E];
      factor(c, f);
      widen<RES, E>(rr[c], r[c]);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        n[c][i] *= k;
        r[c][i] = __builtin_fmaf(asc[c][i], n[c][i] * f[i], r[c][i]);
      }
      if (b.dout) {
        float d[E];
        widen<IO, E>(dor[c], d);
#pragma unroll
        for (int i = 0; i < E; ++i) {
          s2[0] = count<REST>(r[c][i], r[c][i], s2[0], (c * NT + lane) * E, i, D);
          s2[1] = count<REST>(d[i] * pre[c][i], r[c][i], s2[1], (c * NT + lane) * E, i, D);
        }
      }
    }
    float K = 0.0f, kk = 0.0f;
    if (b.dout) {
      row_sum<NT, 2>(s2, lds);
      K = rsqrtf(__builtin_fmaf(s2[0], inv, a.eps));
      kk = K * (K * (s2[1] * inv));  // K * K alone may overflow
    }
    // dr, the sums over rows, dp (kept in r) and mean(e n), e = dp f
    s1[0] = 0.0f;
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      float dr[E], f[E];
      factor(c, f);
      widen<RES, E>(drr[c], dr);
      if (b.dout) {
        float d[E];
        widen<IO, E>(dor[c], d);
#pragma unroll
        for (int i = 0; i < E; ++i) {
          spre[c][i] = __builtin_fmaf(d[i], r[c][i] * K, spre[c][i]);
          dr[i] = __builtin_fmaf(K, __builtin_fmaf(-kk, r[c][i], d[i] * pre[c][i]), dr[i]);
        }
      }
      if (b.dresidual) chunk_out<RES, REST>(static_cast<RES*>(b.dresidual) + at, (c * NT + lane) * E, D, dr);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        sscale[c][i] = __builtin_fmaf(dr[i], n[c][i] * f[i], sscale[c][i]);
        r[c][i] = dr[i] * asc[c][i];
      }
      if (a.post) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
          spost[c][i] = __builtin_fmaf(after_gate ? r[c][i] * s[c][i] : r[c][i], n[c][i], spost[c][i]);
          s1[0] = count<REST>(r[c][i] * f[i], n[c][i], s1[0], (c * NT + lane) * E, i, D);
        }
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
      float dx[E], dg[E], f[E];
      factor(c, f);
#pragma unroll
      for (int i = 0; i < E; ++i) dx[i] = r[c][i] * f[i];
      if (a.post)  // else x itself reaches no gradient of its own, also where it is no number
#pragma unroll
        for (int i = 0; i < E; ++i) dx[i] = k * __builtin_fmaf(-n[c][i], m, dx[i]);
      if (a.gate) {
        if (first_gate) {
          float x[E];
          widen<IO, E>(xr[c], x);
#pragma unroll
          for (int i = 0; i < E; ++i) {
            dg[i] = dx[i] * x[i] * slope[c][i];
            dx[i] *= s[c][i];
          }
        } else {
#pragma unroll
          for (int i = 0; i < E; ++i) dg[i] = r[c][i] * post[c][i] * n[c][i] * slope[c][i];
        }
        if (b.dgate) chunk_out<IO, REST>(static_cast<IO*>(b.dgate) + at, e0, D, dg);
      }
      chunk_out<IO, REST>(static_cast<IO*>(b.dx) + at, e0, D, dx);
    }
  }
  // the sums of the workgroup's row slots, in their order
  const int64_t D = a.D;
  float* out = part + (int64_t)blockIdx.x * 3 * D;
  if constexpr (RPB == 1) {
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int64_t e0 = (c * NT + lane) * E;
      chunk_out<float, REST>(out, e0, D, spost[c]);
      chunk_out<float, REST>(out + D, e0, D, sscale[c]);
      chunk_out<float, REST>(out + 2 * D, e0, D, spre[c]);
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
        chunk_out<float, REST>(out, e0, D, spost[c]);
        chunk_out<float, REST>(out + D, e0, D, sscale[c]);
        chunk_out<float, REST>(out + 2 * D, e0, D, spre[c]);
      }
  }
}

// Long rows, whose sums over rows would not fit the registers beside the row: first each row's k, K,
// K^2 mean(dn' r') and mean(e n) ...
template <typename IO, typename RES, int NT, int NV, int REST>
__global__ __launch_bounds__(NT) void norm_stats_kernel(NormBwdArgs b, float4* stats) {
  static_assert(rows_of(NT) == 1, "a workgroup per row");
  __shared__ float lds[NT / 64][2];
  const NormArgs& a = b.f;
  const int lane = threadIdx.x;
  const int64_t D = a.D, row = blockIdx.x, at = row * D;
  const float inv = 1.0f / (float)D;
  const bool after_gate = a.gate && !a.gate_first;
  raw_t<IO, E> xr[NV], gr[NV], dor[NV];
  raw_t<RES, E> rr[NV], drr[NV];
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    const int64_t e0 = (c * NT + lane) * E;
    xr[c] = chunk_in<IO, REST>(static_cast<const IO*>(a.x) + at, e0, D);
    if (a.gate) gr[c] = chunk_in<IO, REST>(static_cast<const IO*>(a.gate) + at, e0, D);
    if (a.residual) rr[c] = chunk_in<RES, REST>(static_cast<const RES*>(a.residual) + at, e0, D);
    if (b.dout) dor[c] = chunk_in<IO, REST>(static_cast<const IO*>(b.dout) + at, e0, D);
    if (b.dres_out) drr[c] = chunk_in<RES, REST>(static_cast<const RES*>(b.dres_out) + at, e0, D);
  }
  float n[NV][E], f[NV][E], r[NV][E], s1[1] = {0.0f}, s2[2] = {0.0f, 0.0f};
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    const int64_t e0 = (c * NT + lane) * E;
    widen<IO, E>(xr[c], n[c]);
#pragma unroll
    for (int i = 0; i < E; ++i) f[c][i] = 1.0f;
    if (a.gate) {
      float g[E];
      widen<IO, E>(gr[c], g);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        if (after_gate) f[c][i] = silu(g[i]);
        else n[c][i] *= silu(g[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < E; ++i) s1[0] = count<REST>(n[c][i], n[c][i], s1[0], (c * NT + lane) * E, i, D);
  }
  float k = 1.0f;
  if (a.post) {
    row_sum<NT, 1>(s1, reinterpret_cast<float(*)[1]>(lds));
    k = rsqrtf(__builtin_fmaf(s1[0], inv, a.eps));
  }
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    const int64_t e0 = (c * NT + lane) * E;
    float w[E], d[E];
    if (a.post) {
      weights_in<REST>(a.post, e0, D, w);
#pragma unroll
      for (int i = 0; i < E; ++i) f[c][i] *= w[i];
    }
#pragma unroll
    for (int i = 0; i < E; ++i) {
      n[c][i] *= k;
      r[c][i] = a.alpha * n[c][i] * f[c][i];
    }
    if (a.scale) {
      weights_in<REST>(a.scale, e0, D, w);
#pragma unroll
      for (int i = 0; i < E; ++i) r[c][i] *= w[i];
    }
    if (a.residual) {
      widen<RES, E>(rr[c], w);
#pragma unroll
      for (int i = 0; i < E; ++i) r[c][i] += w[i];
    }
    if (b.dout) {
      widen<IO, E>(dor[c], d);
      weights_in<REST>(a.pre, e0, D, w);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        s2[0] = count<REST>(r[c][i], r[c][i], s2[0], e0, i, D);
        s2[1] = count<REST>(d[i] * w[i], r[c][i], s2[1], e0, i, D);
      }
    }
  }
  float K = 0.0f, kk = 0.0f;
  if (b.dout) {
    row_sum<NT, 2>(s2, lds);
    K = rsqrtf(__builtin_fmaf(s2[0], inv, a.eps));
    kk = K * (K * (s2[1] * inv));
  }
  s1[0] = 0.0f;
  if (a.post) {
#pragma unroll
    for (int c = 0; c < NV; ++c) {
      const int64_t e0 = (c * NT + lane) * E;
      float dr[E], w[E], d[E];
#pragma unroll
      for (int i = 0; i < E; ++i) dr[i] = 0.0f;
      if (b.dres_out) widen<RES, E>(drr[c], dr);
      if (b.dout) {
        widen<IO, E>(dor[c], d);
        weights_in<REST>(a.pre, e0, D, w);
#pragma unroll
        for (int i = 0; i < E; ++i) dr[i] = __builtin_fmaf(K, __builtin_fmaf(-kk, r[c][i], d[i] * w[i]), dr[i]);
      }
      if (a.scale) {
        weights_in<REST>(a.scale, e0, D, w);
#pragma unroll
        for (int i = 0; i < E; ++i) dr[i] *= w[i];
      }
#pragma unroll
      for (int i = 0; i < E; ++i) s1[0] = count<REST>(a.alpha * dr[i] * f[c][i], n[c][i], s1[0], e0, i, D);
    }
    row_sum<NT, 1>(s1, reinterpret_cast<float(*)[1]>(lds));
  }
  if (lane == 0) stats[row] = make_float4(k, K, kk, s1[0] * inv);
}

// ... then everything else element by element: a thread has E columns of the rows of its chunk, and their sums.
constexpr int kColRows = 4;  // row chunks (waves) of a workgroup

template <typename IO, typename RES, int REST>
__global__ __launch_bounds__(64 * kColRows) void norm_cols_kernel(NormBwdArgs b, const float4* stats, int64_t chunk,
                                                                  float* part) {
  const NormArgs& a = b.f;
  const int64_t D = a.D, e0 = ((int64_t)blockIdx.x * 64 + (threadIdx.x & 63)) * E;
  const int64_t ch = (int64_t)blockIdx.y * kColRows + (threadIdx.x >> 6);
  const int64_t r0 = ch * chunk, r1 = r0 + chunk < a.rows ? r0 + chunk : a.rows;
  if (r0 >= a.rows) return;
  const bool first_gate = a.gate && a.gate_first, after_gate = a.gate && !a.gate_first;
  float post[E], asc[E], pre[E], spost[E], sscale[E], spre[E];
#pragma unroll
  for (int i = 0; i < E; ++i) {
    post[i] = asc[i] = pre[i] = 1.0f;
    spost[i] = sscale[i] = spre[i] = 0.0f;
  }
  if (a.post) weights_in<REST>(a.post, e0, D, post);
  if (a.scale) weights_in<REST>(a.scale, e0, D, asc);
  if (a.pre) weights_in<REST>(a.pre, e0, D, pre);
#pragma unroll
  for (int i = 0; i < E; ++i) asc[i] *= a.alpha;
  for (int64_t row = r0; row < r1; ++row) {
    const int64_t at = row * D;
    raw_t<IO, E> gr(0u), dor(0u);
    raw_t<RES, E> rr(0u), drr(0u);
    const raw_t<IO, E> xr = chunk_in<IO, REST>(static_cast<const IO*>(a.x) + at, e0, D);
    if (a.gate) gr = chunk_in<IO, REST>(static_cast<const IO*>(a.gate) + at, e0, D);
    if (a.residual) rr = chunk_in<RES, REST>(static_cast<const RES*>(a.residual) + at, e0, D);
    if (b.dout) dor = chunk_in<IO, REST>(static_cast<const IO*>(b.dout) + at, e0, D);
    if (b.dres_out) drr = chunk_in<RES, REST>(static_cast<const RES*>(b.dres_out) + at, e0, D);
    const float4 st = stats[row];  // k, K, K^2 mean(dn' r'), mean(e n)
    float x[E], s[E], slope[E], r[E], d[E], dr[E], dx[E], dg[E];
    widen<IO, E>(xr, x);
    widen<IO, E>(gr, s);
    widen<RES, E>(rr, r);
    widen<IO, E>(dor, d);
    widen<RES, E>(drr, dr);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float sg = sigmoid(s[i]);
      s[i] *= sg;
      slope[i] = __builtin_fmaf(s[i], 1.0f - sg, sg);
      const float n = (first_gate ? x[i] * s[i] : x[i]) * st.x;
      const float f = after_gate ? post[i] * s[i] : post[i];
      const float q = n * f;
      r[i] = __builtin_fmaf(asc[i], q, r[i]);
      if (b.dout) {  // else r' reaches no gradient, also where it is no number
        spre[i] = __builtin_fmaf(d[i], r[i] * st.y, spre[i]);
        dr[i] = __builtin_fmaf(st.y, __builtin_fmaf(-st.z, r[i], d[i] * pre[i]), dr[i]);
      }
      sscale[i] = __builtin_fmaf(dr[i], q, sscale[i]);
      const float dp = dr[i] * asc[i];
      spost[i] = __builtin_fmaf(after_gate ? dp * s[i] : dp, n, spost[i]);
      float dv = dp * f;
      if (a.post) dv = st.x * __builtin_fmaf(-n, st.w, dv);
      dx[i] = first_gate ? dv * s[i] : dv;
      dg[i] = (first_gate ? dv * x[i] : dp * post[i] * n) * slope[i];
    }
    if (b.dresidual) chunk_out<RES, REST>(static_cast<RES*>(b.dresidual) + at, e0, D, dr);
    if (b.dgate) chunk_out<IO, REST>(static_cast<IO*>(b.dgate) + at, e0, D, dg);
    chunk_out<IO, REST>(static_cast<IO*>(b.dx) + at, e0, D, dx);
  }
  float* out = part + ch * 3 * D;
  chunk_out<float, REST>(out, e0, D, spost);
  chunk_out<float, REST>(out + D, e0, D, sscale);
  chunk_out<float, REST>(out + 2 * D, e0, D, spre);
}

template <int C>
__global__ __launch_bounds__(1024) void norm_sum_kernel(const float* part, int64_t rows, int64_t D, float alpha,
                                                        float* dpost, float* dscale, float* dpre) {
  const int64_t col = (int64_t)blockIdx.x * C + threadIdx.x % C;
  const float v = column_sum<C>(part, rows, 3 * D, col);
  if (threadIdx.x >= C || col >= 3 * D) return;
  if (col < D) {
    if (dpost) dpost[col] = v;
  } else if (col < 2 * D) {
    if (dscale) dscale[col - D] = alpha * v;
  } else if (dpre) {
    dpre[col - 2 * D] = v;
  }
}

// Threads and chunks per thread of a row, in steps: a row just above one leaves threads idle, which take a part of the
// workgroup's registers all the same (forward and gradients of 1892 x 4576 bf16: 640 threads 67 us, 1024 78, 512 with four
// chunks 69).  The widest steps are 2561 to 4096 and 8193 to 16384 elements, where up to 37% and a half of them idle.
template <typename F>
void row_shape(int64_t D, F f) {
#define S6_NORM_SHAPE(nt, nv) f(std::integral_constant<int, nt>(), std::integral_constant<int, nv>())
  if (D <= 64) S6_NORM_SHAPE(16, 1);
  else if (D <= 128) S6_NORM_SHAPE(32, 1);
  else if (D <= 256) S6_NORM_SHAPE(64, 1);
  else if (D <= 512) S6_NORM_SHAPE(64, 2);
  else if (D <= 768) S6_NORM_SHAPE(64, 3);
  else if (D <= 1024) S6_NORM_SHAPE(128, 2);
  else if (D <= 1536) S6_NORM_SHAPE(192, 2);
  else if (D <= 2048) S6_NORM_SHAPE(256, 2);
  else if (D <= 2560) S6_NORM_SHAPE(320, 2);
  else if (D <= 4096) S6_NORM_SHAPE(512, 2);
  else if (D <= 5120) S6_NORM_SHAPE(640, 2);
  else if (D <= 6144) S6_NORM_SHAPE(768, 2);
  else if (D <= 8192) S6_NORM_SHAPE(1024, 2);
  else S6_NORM_SHAPE(1024, 4);  // fp32 rows that E does not divide spill four registers (700 x 12003 111 us, 12004 104)
#undef S6_NORM_SHAPE
}

template <typename F>
void by_rest(int64_t D, bool in_place, F f) {
  if (D % E == 0) f(std::integral_constant<int, kEven>());
  else if (D > E && !in_place) f(std::integral_constant<int, kShare>());
  else f(std::integral_constant<int, kParts>());
}

// Whether an output is an input's buffer.
template <int M, int N>
bool share(const void* const (&out)[M], const void* const (&in)[N]) {
  for (const void* o : out)
    for (const void* i : in)
      if (o && o == i) return true;
  return false;
}

template <typename IO, typename RES>
hipError_t fwd_types(const NormArgs& a, hipStream_t s) {
  const bool in_place = share({a.out, a.residual_out}, {a.x, a.gate, a.residual});
  row_shape(a.D, [&](auto nt, auto nv) {
    constexpr int NT = decltype(nt)::value, NV = decltype(nv)::value, RPB = rows_of(NT);
    const dim3 grid((unsigned)((a.rows + RPB - 1) / RPB)), block(NT * RPB);
    by_rest(a.D, in_place, [&](auto rest) {
      hipLaunchKernelGGL((norm_fwd_kernel<IO, RES, NT, NV, decltype(rest)::value>), grid, block, 0, s, a);
    });
  });
  return hipGetLastError();
}

// Rows up to here keep the sums over rows beside the row; beyond, those do not fit its registers (forward and gradients
// 2048 x 4096: 56 us bf16 and 92 fp32 so, 67 and 120 in two passes; 2048 x 8192 bf16: 327 us so, 197 in two passes).
constexpr int64_t kSumsDim = 4096;

struct NormBwdPlan {
  int64_t parts;  // rows of part sums
  int64_t chunk;  // long rows: rows per part
  size_t off_stats, bytes;
};

NormBwdPlan plan_norm_bwd(int64_t rows, int64_t D) {
  NormBwdPlan p{0, 0, 0, 0};
  if (D <= kSumsDim) {
    row_shape(D, [&](auto nt, auto nv) {
      // Workgroups that stay: four a compute unit with one chunk a thread, else two, or one of more than 256 threads.  Two
      // waves per SIMD are what the registers of three chunks leave (225 to 250; 16384 x 768 bf16: 512 workgroups 38 us,
      // 640 53, 768 48, 1024 44); those of two chunks (156 to 190) leave two or three.  Forward and gradients in bf16 or,
      // marked, fp32 with this count, 1.5 and 2 times it: 16384 x 512 38.2, 38.0, 43 us; 9000 x 1024 f 73.5, 79, 78.6;
      // 4611 x 1101 f 47.0, 45.2, 51.5; 8192 x 1536 87.7, 79.0, 91; 5000 x 2048 49.7, 48.5, 54.6; 4096 x 2560 96, 112, 100;
      // 2048 x 4096 43.3, 50, 49.  One chunk, half of it, this count and twice: 40000 x 250 56.7, 48.7, 51.
      const int64_t most = 256 * (nv == 1 ? 4 : (nt * rows_of(nt) <= 256 ? 2 : 1));
      p.parts = (rows + rows_of(nt) - 1) / rows_of(nt);
      p.parts = p.parts < most ? p.parts : most;
    });
  } else {
    // enough waves for the chip, and at least 16 rows each
    const int64_t waves = (D + 64 * E - 1) / (64 * E);
    int64_t n = (4096 + waves - 1) / waves;
    n = n < (rows + 15) / 16 ? n : (rows + 15) / 16;
    p.chunk = n < 1 ? 1 : (rows + n - 1) / n;
    p.parts = p.chunk < 1 ? 0 : (rows + p.chunk - 1) / p.chunk;
  }
  p.off_stats = ((size_t)p.parts * 3 * (size_t)D * sizeof(float) + 255) / 256 * 256;
  p.bytes = D <= kSumsDim ? (size_t)p.parts * 3 * (size_t)D * sizeof(float) : p.off_stats + (size_t)rows * sizeof(float4);
  return p;
}

template <typename IO, typename RES>
hipError_t bwd_types(const NormBwdArgs& b, const NormBwdPlan& p, float* part, hipStream_t s) {
  const int64_t D = b.f.D;
  const bool in_place = share({b.dx, b.dgate, b.dresidual}, {b.f.x, b.f.gate, b.f.residual, b.dout, b.dres_out});
  row_shape(D, [&](auto nt, auto nv) {
    constexpr int NT = decltype(nt)::value, NV = decltype(nv)::value;
    by_rest(D, in_place, [&](auto rest) {
      constexpr int REST = decltype(rest)::value;
      if constexpr (NT * NV * E <= kSumsDim) {
        hipLaunchKernelGGL((norm_bwd_kernel<IO, RES, NT, NV, REST>), dim3((unsigned)p.parts), dim3(NT * rows_of(NT)), 0, s,
                           b, part);
      } else {
        float4* stats = reinterpret_cast<float4*>(reinterpret_cast<uint8_t*>(part) + p.off_stats);
        const dim3 grid((unsigned)((D + 64 * E - 1) / (64 * E)), (unsigned)((p.parts + kColRows - 1) / kColRows));
        hipLaunchKernelGGL((norm_stats_kernel<IO, RES, NT, NV, REST>), dim3((unsigned)b.f.rows), dim3(NT), 0, s, b, stats);
        hipLaunchKernelGGL((norm_cols_kernel<IO, RES, REST>), grid, dim3(64 * kColRows), 0, s, b, stats, p.chunk, part);
      }
    });
  });
  return hipGetLastError();
}

}  // namespace

bool norm_fits(int64_t rows, int64_t D) {
  // a launch counts its threads in 32 bits; row_shape() has no more threads a row than these
  return rows * (D <= 768 ? 64 : (D <= 1536 ? 192 : (D <= 4096 ? 512 : 1024))) < (int64_t(1) << 31);
}

hipError_t launch_norm_fwd(const NormArgs& a, int io, int res, hipStream_t s) {
  if (io == kIoBF16) return res == kIoBF16 ? fwd_types<uint16_t, uint16_t>(a, s) : fwd_types<uint16_t, float>(a, s);
  return fwd_types<float, float>(a, s);
}

size_t norm_bwd_ws_bytes(int64_t rows, int64_t D) { return plan_norm_bwd(rows, D).bytes; }

hipError_t launch_norm_bwd(const NormBwdArgs& b, int io, int res, void* workspace, hipStream_t s) {
  float* part = static_cast<float*>(workspace);
  const int64_t D = b.f.D;
  const NormBwdPlan p = plan_norm_bwd(b.f.rows, D);
  hipError_t e = hipSuccess;
  if (b.f.rows > 0) {
    if (io == kIoBF16)
      e = res == kIoBF16 ? bwd_types<uint16_t, uint16_t>(b, p, part, s) : bwd_types<uint16_t, float>(b, p, part, s);
    else
      e = bwd_types<float, float>(b, p, part, s);
  }
  if (e != hipSuccess || !(b.dpost || b.dscale || b.dpre)) return e;
  by_columns(3 * D, [&](auto c) {
    constexpr int C = decltype(c)::value;
    hipLaunchKernelGGL((norm_sum_kernel<C>), dim3((unsigned)((3 * D + C - 1) / C)), dim3(1024), 0, s, part, p.parts, D,
                       b.f.alpha, b.dpost, b.dscale, b.dpre);
  });
  return hipGetLastError();
}

}  // namespace s6
