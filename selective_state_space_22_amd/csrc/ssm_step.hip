// ssm_step.hip -- one token through a layer's short convolution, its selection projections and its state
// update, on gfx950.
//
// Per row b with place s (window and state of that place), channel d, state n:
//     x_c = SiLU(conv_bias + sum_j conv_weight_j (window, x)_j),   window moves on by x
//     (r, B, C) = x_c W_x^T,   dt = softplus(r W_dt^T + dt_bias)
//     h = e^{dt A} h + (e^{dt A} - 1)/A B x_c,   out = (C . h + D x_c) SiLU(z)
// ("Mamba 状态空间模型原理与 Transformer 对比", kb.agiseed.tech, eq. (2), (3a), (3b) and section 3.2).
//
// With many rows the states bound it (8 N bytes per row and channel against 2 (R + 2 N + R) operations); with
// one row it is latency, and the weights W_x and W_dt are what has to be read.  Two launches, because every
// dt needs all channels' x_c (three where a tile of rows has many part sums):
//   front  16 rows x a slice of channels: convolution, then the slice's part of x_c W_x^T on the matrix cores
//   join   (many rows) the slices' parts of r, B, C added in the order of the slices
//   back   16 rows x a block of channels: the states' loads are issued first and travel while r W_dt^T is
//          formed on the matrix cores; then the update, four states per lane as in the decode step
// x_c, r, B, C and dt stay fp32 between: each bf16 matrix operand made of them is split into three bf16 parts
// (8 + 8 + 8 bits of the 24) whose products are added in fp32, so a token is as exact as in fp32 throughout.
#include <type_traits>

#include "layer_device.h"
#include "layer_internal.h"

namespace s6 {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kRows = 16;     // batch rows of a tile: the matrix instruction's rows
constexpr int kSlice = 128;   // channels of a front workgroup
constexpr int kBlock = 256;
constexpr int kPad = 4;       // floats behind an LDS row: lanes of a quarter wave on distinct banks

// K elements of one matrix step, and of each lane's share (lane l: row l % 16, share l / 16 of the step).
template <typename IO>
constexpr int kStep = sizeof(IO) == 2 ? 32 : 16;
template <typename IO>
constexpr int kShare = kStep<IO> / 4;

// The A operand of one step, from fp32 values: bf16 as three parts, fp32 as it is.
template <typename IO>
struct OperandA;
template <>
struct OperandA<uint16_t> {
  bf16x8 part[3];
  __device__ __forceinline__ void set(const float* v) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float f = v[i];
#pragma unroll
      for (int p = 0; p < 3; ++p) {
        const __bf16 h = (__bf16)f;
        part[p][i] = h;
        f -= (float)h;  // exact: the rounding error of h
      }
    }
  }
  __device__ __forceinline__ f32x4 times(raw_t<uint16_t, 8> b, f32x4 c) const {
    const bf16x8 bb = __builtin_bit_cast(bf16x8, b);
#pragma unroll
    for (int p = 2; p >= 0; --p) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(part[p], bb, c, 0, 0, 0);
    return c;
  }
};
template <>
struct OperandA<float> {
  float f[4];
  __device__ __forceinline__ void set(const float* v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = v[i];
  }
  __device__ __forceinline__ f32x4 times(raw_t<float, 4> b, f32x4 c) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(f[i], __uint_as_float(b[i]), c, 0, 0, 0);
    return c;
  }
};

// A lane's share of a B operand: elements k .. k + kShare - 1 of a weight row of K elements (absent ones zero).
template <typename IO>
__device__ __forceinline__ raw_t<IO, kShare<IO>> operand_b(const IO* row, int64_t k, int64_t K, bool in) {
  constexpr int S = kShare<IO>;
  if (in && k + S <= K) return load_raw<IO, S, true>(row + k, S);
  if (in && k < K) return load_raw<IO, S, false>(row + k, (int)(K - k));
  return raw_t<IO, S>(0u);
}

__device__ __forceinline__ int64_t place_of(const SsmStepArgs& a, int64_t b) {
  if (b >= a.batch) return -1;
  const int64_t s = a.slots ? a.slots[b] : b;
  return s < a.nslots ? s : -1;
}

// x_c of four channels of one row, which also moves the window on.
template <typename IO, int W, bool FULL>
__device__ __forceinline__ void conv_four(const SsmStepArgs& a, int64_t b, int64_t slot, int64_t d0, int nv,
                                          float (&c)[4]) {
  IO* win = static_cast<IO*>(a.window) + slot * (W - 1) * a.D + d0;
  raw_t<IO, 4> row[W];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) row[j] = load_raw<IO, 4, FULL>(win + j * a.D, nv);
  row[W - 1] = load_raw<IO, 4, FULL>(static_cast<const IO*>(a.x) + b * a.D + d0, nv);
  float w[4 * W], bias[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 4 * W; ++i) w[i] = FULL || i < nv * W ? a.conv_weight[d0 * W + i] : 0.0f;
  if (a.conv_bias)
#pragma unroll
    for (int i = 0; i < 4; ++i) bias[i] = FULL || i < nv ? a.conv_bias[d0 + i] : 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = bias[i];
#pragma unroll
  for (int j = 0; j < W; ++j) {
    float v[4];
    widen<IO, 4>(row[j], v);
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = __builtin_fmaf(w[i * W + j], v[i], c[i]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = FULL || i < nv ? silu(c[i]) : 0.0f;
#pragma unroll
  for (int j = 0; j < W - 1; ++j) store_raw<IO, 4, FULL>(win + j * a.D, row[j + 1], nv);
}

// xc: (batch, D) fp32.  part: (slices, batch, F) fp32, F = R + 2 N.
template <typename IO, int W>
__global__ __launch_bounds__(kBlock) void ssm_front_kernel(SsmStepArgs a, int tiles, int slices, float* xc,
                                                           float* part) {
  constexpr int KS = kSlice / kStep<IO>;
  constexpr int TW = 3;  // column tiles of 16 that a wave multiplies together
  __shared__ __attribute__((aligned(16))) float xs[kRows][kSlice + kPad];
  // the tiles of a slice read the same rows of W_x: ids congruent mod 8 (one XCD), 8 apart
  const int id = blockIdx.x, round = id / (8 * tiles), rem = id % (8 * tiles);
  const int slice = round * 8 + rem % 8, tile = rem / 8;
  if (slice >= slices) return;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, q = lane >> 4;
  const int64_t F = a.R + 2 * a.N, d0 = (int64_t)slice * kSlice, b0 = (int64_t)tile * kRows;
  const IO* wx = static_cast<const IO*>(a.Wx);
  const int ntiles = (int)((F + 15) / 16);
  raw_t<IO, kShare<IO>> wb[TW][KS];
  auto load_b = [&](int t0) {
#pragma unroll
    for (int t = 0; t < TW; ++t) {
      const int64_t f = (int64_t)(t0 + 4 * t) * 16 + r16;
#pragma unroll
      for (int k = 0; k < KS; ++k)
        wb[t][k] = operand_b<IO>(wx + (f < F ? f : 0) * a.D, d0 + k * kStep<IO> + q * kShare<IO>, a.D, f < F);
    }
  };
  load_b(w);  // in flight during the convolution
#pragma unroll
  for (int i = 0; i < kRows * kSlice / 4 / kBlock; ++i) {
    const int e = i * kBlock + threadIdx.x, r = e / (kSlice / 4), g = e % (kSlice / 4) * 4;
    const int64_t b = b0 + r, d = d0 + g, slot = place_of(a, b);
    float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (slot >= 0 && d < a.D) {
      const int nv = a.D - d < 4 ? (int)(a.D - d) : 4;
      if (nv == 4) {
        conv_four<IO, W, true>(a, b, slot, d, 4, c);
        store_raw<float, 4, true>(xc + b * a.D + d, narrow<float, 4>(c), 4);
      } else {
        conv_four<IO, W, false>(a, b, slot, d, nv, c);
        store_raw<float, 4, false>(xc + b * a.D + d, narrow<float, 4>(c), nv);
      }
    }
    *reinterpret_cast<float4*>(&xs[r][g]) = make_float4(c[0], c[1], c[2], c[3]);
  }
  __syncthreads();
  OperandA<IO> op[KS];
#pragma unroll
  for (int k = 0; k < KS; ++k) op[k].set(&xs[r16][k * kStep<IO> + q * kShare<IO>]);
  for (int t0 = w; t0 < ntiles; t0 += 4 * TW) {
    f32x4 acc[TW];
#pragma unroll
    for (int t = 0; t < TW; ++t) {
      acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < KS; ++k) acc[t] = op[k].times(wb[t][k], acc[t]);
    }
    if (t0 + 4 * TW < ntiles) load_b(t0 + 4 * TW);
#pragma unroll
    for (int t = 0; t < TW; ++t) {
      const int64_t f = (int64_t)(t0 + 4 * t) * 16 + r16;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t b = b0 + 4 * q + i;
        if (f < F && b < a.batch) part[((int64_t)slice * a.batch + b) * F + f] = acc[t][i];
      }
    }
  }
}

// out: (batch, F), the slices' parts added in their order.
__global__ __launch_bounds__(kBlock) void ssm_join_kernel(const float* part, int64_t count, int slices, float* out) {
  const int64_t i = (int64_t)blockIdx.x * kBlock + threadIdx.x;
  if (i >= count) return;
  float v = 0.0f;
#pragma unroll 8
  for (int s = 0; s < slices; ++s) v += part[s * count + i];
  out[i] = v;
}

template <int N>
struct Lanes {
  static constexpr int kStates = N < 4 ? N : 4;       // states per lane
  static constexpr int kPer = N / kStates;            // lanes per channel
  static constexpr int kChannels = kBlock / kPer;     // channels per workgroup
};

// sel: (slices, batch, F) part sums of r, B, C.
template <typename IO, int N>
__global__ __launch_bounds__(kBlock) void ssm_back_kernel(SsmStepArgs a, int tiles, int ldx, const float* xc,
                                                          const float* sel, int slices) {
  constexpr int NS = Lanes<N>::kStates, LPC = Lanes<N>::kPer, CB = Lanes<N>::kChannels;
  constexpr int CT = CB / 16 / 4;  // channel tiles of 16 per wave
  extern __shared__ __attribute__((aligned(16))) float lds[];
  float* xd = lds;                        // (kRows, ldx): r, B, C of the rows
  float* dl = lds + kRows * ldx;          // (kRows, CB + kPad): r W_dt^T
  const int tile = blockIdx.x % (uint32_t)tiles;
  const int64_t d0 = (int64_t)(blockIdx.x / (uint32_t)tiles) * CB, b0 = (int64_t)tile * kRows;
  const int nrows = a.batch - b0 < kRows ? (int)(a.batch - b0) : kRows;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, q = lane >> 4;
  const int64_t F = a.R + 2 * N;
  // this lane's channel and states
  const int cl = threadIdx.x / LPC, n0 = threadIdx.x % LPC * NS;
  const int64_t d = d0 + cl;
  const bool in = d < a.D;
  float h[kRows][NS];
  int64_t at[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int64_t slot = r < nrows ? place_of(a, b0 + r) : -1;
    at[r] = in && slot >= 0 ? (slot * a.D + d) * N + n0 : -1;
#pragma unroll
    for (int n = 0; n < NS; ++n) h[r][n] = 0.0f;
    if (at[r] >= 0) {
      if constexpr (NS == 4) {
        const f32x4 v = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(a.state + at[r]));
#pragma unroll
        for (int n = 0; n < 4; ++n) h[r][n] = v[n];
      } else {
#pragma unroll
        for (int n = 0; n < NS; ++n) h[r][n] = a.state[at[r] + n];
      }
    }
  }
  // r, B, C of the tile's rows; what lies behind r in a matrix step is zero
  const int64_t RK = (a.R + kStep<IO> - 1) / kStep<IO> * kStep<IO>;
  float* xr = xd;                  // r at 0 .. RK, B and C behind
  for (int e = threadIdx.x; e < kRows * ldx; e += kBlock) {
    const int r = e / ldx, c = e % ldx;
    const int64_t f = c < RK ? c : a.R + (c - RK);
    float v = 0.0f;
    if (r < nrows && (c < a.R || (c >= RK && f < F)))
      for (int s = 0; s < slices; ++s) v += sel[((int64_t)s * a.batch + b0 + r) * F + f];
    xr[e] = v;
  }
  __syncthreads();
  const IO* wdt = static_cast<const IO*>(a.Wdt);
  f32x4 acc[CT];
#pragma unroll
  for (int t = 0; t < CT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int64_t k = 0; k < RK; k += kStep<IO>) {
    OperandA<IO> op;
    op.set(xd + r16 * ldx + k + q * kShare<IO>);
#pragma unroll
    for (int t = 0; t < CT; ++t) {
      const int64_t c = d0 + (w * CT + t) * 16 + r16;
      acc[t] = op.times(operand_b<IO>(wdt + (c < a.D ? c : 0) * a.R, k + q * kShare<IO>, a.R, c < a.D), acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < CT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) dl[(4 * q + i) * (CB + kPad) + (w * CT + t) * 16 + r16] = acc[t][i];
  __syncthreads();
  if (!in) return;
  ChanConst<NS> cc;
#pragma unroll
  for (int n = 0; n < NS; ++n) cc.set(n, a.A[d * N + n0 + n]);
  const float bias = a.dt_bias ? a.dt_bias[d] : 0.0f, dskip = a.dskip ? a.dskip[d] : 0.0f;
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (at[r] < 0) continue;  // the channel's lanes agree
    const int64_t i = (b0 + r) * a.D + d;
    const float* sel_r = xd + r * ldx + RK;
    float Bt[NS], Ct[NS];
#pragma unroll
    for (int n = 0; n < NS; ++n) {
      Bt[n] = sel_r[n0 + n];
      Ct[n] = sel_r[N + n0 + n];
    }
    const float x = xc[i];
    const TokenFront f = make_front(dl[r * (CB + kPad) + cl], bias, true);
    float y = token_step<NS>(cc, f, x, Bt, Ct, h[r]);
    if constexpr (LPC >= 2) y += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(y), 0xB1, 0xf, 0xf, false));
    if constexpr (LPC == 4) y += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(y), 0x4E, 0xf, 0xf, false));
    if constexpr (NS == 4) {
      const f32x4 v = {h[r][0], h[r][1], h[r][2], h[r][3]};
      __builtin_nontemporal_store(v, reinterpret_cast<f32x4*>(a.state + at[r]));
    } else {
#pragma unroll
      for (int n = 0; n < NS; ++n) a.state[at[r] + n] = h[r][n];
    }
    if (n0 == 0)
      store_io(static_cast<IO*>(a.out), i,
               epilogue(y, x, dskip, a.z != nullptr, a.z ? load_io(static_cast<const IO*>(a.z), i) : 0.0f));
  }
}

struct StepPlan {
  int tiles, slices, ldx;
  bool join;
  size_t off_part, off_sel, bytes;
};

StepPlan plan_step(int64_t batch, int64_t D, int64_t N, int64_t R, int io) {
  StepPlan p;
  const int64_t F = R + 2 * N, step = io == kIoBF16 ? kStep<uint16_t> : kStep<float>;
  p.tiles = (int)((batch + kRows - 1) / kRows);
  p.slices = (int)((D + kSlice - 1) / kSlice);
  p.ldx = (int)((R + step - 1) / step * step + 2 * N + kPad);
  p.ldx = (p.ldx + 3) / 4 * 4;
  // every back workgroup adds its rows' parts again: worth a launch less while they are few
  p.join = p.slices > 1 && batch > 4;
  auto al = [](size_t v) { return (v + 255) / 256 * 256; };
  p.off_part = al((size_t)batch * D * 4);
  p.off_sel = p.off_part + al((size_t)p.slices * batch * F * 4);
  p.bytes = p.off_sel + (p.join ? al((size_t)batch * F * 4) : 0);
  return p;
}

template <typename IO, int N>
hipError_t back(const SsmStepArgs& a, const StepPlan& p, const float* xc, const float* sel, int slices,
                hipStream_t s) {
  constexpr int CB = Lanes<N>::kChannels;
  const size_t lds = (size_t)kRows * (p.ldx + CB + kPad) * sizeof(float);
  hipLaunchKernelGGL((ssm_back_kernel<IO, N>), dim3((unsigned)(p.tiles * ((a.D + CB - 1) / CB))), dim3(kBlock), lds, s,
                     a, p.tiles, p.ldx, xc, sel, slices);
  return hipGetLastError();
}

template <typename IO>
hipError_t launch_t(const SsmStepArgs& a, const StepPlan& p, uint8_t* ws, hipStream_t s) {
  float* xc = reinterpret_cast<float*>(ws);
  float* part = reinterpret_cast<float*>(ws + p.off_part);
  float* sel = reinterpret_cast<float*>(ws + p.off_sel);
  const dim3 grid((unsigned)((p.slices + 7) / 8 * 8 * p.tiles));
  if (a.W == 2) hipLaunchKernelGGL((ssm_front_kernel<IO, 2>), grid, dim3(kBlock), 0, s, a, p.tiles, p.slices, xc, part);
  else if (a.W == 3) hipLaunchKernelGGL((ssm_front_kernel<IO, 3>), grid, dim3(kBlock), 0, s, a, p.tiles, p.slices, xc, part);
  else hipLaunchKernelGGL((ssm_front_kernel<IO, 4>), grid, dim3(kBlock), 0, s, a, p.tiles, p.slices, xc, part);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  int slices = p.slices;
  if (p.join) {
    const int64_t count = a.batch * (a.R + 2 * a.N);
    hipLaunchKernelGGL(ssm_join_kernel, dim3((unsigned)((count + kBlock - 1) / kBlock)), dim3(kBlock), 0, s, part, count,
                       slices, sel);
    slices = 1;
  } else {
    sel = part;
  }
  switch (a.N) {
    case 1: return back<IO, 1>(a, p, xc, sel, slices, s);
    case 2: return back<IO, 2>(a, p, xc, sel, slices, s);
    case 4: return back<IO, 4>(a, p, xc, sel, slices, s);
    case 8: return back<IO, 8>(a, p, xc, sel, slices, s);
    case 16: return back<IO, 16>(a, p, xc, sel, slices, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

size_t ssm_step_ws_bytes(int64_t batch, int64_t D, int64_t N, int64_t R, int io) {
  return plan_step(batch, D, N, R, io).bytes;
}

hipError_t launch_ssm_step(const SsmStepArgs& a, int io, void* workspace, hipStream_t s) {
  const StepPlan p = plan_step(a.batch, a.D, a.N, a.R, io);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  return io == kIoBF16 ? launch_t<uint16_t>(a, p, ws, s) : launch_t<float>(a, p, ws, s);
}

}  // namespace s6
