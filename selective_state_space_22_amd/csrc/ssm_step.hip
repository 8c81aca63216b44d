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

// x_c of four channels of kItems rows, kBlock threads apart, which also moves the windows on.  All loads are
// issued before the first of them is needed.
constexpr int kItems = kRows * kSlice / 4 / kBlock;

template <typename IO, int W, bool FULL>
__device__ __forceinline__ void conv_four(const SsmStepArgs& a, int64_t b0, int r0, int64_t d0, int nv, float* xc,
                                          float (&c)[kItems][4]) {
  constexpr int kApart = kBlock / (kSlice / 4);  // rows between two items of a thread
  int64_t slot[kItems];
  raw_t<IO, 4> row[kItems][W];
#pragma unroll
  for (int i = 0; i < kItems; ++i) slot[i] = place_of(a, b0 + r0 + i * kApart);
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
#pragma unroll
    for (int j = 0; j < W; ++j) row[i][j] = raw_t<IO, 4>(0u);
    if (slot[i] < 0) continue;
    row[i][W - 1] = load_raw<IO, 4, FULL>(static_cast<const IO*>(a.x) + (b0 + r0 + i * kApart) * a.D + d0, nv);
    const IO* win = static_cast<const IO*>(a.window) + slot[i] * (W - 1) * a.D + d0;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) row[i][j] = load_raw<IO, 4, FULL>(win + j * a.D, nv);
  }
  float w[W][4], bias[4] = {0.0f, 0.0f, 0.0f, 0.0f};  // the 4 W weights side by side
#pragma unroll
  for (int k = 0; k < W; ++k)
    widen<float, 4>(load_raw<float, 4, FULL>(a.conv_weight + d0 * W + 4 * k, nv * W - 4 * k), w[k]);
  if (a.conv_bias) widen<float, 4>(load_raw<float, 4, FULL>(a.conv_bias + d0, nv), bias);
#pragma unroll
  for (int i = 0; i < kItems; ++i) {
#pragma unroll
    for (int k = 0; k < 4; ++k) c[i][k] = 0.0f;
    if (slot[i] < 0) continue;
#pragma unroll
    for (int k = 0; k < 4; ++k) c[i][k] = bias[k];
#pragma unroll
    for (int j = 0; j < W; ++j) {
      float v[4];
      widen<IO, 4>(row[i][j], v);
#pragma unroll
      for (int k = 0; k < 4; ++k) c[i][k] = __builtin_fmaf(w[(k * W + j) / 4][(k * W + j) % 4], v[k], c[i][k]);
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) c[i][k] = FULL || k < nv ? silu(c[i][k]) : 0.0f;
    IO* win = static_cast<IO*>(a.window) + slot[i] * (W - 1) * a.D + d0;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) store_raw<IO, 4, FULL>(win + j * a.D, row[i][j + 1], nv);
    store_raw<float, 4, FULL>(xc + (b0 + r0 + i * kApart) * a.D + d0, narrow<float, 4>(c[i]), nv);
  }
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
  {
    const int r = threadIdx.x / (kSlice / 4), g = threadIdx.x % (kSlice / 4) * 4;
    const int64_t d = d0 + g;
    float c[kItems][4] = {};
    if (d + 4 <= a.D) conv_four<IO, W, true>(a, b0, r, d, 4, xc, c);
    else if (d < a.D) conv_four<IO, W, false>(a, b0, r, d, (int)(a.D - d), xc, c);
#pragma unroll
    for (int i = 0; i < kItems; ++i)
      *reinterpret_cast<float4*>(&xs[r + i * (kBlock / (kSlice / 4))][g]) = make_float4(c[i][0], c[i][1], c[i][2], c[i][3]);
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

// Sum over the slices of one value, in their order, 16 loads in flight.
__device__ __forceinline__ float slice_sum(const float* p, int64_t stride, int slices) {
  float v = 0.0f;
  int s = 0;
  for (; s + 16 <= slices; s += 16) {
    float q[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) q[i] = p[(s + i) * stride];
#pragma unroll
    for (int i = 0; i < 16; ++i) v += q[i];
  }
  for (; s + 4 <= slices; s += 4) {
    float q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = p[(s + i) * stride];
#pragma unroll
    for (int i = 0; i < 4; ++i) v += q[i];
  }
  for (; s < slices; ++s) v += p[s * stride];
  return v;
}

// out: (batch, F), the slices' parts added in their order.
__global__ __launch_bounds__(kBlock) void ssm_join_kernel(const float* part, int64_t count, int slices, float* out) {
  const int64_t i = (int64_t)blockIdx.x * kBlock + threadIdx.x;
  if (i < count) out[i] = slice_sum(part + i, count, slices);
}

constexpr int kChannels = 64;  // channels of a back workgroup

template <int N>
struct Lanes {
  static constexpr int kStates = N < 4 ? N : 4;                    // states per lane
  static constexpr int kPer = N / kStates;                         // lanes per channel
  static constexpr int kGroups = kBlock / (kChannels * kPer);      // row groups: a lane has every kGroups-th row
  static constexpr int kRowsPer = kRows / kGroups;                 // rows per lane
};

// sel: (slices, batch, F) part sums of r, B, C.
template <typename IO, int N>
__global__ __launch_bounds__(kBlock, 3) void ssm_back_kernel(SsmStepArgs a, int tiles, int ldx, const float* xc,
                                                          const float* sel, int slices) {
  constexpr int NS = Lanes<N>::kStates, LPC = Lanes<N>::kPer, RG = Lanes<N>::kGroups, RP = Lanes<N>::kRowsPer;
  constexpr int CB = kChannels, LD = CB + kPad;
  constexpr int PRE = 6;  // matrix steps whose weights are loaded ahead
  __shared__ int place[kRows];
  extern __shared__ __attribute__((aligned(16))) float lds[];
  float* xd = lds;               // (kRows, ldx): r, B, C of the rows
  float* dl = xd + kRows * ldx;  // (kRows, LD): r W_dt^T
  float* xl = dl + kRows * LD;   // (kRows, LD): x_c
  float* zl = xl + kRows * LD;   // (kRows, LD): z, then out
  const int tile = blockIdx.x % (uint32_t)tiles;
  const int64_t d0 = (int64_t)(blockIdx.x / (uint32_t)tiles) * CB, b0 = (int64_t)tile * kRows;
  const int nrows = a.batch - b0 < kRows ? (int)(a.batch - b0) : kRows;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, q = lane >> 4;
  const int64_t F = a.R + 2 * N;
  const int64_t RK = (a.R + kStep<IO> - 1) / kStep<IO> * kStep<IO>;
  // this lane's channel, states and first row
  const int cl = threadIdx.x / LPC % CB, n0 = threadIdx.x % LPC * NS, rg = threadIdx.x / (LPC * CB);
  const int64_t d = d0 + cl;
  const bool in = d < a.D;
  if (threadIdx.x < kRows) place[threadIdx.x] = (int)place_of(a, b0 + threadIdx.x);
  // weights of r, ahead of everything that waits; wave w multiplies channels 16 w .. 16 w + 15
  const int64_t cw = d0 + w * 16 + r16;
  const IO* wdt = static_cast<const IO*>(a.Wdt) + (cw < a.D ? cw : 0) * a.R;
  raw_t<IO, kShare<IO>> pre[PRE];
#pragma unroll
  for (int p = 0; p < PRE; ++p) pre[p] = operand_b<IO>(wdt, p * kStep<IO> + q * kShare<IO>, a.R, cw < a.D);
  // the states: needed last, so they travel while the rest is formed
  float h[RP][NS];
#pragma unroll
  for (int i = 0; i < RP; ++i) {
    const int64_t slot = place_of(a, b0 + i * RG + rg);
#pragma unroll
    for (int n = 0; n < NS; ++n) h[i][n] = 0.0f;
    if (in && slot >= 0) {
      const float* st = a.state + (slot * a.D + d) * N + n0;
      if constexpr (NS == 4) {
        const f32x4 v = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(st));
#pragma unroll
        for (int n = 0; n < 4; ++n) h[i][n] = v[n];
      } else {
#pragma unroll
        for (int n = 0; n < NS; ++n) h[i][n] = st[n];
      }
    }
  }
  // r, B, C of the tile's rows (r at 0 .. RK, zero behind R; B and C behind that), x_c and z
  for (int e = threadIdx.x; e < nrows * ldx; e += kBlock) {
    const int r = e / ldx, c = e % ldx;
    const int64_t f = c < RK ? c : a.R + (c - RK);
    float v = 0.0f;
    if (c < a.R || (c >= RK && f < F)) v = slice_sum(sel + (b0 + r) * F + f, a.batch * F, slices);
    xd[e] = v;
  }
  for (int e = nrows * ldx + threadIdx.x; e < kRows * ldx; e += kBlock) xd[e] = 0.0f;
  for (int e = threadIdx.x; e < nrows * (CB / 4); e += kBlock) {
    const int r = e / (CB / 4), g = e % (CB / 4) * 4;
    const int64_t dg = d0 + g, i = (b0 + r) * a.D + dg;
    const int nv = a.D - dg < 4 ? (int)(a.D - dg) : 4;
    raw_t<float, 4> xv(0u);
    raw_t<IO, 4> zv(0u);
    if (nv == 4) {
      xv = load_raw<float, 4, true>(xc + i, 4);
      if (a.z) zv = load_raw<IO, 4, true>(static_cast<const IO*>(a.z) + i, 4);
    } else {
      xv = load_raw<float, 4, false>(xc + i, nv);
      if (a.z) zv = load_raw<IO, 4, false>(static_cast<const IO*>(a.z) + i, nv);
    }
    float z4[4];
    widen<IO, 4>(zv, z4);
    *reinterpret_cast<raw_t<float, 4>*>(xl + r * LD + g) = xv;
    *reinterpret_cast<float4*>(zl + r * LD + g) = make_float4(z4[0], z4[1], z4[2], z4[3]);
  }
  __syncthreads();
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int p = 0; p < PRE; ++p) {
    if (p * kStep<IO> >= RK) break;
    OperandA<IO> op;
    op.set(xd + r16 * ldx + p * kStep<IO> + q * kShare<IO>);
    acc = op.times(pre[p], acc);
  }
  for (int64_t k = PRE * kStep<IO>; k < RK; k += kStep<IO>) {
    OperandA<IO> op;
    op.set(xd + r16 * ldx + k + q * kShare<IO>);
    acc = op.times(operand_b<IO>(wdt, k + q * kShare<IO>, a.R, cw < a.D), acc);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) dl[(4 * q + i) * LD + w * 16 + r16] = acc[i];
  __syncthreads();
  if (in) {
    ChanConst<NS> cc;
#pragma unroll
    for (int n = 0; n < NS; ++n) cc.set(n, a.A[d * N + n0 + n]);
    const float bias = a.dt_bias ? a.dt_bias[d] : 0.0f, dskip = a.dskip ? a.dskip[d] : 0.0f;
#pragma unroll
    for (int i = 0; i < RP; ++i) {
      const int r = i * RG + rg;
      const int64_t slot = place[r];
      if (slot < 0) continue;  // the channel's lanes agree
      const float* sel_r = xd + r * ldx + RK;
      float Bt[NS], Ct[NS];
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        Bt[n] = sel_r[n0 + n];
        Ct[n] = sel_r[N + n0 + n];
      }
      const float x = xl[r * LD + cl];
      const TokenFront f = make_front(dl[r * LD + cl], bias, true);
      float y = token_step<NS>(cc, f, x, Bt, Ct, h[i]);
      if constexpr (LPC >= 2) y += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(y), 0xB1, 0xf, 0xf, false));
      if constexpr (LPC == 4) y += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(y), 0x4E, 0xf, 0xf, false));
      float* st = a.state + (slot * a.D + d) * N + n0;
      if constexpr (NS == 4) {
        const f32x4 v = {h[i][0], h[i][1], h[i][2], h[i][3]};
        __builtin_nontemporal_store(v, reinterpret_cast<f32x4*>(st));
      } else {
#pragma unroll
        for (int n = 0; n < NS; ++n) st[n] = h[i][n];
      }
      if (n0 == 0) zl[r * LD + cl] = epilogue(y, x, dskip, a.z != nullptr, zl[r * LD + cl]);
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < nrows * (CB / 4); e += kBlock) {
    const int r = e / (CB / 4), g = e % (CB / 4) * 4;
    const int64_t dg = d0 + g;
    if (dg >= a.D || place[r] < 0) continue;
    const float4 v = *reinterpret_cast<const float4*>(zl + r * LD + g);
    const float o[4] = {v.x, v.y, v.z, v.w};
    IO* out = static_cast<IO*>(a.out) + (b0 + r) * a.D + dg;
    if (a.D - dg >= 4) store_raw<IO, 4, true>(out, narrow<IO, 4>(o), 4);
    else store_raw<IO, 4, false>(out, narrow<IO, 4>(o), (int)(a.D - dg));
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
  constexpr int CB = kChannels;
  const size_t lds = (size_t)kRows * (p.ldx + 3 * (CB + kPad)) * sizeof(float);
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
