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
//   back   4 or 8 rows x a block of channels: the states' loads are issued first and travel while r W_dt^T is
//          formed on the matrix cores; then the update, four states per lane as in the decode step
// x_c, r, B, C and dt stay fp32 between: each bf16 matrix operand made of them is split into three bf16 parts
// (8 + 8 + 8 bits of the 24) whose products are added in fp32, so a token is as exact as in fp32 throughout.
// (An infinite x_c has no such parts: its row comes out NaN.)
//
// Measured, bf16, N = 16, R = 160, W = 4 (a streaming copy reaches 6.1 TB/s):
//   256 x 5120   front 13 us, join 5, back 39: 186 MB moved, 4.8 TB/s, vector operations 36% of the time; bound by
//                the states' traffic, the front by the latency of its one round of loads
//   1 x 5120     front 5.4 us, back 6.9: latency of three dependent rounds of loads
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
constexpr int kPad = 4;       // floats behind an LDS row

// K elements of one matrix step, and of each lane's share (lane l: row l % 16, share l / 16 of the step).
template <typename IO>
constexpr int kStep = sizeof(IO) == 2 ? 32 : 16;
template <typename IO>
constexpr int kShare = kStep<IO> / 4;

// The A operands of a tile's rows in LDS, split once for all waves: bf16 as three parts, fp32 as it is.  K
// elements to a row, and 16 bytes more: the 16 rows that a quarter wave reads lie on distinct banks.
template <typename IO>
struct Operands;
template <>
struct Operands<uint16_t> {
  static __host__ __device__ constexpr size_t bytes(int64_t rows, int64_t K) { return 3 * rows * (K + 8) * 2; }
  // Three bf16 values whose sum is f to 24 bits.
  static __device__ __forceinline__ void put(uint8_t* base, int rows, int K, int r, int k, float f) {
    uint16_t* p = reinterpret_cast<uint16_t*>(base) + r * (K + 8) + k;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const uint16_t h = f32_to_bf16(f);
      p[i * rows * (K + 8)] = h;
      f -= bf16_to_f32(h);  // exact: the rounding error of h
    }
  }
  static __device__ __forceinline__ void put4(uint8_t* base, int rows, int K, int r, int k, const float (&v)[4]) {
    uint16_t* p = reinterpret_cast<uint16_t*>(base) + r * (K + 8) + k;
    float f[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const raw_t<uint16_t, 4> h = narrow<uint16_t, 4>(f);
      *reinterpret_cast<raw_t<uint16_t, 4>*>(p + i * rows * (K + 8)) = h;
      float back[4];
      widen<uint16_t, 4>(h, back);
#pragma unroll
      for (int e = 0; e < 4; ++e) f[e] -= back[e];
    }
  }
  // c + (row's elements k0 + 8 q .. + 7 and those of the other shares) times b
  static __device__ __forceinline__ f32x4 times(const uint8_t* base, int rows, int K, int r, int k, raw_t<uint16_t, 8> b,
                                                f32x4 c) {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(base) + r * (K + 8) + k;
    const bf16x8 bb = __builtin_bit_cast(bf16x8, b);
#pragma unroll
    for (int i = 2; i >= 0; --i)
      c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(*reinterpret_cast<const bf16x8*>(p + i * rows * (K + 8)), bb, c, 0, 0, 0);
    return c;
  }
};
template <>
struct Operands<float> {
  static __host__ __device__ constexpr size_t bytes(int64_t rows, int64_t K) { return rows * (K + 4) * 4; }
  static __device__ __forceinline__ void put(uint8_t* base, int, int K, int r, int k, float f) {
    reinterpret_cast<float*>(base)[r * (K + 4) + k] = f;
  }
  static __device__ __forceinline__ void put4(uint8_t* base, int, int K, int r, int k, const float (&v)[4]) {
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(base) + r * (K + 4) + k) = make_float4(v[0], v[1], v[2], v[3]);
  }
  static __device__ __forceinline__ f32x4 times(const uint8_t* base, int, int K, int r, int k, raw_t<float, 4> b, f32x4 c) {
    const float4 f = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + r * (K + 4) + k);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(f.x, __uint_as_float(b[0]), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(f.y, __uint_as_float(b[1]), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(f.z, __uint_as_float(b[2]), c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x4f32(f.w, __uint_as_float(b[3]), c, 0, 0, 0);
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
  __shared__ __attribute__((aligned(16))) uint8_t xs[Operands<IO>::bytes(kRows, kSlice)];
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
    for (int i = 0; i < kItems; ++i) Operands<IO>::put4(xs, kRows, kSlice, r + i * (kBlock / (kSlice / 4)), g, c[i]);
  }
  __syncthreads();
  for (int t0 = w; t0 < ntiles; t0 += 4 * TW) {
    f32x4 acc[TW];
#pragma unroll
    for (int t = 0; t < TW; ++t) {
      acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < KS; ++k) acc[t] = Operands<IO>::times(xs, kRows, kSlice, r16, k * kStep<IO> + q * kShare<IO>, wb[t][k], acc[t]);
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

// Sum over the slices of one value, in their order, U loads in flight.
template <int U>
__device__ __forceinline__ float slice_sum(const float* p, int64_t stride, int slices) {
  float v = 0.0f;
  int s = 0;
  for (; s + U <= slices; s += U) {
    float q[U];
#pragma unroll
    for (int i = 0; i < U; ++i) q[i] = p[(s + i) * stride];
#pragma unroll
    for (int i = 0; i < U; ++i) v += q[i];
  }
  for (; s < slices; ++s) v += p[s * stride];
  return v;
}

// out: (batch, F), the slices' parts added in their order.
__global__ __launch_bounds__(kBlock) void ssm_join_kernel(const float* part, int64_t count, int slices, float* out) {
  const int64_t i = (int64_t)blockIdx.x * kBlock + threadIdx.x;
  if (i < count) out[i] = slice_sum<8>(part + i, count, slices);
}

constexpr int kChannels = 128;        // channels of a back workgroup
constexpr int kBack = 4 * kChannels;  // its threads: four lanes per channel at N = 16
// Up to these, the back adds the slices itself, once per workgroup, instead of a launch that does it for all (D 5120:
// 2 rows 11.9 us so, 14.1 with the launch; 4 rows 13.8, 15.4; a tile of 7 rows has 6 rows in 15.6, with the launch 16.1,
// but 1 to 4 rows 0.4 later).
constexpr int kFewRows = 4;
constexpr int kBackRows = 8;          // batch rows of its tile otherwise (at most the matrix instruction's 16)

template <int N, int ROWS>
struct Lanes {
  static constexpr int kStates = N < 4 ? N : 4;                    // states per lane
  static constexpr int kPer = N / kStates;                         // lanes per channel
  static constexpr int kGroups = kBack / (kChannels * kPer);      // row groups: a lane has every kGroups-th row
  static constexpr int kRowsPer = (ROWS + kGroups - 1) / kGroups;  // rows per lane
};

// sel: (slices, batch, F) part sums of r, B, C, or joined, one slice: always so with kBackRows.
template <typename IO, int N, int ROWS>
__global__ __launch_bounds__(kBack, ROWS == kFewRows ? 1 : 6) void ssm_back_kernel(SsmStepArgs a, int tiles, const float* xc,
                                                                                   const float* sel, int slices) {
  constexpr int NS = Lanes<N, ROWS>::kStates, LPC = Lanes<N, ROWS>::kPer, RG = Lanes<N, ROWS>::kGroups, RP = Lanes<N, ROWS>::kRowsPer;
  constexpr int CB = kChannels, LD = CB + kPad;
  // Matrix steps whose weights are loaded ahead.  With few rows that is latency saved; with many it is registers
  // that other waves need (256 x 5120: 45 us with six steps and two workgroups per CU, 39 with two and three).
  constexpr int PRE = ROWS == kFewRows ? 6 : 2;
  __shared__ int place[ROWS];
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int RK = (int)((a.R + kStep<IO> - 1) / kStep<IO> * kStep<IO>);
  uint8_t* rd = lds;                                                                    // r of the rows, as operands
  float* bc = reinterpret_cast<float*>(lds + Operands<IO>::bytes(ROWS, RK));  // (ROWS, 2 N): B, C
  float* dl = bc + ROWS * 2 * N;                                                   // (ROWS, LD): dt
  float* xl = dl + ROWS * LD;                                                      // (ROWS, LD): x_c
  float* yl = xl + ROWS * LD;                                                      // (ROWS, LD): C . h
  const int tile = blockIdx.x % (uint32_t)tiles;
  const int64_t d0 = (int64_t)(blockIdx.x / (uint32_t)tiles) * CB, b0 = (int64_t)tile * ROWS;
  const int nrows = a.batch - b0 < ROWS ? (int)(a.batch - b0) : ROWS;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, q = lane >> 4;
  const int64_t F = a.R + 2 * N;
  // this lane's channel, states and first row
  const int cl = threadIdx.x / LPC % CB, n0 = threadIdx.x % LPC * NS, rg = threadIdx.x / (LPC * CB);
  const int64_t d = d0 + cl;
  const bool in = d < a.D;
  if (threadIdx.x < ROWS) place[threadIdx.x] = (int)place_of(a, b0 + threadIdx.x);
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
    const int64_t slot = i * RG + rg < ROWS ? place_of(a, b0 + i * RG + rg) : -1;
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
  // r (zero behind R), B and C of the tile's rows: a wave per row, more where there are fewer rows
  {
    const int per = nrows == 1 ? kBack : (nrows == 2 ? kBack / 2 : (nrows <= 4 ? kBack / 4 : 64));
    const int cols = RK + 2 * N;
    for (int r = threadIdx.x / per; r < nrows; r += kBack / per)
      for (int c = threadIdx.x & (per - 1); c < cols; c += per) {
        const float* p = sel + (b0 + r) * F + (c < RK ? c : a.R + (c - RK));
        float v = 0.0f;
        if (c < a.R || c >= RK) v = ROWS == kFewRows ? slice_sum<20>(p, a.batch * F, slices) : *p;
        if (c >= RK) bc[r * 2 * N + (c - RK)] = v;
        else Operands<IO>::put(rd, ROWS, RK, r, c, v);
      }
  }
  const int er = threadIdx.x / (CB / 4), eg = threadIdx.x % (CB / 4) * 4;  // row and channels that this thread stages
  const int64_t ed = d0 + eg;
  const int env = a.D - ed < 4 ? (int)(a.D - ed) : 4;
#pragma unroll
  for (int i = 0; i < (ROWS * CB / 4 + kBack - 1) / kBack; ++i) {
    const int r = er + i * (kBack / (CB / 4));
    if (r >= nrows) break;
    const float* p = xc + (b0 + r) * a.D + ed;
    *reinterpret_cast<raw_t<float, 4>*>(xl + r * LD + eg) =
        env == 4 ? load_raw<float, 4, true>(p, 4) : load_raw<float, 4, false>(p, env);
  }
  const float bias = a.dt_bias && cw < a.D ? a.dt_bias[cw] : 0.0f;
  __syncthreads();
  {
    // rows that are not there repeat one that is: their products are not looked at
    const int r = r16 < nrows ? r16 : 0;
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int p = 0; p < PRE; ++p) {
      if (p * kStep<IO> >= RK) break;
      acc = Operands<IO>::times(rd, ROWS, RK, r, p * kStep<IO> + q * kShare<IO>, pre[p], acc);
    }
    for (int k = PRE * kStep<IO>; k < RK; k += kStep<IO>)
      acc = Operands<IO>::times(rd, ROWS, RK, r, k + q * kShare<IO>,
                                operand_b<IO>(wdt, k + q * kShare<IO>, a.R, cw < a.D), acc);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (4 * q + i < ROWS) dl[(4 * q + i) * LD + w * 16 + r16] = softplus(acc[i] + bias);
  }
  __syncthreads();
  if (in) {
    ChanConst<NS> cc;
#pragma unroll
    for (int n = 0; n < NS; ++n) cc.set(n, a.A[d * N + n0 + n]);
#pragma unroll
    for (int i = 0; i < RP; ++i) {
      const int r = i * RG + rg;
      const int64_t slot = r < ROWS ? place[r] : -1;
      if (slot < 0) continue;  // the channel's lanes agree
      const float* sel_r = bc + r * 2 * N;
      float Bt[NS], Ct[NS];
#pragma unroll
      for (int n = 0; n < NS; ++n) {
        Bt[n] = sel_r[n0 + n];
        Ct[n] = sel_r[N + n0 + n];
      }
      TokenFront f;
      f.dt = dl[r * LD + cl];
      f.dt2 = f.dt * f.dt;
      f.dth = 0.5f * f.dt;
      f.pos = true;
      float y = token_step<NS>(cc, f, xl[r * LD + cl], Bt, Ct, h[i]);
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
      if (n0 == 0) yl[r * LD + cl] = y;
    }
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < (ROWS * CB / 4 + kBack - 1) / kBack; ++i) {
    const int r = er + i * (kBack / (CB / 4));
    if (r >= nrows || env <= 0 || place[r] < 0) continue;
    const int64_t at = (b0 + r) * a.D + ed;
    raw_t<IO, 4> zr(0u);
    raw_t<float, 4> dr(0u);
    if (env == 4) {
      if (a.z) zr = load_raw<IO, 4, true>(static_cast<const IO*>(a.z) + at, 4);
      if (a.dskip) dr = load_raw<float, 4, true>(a.dskip + ed, 4);
    } else {
      if (a.z) zr = load_raw<IO, 4, false>(static_cast<const IO*>(a.z) + at, env);
      if (a.dskip) dr = load_raw<float, 4, false>(a.dskip + ed, env);
    }
    float z[4], ds[4], o[4];
    widen<IO, 4>(zr, z);
    widen<float, 4>(dr, ds);
#pragma unroll
    for (int k = 0; k < 4; ++k) o[k] = epilogue(yl[r * LD + eg + k], xl[r * LD + eg + k], ds[k], a.z != nullptr, z[k]);
    IO* out = static_cast<IO*>(a.out) + at;
    if (env == 4) store_raw<IO, 4, true>(out, narrow<IO, 4>(o), 4);
    else store_raw<IO, 4, false>(out, narrow<IO, 4>(o), env);
  }
}

struct StepPlan {
  int tiles, back_tiles, slices;
  bool join, few;
  size_t off_part, off_sel, bytes;
};

StepPlan plan_step(int64_t batch, int64_t D, int64_t N, int64_t R) {
  StepPlan p;
  const int64_t F = R + 2 * N;
  p.tiles = (int)((batch + kRows - 1) / kRows);
  p.slices = (int)((D + kSlice - 1) / kSlice);
  // every back workgroup adds its rows' parts again: cheaper than a launch while they are few
  p.join = batch > kFewRows;
  p.back_tiles = p.join ? (int)((batch + kBackRows - 1) / kBackRows) : 1;
  // Tiles of few rows also where each then has a compute unit of its own (D 5120: 8 rows 15.6 us so, 16.9 in the larger
  // tile; 16 rows 17.2, 18.7; beyond, 36 x 4768 28.9, 22.7).
  const int few_tiles = (int)((batch + kFewRows - 1) / kFewRows);
  p.few = !p.join || few_tiles * ((D + kChannels - 1) / kChannels) <= 256;
  if (p.few) p.back_tiles = few_tiles;
  auto al = [](size_t v) { return (v + 255) / 256 * 256; };
  p.off_part = al((size_t)batch * D * 4);
  p.off_sel = p.off_part + al((size_t)p.slices * batch * F * 4);
  p.bytes = p.off_sel + (p.join ? al((size_t)batch * F * 4) : 0);
  return p;
}

template <typename IO, int N, int ROWS>
hipError_t back(const SsmStepArgs& a, const StepPlan& p, const float* xc, const float* sel, int slices,
                hipStream_t s) {
  constexpr int CB = kChannels;
  const size_t lds = Operands<IO>::bytes(ROWS, (a.R + kStep<IO> - 1) / kStep<IO> * kStep<IO>) +
                     (size_t)ROWS * (2 * N + 3 * (CB + kPad)) * sizeof(float);
  hipLaunchKernelGGL((ssm_back_kernel<IO, N, ROWS>), dim3((unsigned)(p.back_tiles * ((a.D + CB - 1) / CB))), dim3(kBack), lds, s,
                     a, p.back_tiles, xc, sel, slices);
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
  auto go = [&](auto n) {
    constexpr int N = decltype(n)::value;
    return p.few ? back<IO, N, kFewRows>(a, p, xc, sel, slices, s) : back<IO, N, kBackRows>(a, p, xc, sel, slices, s);
  };
  switch (a.N) {
    case 1: return go(std::integral_constant<int, 1>());
    case 2: return go(std::integral_constant<int, 2>());
    case 4: return go(std::integral_constant<int, 4>());
    case 8: return go(std::integral_constant<int, 8>());
    case 16: return go(std::integral_constant<int, 16>());
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

size_t ssm_step_ws_bytes(int64_t batch, int64_t D, int64_t N, int64_t R) {
  return plan_step(batch, D, N, R).bytes;
}

hipError_t launch_ssm_step(const SsmStepArgs& a, int io, void* workspace, hipStream_t s) {
  const StepPlan p = plan_step(a.batch, a.D, a.N, a.R);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  return io == kIoBF16 ? launch_t<uint16_t>(a, p, ws, s) : launch_t<float>(a, p, ws, s);
}

}  // namespace s6
