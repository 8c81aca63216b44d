// conv.hip -- the short causal convolution in front of a scan, on gfx950.
//
// Per channel, with W taps (2 to 4) and age_t the number of tokens since the last reset (no reset so far:
// as many as there are taps):
//     c_t = bias + sum_{o = 0}^{W-1, o <= age_t} weight_{W-1-o} x_{t-o},   out_t = SiLU(c_t) or c_t,
// where x at negative t is the carried window.  Backward, with dc_t = dout_t SiLU'(c_t):
//     dx_t = sum_{o <= age_{t+o}} weight_{W-1-o} dc_{t+o},   dweight_{W-1-o} = sum dc_t x_{t-o},   dbias = sum dc_t.
//
// A few operations per element, so memory bounds it.  A thread owns four channels and walks a chunk
// of tokens with the taps in registers: every input is loaded once (and W - 1 rows again per chunk) in
// coalesced loads, a batch of tokens in flight ahead of the one that is computed.
#include <type_traits>

#include "layer_device.h"
#include "layer_internal.h"

namespace s6 {
namespace {

constexpr int kBlock = 256;
constexpr int V = 4;              // channels per thread
constexpr int kAhead = 8;         // tokens whose loads are in flight together
constexpr int64_t kFwdChunk = 64;  // tokens per thread, forward
constexpr int64_t kThreads = 256 * 8 * 64;  // threads that fill the chip

int64_t groups(int64_t D) { return (D + V - 1) / V; }

// Tokens per thread: as many as leave the chip filled, between 8 and `most` (a multiple of 8).
int64_t chunk_of(int64_t batch, int64_t L, int64_t D, int64_t most) {
  const double t = (double)batch * (double)L * (double)groups(D) / (double)kThreads;
  int64_t c = t >= (double)most ? most : (int64_t)t / 8 * 8;
  return c < 8 ? 8 : c;
}

struct Item {
  int64_t b, chunk;
  int64_t d0;  // first channel
  int nv;      // channels that exist from d0 on
  bool in;
};

// Work item of this thread: channel group fastest (coalesced), then chunk, then batch row.
__device__ __forceinline__ Item item_of(int64_t batch, int64_t nchunks, int64_t D) {
  const int64_t G = (D + V - 1) / V;
  const int64_t id = (int64_t)blockIdx.x * kBlock + threadIdx.x;
  int64_t g, c, ch, b;
  if (batch * nchunks * G < 0x7fffffff) {  // one 32-bit division is a tenth of a 64-bit one
    const uint32_t c32 = (uint32_t)id / (uint32_t)G;
    g = (uint32_t)id - c32 * (uint32_t)G;
    const uint32_t b32 = c32 / (uint32_t)nchunks;
    ch = c32 - b32 * (uint32_t)nchunks;
    b = b32;
  } else {
    c = id / G;
    g = id - c * G;
    b = c / nchunks;
    ch = c - b * nchunks;
  }
  Item it;
  it.b = b;
  it.chunk = ch;
  it.d0 = g * V;
  it.nv = D - it.d0 < V ? (int)(D - it.d0) : V;
  it.in = b < batch;
  return it;
}

// Tokens since the last reset as they stand behind token t - 1, at most W.
template <int W>
__device__ __forceinline__ int age_before(const uint8_t* reset, int64_t t) {
  int age = W;
#pragma unroll
  for (int o = W - 2; o >= 0; --o)
    if (t - 1 - o >= 0 && reset[t - 1 - o]) age = o;
  return age;
}

template <typename IO, int W, bool FULL>
__device__ __forceinline__ raw_t<IO, V> row_before(const ConvArgs& a, const Item& it, int64_t t) {
  // input row t < L; negative t: the carried window
  if (t >= 0) return load_raw<IO, V, FULL>(static_cast<const IO*>(a.x) + (it.b * a.L + t) * a.D + it.d0, it.nv);
  if (!a.window) return raw_t<IO, V>(0u);
  return load_raw<IO, V, FULL>(static_cast<const IO*>(a.window) + (it.b * (W - 1) + (t + W - 1)) * a.D + it.d0, it.nv);
}

template <typename IO, int W, bool FULL>
__device__ __forceinline__ void load_weights(const ConvArgs& a, const Item& it, float (&w)[W][V],
                                             float (&bias)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const bool in = FULL || i < it.nv;
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][i] = in ? a.weight[(it.d0 + i) * W + j] : 0.0f;
    bias[i] = in && a.bias ? a.bias[it.d0 + i] : 0.0f;
  }
}

// The last W - 1 inputs of the row, zero bits where a reset behind them cut them off.
template <typename IO, int W, bool FULL>
__device__ __forceinline__ void conv_tail(const ConvArgs& a, const Item& it, int64_t len) {
  const int age = a.reset ? age_before<W>(a.reset + it.b * a.L, len) : W;
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    const int back = W - 2 - j;  // tokens between the entry and the last token
    const raw_t<IO, V> v = back <= age ? row_before<IO, W, FULL>(a, it, len - 1 - back) : raw_t<IO, V>(0u);
    store_raw<IO, V, FULL>(static_cast<IO*>(a.last) + (it.b * (W - 1) + j) * a.D + it.d0, v, it.nv);
  }
}

template <typename IO, int W, bool RESET, bool FULL>
__device__ __forceinline__ void conv_chunk(const ConvArgs& a, const Item& it, int64_t t0, int64_t t1, int64_t len) {
  IO* out = static_cast<IO*>(a.out) + it.b * a.L * a.D + it.d0;
  const IO* x = static_cast<const IO*>(a.x) + it.b * a.L * a.D + it.d0;
  const int64_t e1 = t1 < len ? t1 : len;
  if (t0 < e1) {
    float w[W][V], bias[V];
    load_weights<IO, W, FULL>(a, it, w, bias);
    raw_t<IO, V> row[W - 1 + kAhead];  // the W - 1 rows before the batch, then the batch
#pragma unroll
    for (int j = 0; j < W - 1; ++j) row[j] = row_before<IO, W, FULL>(a, it, t0 - (W - 1) + j);
    int age = W;
    if constexpr (RESET) age = age_before<W>(a.reset + it.b * a.L, t0);
    raw_t<IO, V> next[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      next[u] = t0 + u < e1 ? load_raw<IO, V, FULL>(x + (t0 + u) * a.D, it.nv) : raw_t<IO, V>(0u);
    for (int64_t t = t0; t < e1; t += kAhead) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) row[W - 1 + u] = next[u];
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (t + kAhead + u < e1) next[u] = load_raw<IO, V, FULL>(x + (t + kAhead + u) * a.D, it.nv);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (t + u >= e1) break;
        if constexpr (RESET) age = a.reset[it.b * a.L + t + u] ? 0 : (age < W ? age + 1 : W);
        float c[V];
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] = bias[i];
#pragma unroll
        for (int o = W - 1; o >= 0; --o) {
          float v[V];
          widen<IO, V>(row[W - 1 + u - o], v);
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float s = __builtin_fmaf(w[W - 1 - o][i], v[i], c[i]);
            c[i] = !RESET || o <= age ? s : c[i];
          }
        }
        if (a.silu)
#pragma unroll
          for (int i = 0; i < V; ++i) c[i] = silu(c[i]);
        store_raw<IO, V, FULL>(out + (t + u) * a.D, narrow<IO, V>(c), it.nv);
      }
#pragma unroll
      for (int j = 0; j < W - 1; ++j) row[j] = row[kAhead + j];
    }
  }
  for (int64_t t = t0 > len ? t0 : len; t < t1; ++t) store_raw<IO, V, FULL>(out + t * a.D, raw_t<IO, V>(0u), it.nv);
}

template <typename IO, int W, bool RESET>
__global__ __launch_bounds__(kBlock) void conv_fwd_kernel(ConvArgs a, int64_t nchunks, int64_t chunk) {
  // one more item per (row, channel group) than there are chunks: the window carried on
  const Item it = item_of(a.batch, nchunks + 1, a.D);
  if (!it.in) return;
  int64_t len = a.L;
  if (a.lengths) {
    const int64_t l = a.lengths[it.b];
    len = l < 0 ? 0 : (l < a.L ? l : a.L);
  }
  const bool full = it.nv == V;
  if (it.chunk == nchunks) {
    if (!a.last) return;
    if (full) conv_tail<IO, W, true>(a, it, len);
    else conv_tail<IO, W, false>(a, it, len);
    return;
  }
  const int64_t t0 = it.chunk * chunk, t1 = t0 + chunk < a.L ? t0 + chunk : a.L;
  if (full) conv_chunk<IO, W, RESET, true>(a, it, t0, t1, len);
  else conv_chunk<IO, W, RESET, false>(a, it, t0, t1, len);
}

// ---------------------------------------------------------------- backward

// Part sums of dweight and dbias: (item row, W + 1, D), an item row per (batch row, chunk).
template <typename IO, int W, bool RESET, bool FULL>
__device__ __forceinline__ void conv_bwd_chunk(const ConvBwdArgs& a, const Item& it, int64_t t0, int64_t t1,
                                               float* part) {
  const ConvArgs& f = a.f;
  const int64_t L = f.L, D = f.D, base = it.b * L * D + it.d0;
  const IO* x = static_cast<const IO*>(f.x) + base;
  const IO* dout = static_cast<const IO*>(a.dout) + base;
  IO* dx = static_cast<IO*>(a.dx) + base;
  const raw_t<IO, V> zero(0u);
  float w[W][V], bias[V];
  load_weights<IO, W, FULL>(f, it, w, bias);
  float dw[W][V], db[V], acc[W][V];  // acc[o]: gradient so far at token t - o
  raw_t<IO, V> hist[W - 1];               // input rows t - (W - 1) .. t - 1
#pragma unroll
  for (int i = 0; i < V; ++i) {
    db[i] = 0.0f;
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j][i] = acc[j][i] = 0.0f;
  }
#pragma unroll
  for (int j = 0; j < W - 1; ++j) hist[j] = row_before<IO, W, FULL>(f, it, t0 - (W - 1) + j);
  int age = W;
  if constexpr (RESET) age = age_before<W>(f.reset + it.b * L, t0);
  // The W - 1 tokens behind the chunk still send gradients into it; behind the sequence there is
  // only what the carried window sends.
  const int64_t end = t1 + W - 1, live = end < L ? end : L;
  raw_t<IO, V> nx[kAhead], nd[kAhead];
#pragma unroll
  for (int u = 0; u < kAhead; ++u) {
    nx[u] = t0 + u < live ? load_raw<IO, V, FULL>(x + (t0 + u) * D, it.nv) : zero;
    nd[u] = t0 + u < live ? load_raw<IO, V, FULL>(dout + (t0 + u) * D, it.nv) : zero;
  }
  for (int64_t tb = t0; tb < end; tb += kAhead) {
    raw_t<IO, V> cx[kAhead], cd[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      cx[u] = nx[u];
      cd[u] = nd[u];
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (tb + kAhead + u < live) {
        nx[u] = load_raw<IO, V, FULL>(x + (tb + kAhead + u) * D, it.nv);
        nd[u] = load_raw<IO, V, FULL>(dout + (tb + kAhead + u) * D, it.nv);
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t t = tb + u;
      if (t >= end) break;
      if (t < live) {
        if constexpr (RESET) age = f.reset[it.b * L + t] ? 0 : (age < W ? age + 1 : W);
        float tap[W][V], g[V];  // tap[o]: input t - o
        widen<IO, V>(cx[u], tap[0]);
#pragma unroll
        for (int o = 1; o < W; ++o) widen<IO, V>(hist[W - 1 - o], tap[o]);
        widen<IO, V>(cd[u], g);
        if (f.silu) {
          float c[V];
#pragma unroll
          for (int i = 0; i < V; ++i) c[i] = bias[i];
#pragma unroll
          for (int o = W - 1; o >= 0; --o)
#pragma unroll
            for (int i = 0; i < V; ++i) {
              const float s = __builtin_fmaf(w[W - 1 - o][i], tap[o][i], c[i]);
              c[i] = !RESET || o <= age ? s : c[i];
            }
#pragma unroll
          for (int i = 0; i < V; ++i) g[i] *= silu_slope(c[i]);
        }
#pragma unroll
        for (int o = 0; o < W; ++o) {
          const bool on = !RESET || o <= age;
#pragma unroll
          for (int i = 0; i < V; ++i) {
            const float s = __builtin_fmaf(w[W - 1 - o][i], g[i], acc[o][i]);
            acc[o][i] = on ? s : acc[o][i];
          }
          if (t < t1) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
              const float s = __builtin_fmaf(g[i], tap[o][i], dw[W - 1 - o][i]);
              dw[W - 1 - o][i] = on ? s : dw[W - 1 - o][i];
            }
          }
        }
        if (t < t1)
#pragma unroll
          for (int i = 0; i < V; ++i) db[i] += g[i];
      }
      // token (or window entry) p = t - (W - 1) has all its gradients
      const int64_t p = t - (W - 1);
      if (t >= L && a.dlast && (!RESET || L - 1 - p <= age)) {
        float v[V];
        widen<IO, V>(load_raw<IO, V, FULL>(
                      static_cast<const IO*>(a.dlast) + (it.b * (W - 1) + (p - (L - (W - 1)))) * D + it.d0, it.nv), v);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[W - 1][i] += v[i];
      }
      if (p >= t0) store_raw<IO, V, FULL>(dx + p * D, narrow<IO, V>(acc[W - 1]), it.nv);
      else if (t0 == 0 && a.dwindow)
        store_raw<IO, V, FULL>(static_cast<IO*>(a.dwindow) + (it.b * (W - 1) + (p + W - 1)) * D + it.d0,
                            narrow<IO, V>(acc[W - 1]), it.nv);
#pragma unroll
      for (int o = W - 1; o > 0; --o)
#pragma unroll
        for (int i = 0; i < V; ++i) acc[o][i] = acc[o - 1][i];
#pragma unroll
      for (int i = 0; i < V; ++i) acc[0][i] = 0.0f;
#pragma unroll
      for (int j = 0; j + 1 < W - 1; ++j) hist[j] = hist[j + 1];
      hist[W - 2] = cx[u];
    }
  }
#pragma unroll
  for (int j = 0; j <= W; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (FULL || i < it.nv) part[(int64_t)j * D + it.d0 + i] = j < W ? dw[j < W ? j : 0][i] : db[i];
}

template <typename IO, int W, bool RESET>
__global__ __launch_bounds__(kBlock) void conv_bwd_kernel(ConvBwdArgs a, int64_t nchunks, int64_t chunk, float* part) {
  const Item it = item_of(a.f.batch, nchunks, a.f.D);
  if (!it.in) return;
  const int64_t t0 = it.chunk * chunk, t1 = t0 + chunk < a.f.L ? t0 + chunk : a.f.L;
  float* p = part + (it.b * nchunks + it.chunk) * (W + 1) * a.f.D;
  if (it.nv == V) conv_bwd_chunk<IO, W, RESET, true>(a, it, t0, t1, p);
  else conv_bwd_chunk<IO, W, RESET, false>(a, it, t0, t1, p);
}

// dweight and dbias: the part sums of a column (one of (W + 1) D).
__global__ __launch_bounds__(1024) void conv_sum_kernel(const float* part, int64_t rows, int64_t D, int W,
                                                        float* dweight, float* dbias) {
  const int64_t col = (int64_t)blockIdx.x * 32 + (threadIdx.x & 31), cols = (W + 1) * D;
  const float v = column_sum(part, rows, cols, col);
  if (threadIdx.x >= 32 || col >= cols) return;
  const int64_t j = col / D, d = col % D;
  if (j < W) dweight[d * W + j] = v;
  else if (dbias) dbias[d] = v;
}

// ---------------------------------------------------------------- one token

template <typename IO, int W, bool FULL>
__device__ __forceinline__ void conv_step(const ConvStepArgs& a, const Item& it, int64_t slot) {
  IO* win = static_cast<IO*>(a.window) + slot * (W - 1) * a.D + it.d0;
  raw_t<IO, V> row[W];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) row[j] = load_raw<IO, V, FULL>(win + j * a.D, it.nv);
  row[W - 1] = load_raw<IO, V, FULL>(static_cast<const IO*>(a.x) + it.b * a.D + it.d0, it.nv);
  float c[V];
#pragma unroll
  for (int i = 0; i < V; ++i) c[i] = a.bias && (FULL || i < it.nv) ? a.bias[it.d0 + i] : 0.0f;
#pragma unroll
  for (int j = 0; j < W; ++j) {
    float v[V];
    widen<IO, V>(row[j], v);
#pragma unroll
    for (int i = 0; i < V; ++i)
      c[i] = __builtin_fmaf(FULL || i < it.nv ? a.weight[(it.d0 + i) * W + j] : 0.0f, v[i], c[i]);
  }
  if (a.silu)
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = silu(c[i]);
  store_raw<IO, V, FULL>(static_cast<IO*>(a.out) + it.b * a.D + it.d0, narrow<IO, V>(c), it.nv);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) store_raw<IO, V, FULL>(win + j * a.D, row[j + 1], it.nv);
}

template <typename IO, int W>
__global__ __launch_bounds__(kBlock) void conv_step_kernel(ConvStepArgs a) {
  const Item it = item_of(a.batch, 1, a.D);
  if (!it.in) return;
  const int64_t slot = a.slots ? a.slots[it.b] : it.b;
  if (slot < 0 || slot >= a.nslots) return;
  if (it.nv == V) conv_step<IO, W, true>(a, it, slot);
  else conv_step<IO, W, false>(a, it, slot);
}

// ---------------------------------------------------------------- plans and launches

struct ConvPlan {
  int64_t chunk, nchunks;
};

ConvPlan plan_fwd(int64_t batch, int64_t L, int64_t D) {
  const int64_t c = chunk_of(batch, L, D, kFwdChunk);
  return {c, (L + c - 1) / c};
}

ConvPlan plan_conv_bwd(int64_t batch, int64_t L, int64_t D) {
  const int64_t c = chunk_of(batch, L, D, 128);
  const int64_t n = (L + c - 1) / c;
  return {c, n < 1 ? 1 : n};  // a sequence of no tokens still hands dlast_window on
}

unsigned blocks(int64_t batch, int64_t n, int64_t D) {
  return (unsigned)((batch * n * groups(D) + kBlock - 1) / kBlock);
}

template <typename IO, int W>
void fwd_w(const ConvArgs& a, const ConvPlan& p, unsigned grid, hipStream_t s) {
  if (a.reset) hipLaunchKernelGGL((conv_fwd_kernel<IO, W, true>), dim3(grid), dim3(kBlock), 0, s, a, p.nchunks, p.chunk);
  else hipLaunchKernelGGL((conv_fwd_kernel<IO, W, false>), dim3(grid), dim3(kBlock), 0, s, a, p.nchunks, p.chunk);
}

template <typename IO, int W>
void bwd_w(const ConvBwdArgs& a, const ConvPlan& p, unsigned grid, float* part, hipStream_t s) {
  if (a.f.reset)
    hipLaunchKernelGGL((conv_bwd_kernel<IO, W, true>), dim3(grid), dim3(kBlock), 0, s, a, p.nchunks, p.chunk, part);
  else
    hipLaunchKernelGGL((conv_bwd_kernel<IO, W, false>), dim3(grid), dim3(kBlock), 0, s, a, p.nchunks, p.chunk, part);
}

template <typename F>
hipError_t by_type_and_width(int io, int W, F f) {
  if (io == kIoBF16) {
    if (W == 2) f(uint16_t(0), std::integral_constant<int, 2>());
    else if (W == 3) f(uint16_t(0), std::integral_constant<int, 3>());
    else f(uint16_t(0), std::integral_constant<int, 4>());
  } else {
    if (W == 2) f(0.0f, std::integral_constant<int, 2>());
    else if (W == 3) f(0.0f, std::integral_constant<int, 3>());
    else f(0.0f, std::integral_constant<int, 4>());
  }
  return hipGetLastError();
}

}  // namespace

bool conv_fits(int64_t batch, int64_t L, int64_t D) {
  // a launch counts its threads in 32 bits; the forward has one item more per row than it has chunks
  const double g = (double)batch * (double)groups(D), most = 4294967296.0 - kBlock;
  return g * ((double)plan_fwd(batch, L, D).nchunks + 1.0) < most && g * (double)plan_conv_bwd(batch, L, D).nchunks < most;
}

hipError_t launch_conv_fwd(const ConvArgs& a, int io, hipStream_t s) {
  const ConvPlan p = plan_fwd(a.batch, a.L, a.D);
  const unsigned grid = blocks(a.batch, p.nchunks + 1, a.D);
  return by_type_and_width(io, a.W, [&](auto t, auto w) { fwd_w<decltype(t), decltype(w)::value>(a, p, grid, s); });
}

size_t conv_bwd_ws_bytes(int64_t batch, int64_t L, int64_t D, int64_t W) {
  return (size_t)batch * (size_t)plan_conv_bwd(batch, L, D).nchunks * (size_t)(W + 1) * (size_t)D * sizeof(float);
}

hipError_t launch_conv_bwd(const ConvBwdArgs& a, int io, void* workspace, hipStream_t s) {
  const ConvArgs& f = a.f;
  const ConvPlan p = plan_conv_bwd(f.batch, f.L, f.D);
  float* part = static_cast<float*>(workspace);
  if (f.batch > 0) {
    const unsigned grid = blocks(f.batch, p.nchunks, f.D);
    const hipError_t e = by_type_and_width(
        io, f.W, [&](auto t, auto w) { bwd_w<decltype(t), decltype(w)::value>(a, p, grid, part, s); });
    if (e != hipSuccess) return e;
  }
  const int64_t cols = (f.W + 1) * f.D;
  hipLaunchKernelGGL(conv_sum_kernel, dim3((unsigned)((cols + 31) / 32)), dim3(1024), 0, s, part, f.batch * p.nchunks,
                     f.D, f.W, a.dweight, a.dbias);
  return hipGetLastError();
}

hipError_t launch_conv_step(const ConvStepArgs& a, int io, hipStream_t s) {
  const unsigned grid = blocks(a.batch, 1, a.D);
  return by_type_and_width(io, a.W, [&](auto t, auto w) {
    using T = decltype(t);
    hipLaunchKernelGGL((conv_step_kernel<T, decltype(w)::value>), dim3(grid), dim3(kBlock), 0, s, a);
  });
}

}  // namespace s6
