// conv.hip -- the short causal convolution in front of a scan, on gfx950.
//
// Per channel, with W taps (2 to 4) and age_t the number of tokens since the last reset (no reset so far:
// as many as there are taps):
//     c_t = bias + sum_{o = 0}^{W-1, o <= age_t} weight_{W-1-o} x_{t-o},   out_t = SiLU(c_t) or c_t,
// where x at negative t is the carried window.  Backward, with dc_t = dout_t SiLU'(c_t):
//     dx_t = sum_{o <= age_{t+o}} weight_{W-1-o} dc_{t+o},   dweight_{W-1-o} = sum dc_t x_{t-o},   dbias = sum dc_t.
//
// A thread owns two channels and walks a chunk of tokens with the taps in registers: every input is loaded
// once (and W - 1 rows again per chunk) in coalesced loads, the next tile of four tokens in flight while one is
// computed.  Chunks are as short as a count of threads allows (kThreads): a token needs what its neighbours load, but
// no order among chunks.  Measured (a streaming copy reaches 6.1 TB/s; bytes as the formulas need them):
//   forward 4 x 4096 x 5120 bf16, rows three quarters full   49 us, 294 MB: 6.0 TB/s; bound by memory (60 a call
//                                          where the inputs change from call to call)
//   forward 8 x 2048 x 1536 bf16, resets   26 us, 101 MB: 3.9 TB/s; 22 vector operations an element, half of the time
//   gradients of the same                  41 us, 151 MB: 3.7 TB/s; 40 vector operations an element, 61% of the time
//   3 x 1537 x 1101 fp32                   12 us, 41 MB: 3.4 TB/s; gradients 14 us, 61 MB: 4.4 TB/s.  These read 53 MB
//                                          where the formulas need 41: with three taps a chunk (here 16 tokens) reads
//                                          four rows of x and two of dout beside its own, 19%; the other 10% have
//                                          not been explained
//   sum over the chunks' parts             4 to 5 us, a launch and its latency
//   one token 256 x 5120 bf16              6 us, 21 MB: 3.5 TB/s; latency of one round of loads
#include <type_traits>

#include "layer_device.h"
#include "layer_internal.h"

namespace s6 {
namespace {

constexpr int kBlock = 256;
// Tokens of a tile: its loads are in flight together while the tile before it is computed.
constexpr int kTile = 4;
constexpr int kTileBwd = 4;
// Channels per thread (two, four: forward 4 x 4096 x 5120 bf16 68, 69 us and fp32 137, 138; forward and gradients
// 8 x 2048 x 1536 bf16 65, 72 and fp32 106, 118; step 256 x 5120 bf16 5.3, 5.6 and fp32 8.3, 8.1).
constexpr int kGroup = 2;
constexpr int64_t kLeastFwd = 8, kMostFwd = 32, kLeastBwd = 8, kMostBwd = 128;  // tokens per thread
// Threads that a launch is split into where the sequences are long enough: three waves per SIMD, fewer than the
// registers of either kernel let run at once (forward 50 to 77: 6 to 8 waves; gradients 76 to 138: 3 to 6), since
// every chunk reads its neighbours' tokens again.  2, 3, 4, 6 waves: forward and gradients 8 x 2048 x 1536 bf16 69.5, 66,
// 68, 70 us and 3 x 1537 x 1101 fp32 30.5, 29, 31, 31.5; the latter's forward alone 12.1, 11.5, 11.1, 10.3.
constexpr int64_t kThreads = 256 * 12 * 64;

int64_t groups(int64_t D) { return (D + kGroup - 1) / kGroup; }

// Tokens per thread, between `least` and `most`: the fewest with which there are no more than kThreads threads, so that
// no few of them are left for a second round.
int64_t chunk_of(int64_t batch, int64_t L, int64_t D, int64_t least, int64_t most) {
  const int64_t rows = batch * groups(D);  // threads per chunk of the sequence
  const int64_t n = rows < kThreads ? kThreads / (rows < 1 ? 1 : rows) : 1;
  const int64_t c = ((L + n - 1) / n + 3) / 4 * 4;
  return c < least ? least : (c < most ? c : most);
}

struct Item {
  int64_t b, chunk;
  int64_t d0;  // first channel
  int nv;      // channels that exist from d0 on
  bool in;
};

// Work item of this thread: channel group fastest (coalesced), then chunk, then batch row.  WHOLE: the last group
// of a row that V does not divide begins earlier and shares channels with the one before, which gives them the same
// values: a group of fewer channels would hold up the waves it falls into (3 x 1537 x 1101 bf16, forward
// and gradients: 37 us, so 24).
template <int V, bool WHOLE>
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
  it.d0 = WHOLE && g * V + V > D ? D - V : g * V;
  it.nv = D - it.d0 < V ? (int)(D - it.d0) : V;
  it.in = b < batch;
  return it;
}

// Reset marks as bits: bit k of the marks at token t is the mark of token t - k.  Token t sees the input o
// tokens back if none of its marks 0 .. o - 1 is set.
__device__ __forceinline__ bool sees(uint32_t marks, int o) { return (marks & ((1u << o) - 1u)) == 0u; }

// The marks at token t - 1, as far back as they matter.
template <int W>
__device__ __forceinline__ uint32_t marks_before(const uint8_t* reset, int64_t t) {
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < W - 1; ++k)
    if (t - 1 - k >= 0 && reset[t - 1 - k]) m |= 1u << k;
  return m;
}

// The reset bytes of tokens t .. t + T - 1 of a row that ends at `to`, the first token's lowest.  They stay raw
// until their tile is computed: looking at them earlier would wait for the loads around them.
template <int T>
using bytes_t = std::conditional_t<T == 4, uint32_t, uint64_t>;
template <int T>
__device__ __forceinline__ bytes_t<T> reset_bytes(const uint8_t* reset, int64_t t, int64_t to) {
  static_assert(T == 4 || T == 8, "bytes of a word");
  bytes_t<T> m = 0;
  if (t + T <= to) {
    __builtin_memcpy(&m, reset + t, T);
  } else {
#pragma unroll
    for (int u = 0; u < T; ++u)
      if (t + u < to) m |= (bytes_t<T>)reset[t + u] << (8 * u);
  }
  return m;
}
// As marks, the first token highest.
template <int T>
__device__ __forceinline__ uint32_t marks_of(bytes_t<T> bytes) {
  uint32_t m = 0;
#pragma unroll
  for (int u = 0; u < T; ++u)
    if (bytes & ((bytes_t<T>)0xff << (8 * u))) m |= 1u << (T - 1 - u);
  return m;
}

template <typename IO, int V, int W, bool FULL>
__device__ __forceinline__ raw_t<IO, V> row_before(const ConvArgs& a, const Item& it, int64_t t) {
  // input row t < L; negative t: the carried window
  if (t >= 0) return load_raw<IO, V, FULL>(static_cast<const IO*>(a.x) + (it.b * a.L + t) * a.D + it.d0, it.nv);
  if (!a.window) return raw_t<IO, V>(0u);
  return load_raw<IO, V, FULL>(static_cast<const IO*>(a.window) + (it.b * (W - 1) + (t + W - 1)) * a.D + it.d0, it.nv);
}

// Weights by tap, and the bias, of the item's channels.
template <int V, int W, bool FULL>
__device__ __forceinline__ void load_weights(const float* weight, const float* bias, int64_t d0, int nv,
                                             float (&w)[W][V], float (&b)[V]) {
  float q[W][V];  // the V W weights side by side
#pragma unroll
  for (int k = 0; k < W; ++k) widen<float, V>(load_raw<float, V, FULL>(weight + d0 * W + k * V, nv * W - k * V), q[k]);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    b[i] = 0.0f;
#pragma unroll
    for (int j = 0; j < W; ++j) w[j][i] = q[(i * W + j) / V][(i * W + j) % V];
  }
  if (bias) widen<float, V>(load_raw<float, V, FULL>(bias + d0, nv), b);
}

// c_t of one token: x[-o] is the input o tokens back; CUT: of these only what its marks let it see.
template <int V, int W, bool CUT>
__device__ __forceinline__ void conv_sum(const float (&w)[W][V], const float (&bias)[V], const float (*x)[V],
                                         uint32_t marks, float (&c)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) c[i] = bias[i];
#pragma unroll
  for (int o = W - 1; o >= 0; --o) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float s = __builtin_fmaf(w[W - 1 - o][i], x[-o][i], c[i]);
      c[i] = !CUT || sees(marks, o) ? s : c[i];
    }
  }
}

// The last W - 1 inputs of the row, zero bits where a reset behind them cut them off.
template <typename IO, int V, int W, bool FULL>
__device__ __forceinline__ void conv_tail(const ConvArgs& a, const Item& it, int64_t len) {
  const uint32_t marks = a.reset ? marks_before<W>(a.reset + it.b * a.L, len) : 0u;
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    const int back = W - 2 - j;  // tokens between the entry and the last token
    const raw_t<IO, V> v = sees(marks, back) ? row_before<IO, V, W, FULL>(a, it, len - 1 - back) : raw_t<IO, V>(0u);
    store_raw<IO, V, FULL>(static_cast<IO*>(a.last) + (it.b * (W - 1) + j) * a.D + it.d0, v, it.nv);
  }
}

template <typename IO, int V, int W, bool ACT, bool RESET, bool FULL>
__device__ __forceinline__ void conv_chunk(const ConvArgs& a, const Item& it, int64_t t0, int64_t t1, int64_t len) {
  constexpr int T = kTile;
  const int64_t D = a.D;
  IO* out = static_cast<IO*>(a.out) + (it.b * a.L + t0) * D + it.d0;
  const IO* x = static_cast<const IO*>(a.x) + (it.b * a.L + t0) * D + it.d0;
  const uint8_t* reset = RESET ? a.reset + it.b * a.L + t0 : nullptr;
  const int n = chunk_tokens(t0, t1, len);
  if (n > 0) {
    float w[W][V], bias[V], row[W - 1 + T][V];  // row: the W - 1 inputs before the tile, then the tile
    load_weights<V, W, FULL>(a.weight, a.bias, it.d0, it.nv, w, bias);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) widen<IO, V>(row_before<IO, V, W, FULL>(a, it, t0 - (W - 1) + j), row[j]);
    uint32_t marks = RESET ? marks_before<W>(a.reset + it.b * a.L, t0) : 0u;
    raw_t<IO, V> next[T];
    bytes_t<T> nr = 0;  // the tile's reset bytes
    auto load = [&](int t) {
      if (t + T <= n) {
#pragma unroll
        for (int u = 0; u < T; ++u) next[u] = load_raw<IO, V, FULL>(x + u * D, it.nv);
      } else {
#pragma unroll
        for (int u = 0; u < T; ++u) {
          next[u] = raw_t<IO, V>(0u);
          if (t + u < n) next[u] = load_raw<IO, V, FULL>(x + u * D, it.nv);
        }
      }
      if (RESET) nr = reset_bytes<T>(reset, t, n);
    };
    load(0);
    for (int t = 0; t < n; t += T) {
#pragma unroll
      for (int u = 0; u < T; ++u) widen<IO, V>(next[u], row[W - 1 + u]);
      const bool cut = RESET && (nr != 0 || !sees(marks, W - 2));
      marks = (marks << T) | (RESET ? marks_of<T>(nr) : 0u);
      x += T * D;
      load(t + T);
      auto token = [&](int u, auto masked) {
        float c[V];
        conv_sum<V, W, decltype(masked)::value>(w, bias, &row[W - 1 + u], marks >> (T - 1 - u), c);
        if constexpr (ACT)
#pragma unroll
          for (int i = 0; i < V; ++i) c[i] = silu(c[i]);
        if (t + u < n) store_raw<IO, V, FULL>(out + u * D, narrow<IO, V>(c), it.nv);
      };
      // few tiles hold a reset or the tokens behind one: only those mask their taps
      if (RESET && __any(cut)) {
#pragma unroll
        for (int u = 0; u < T; ++u) token(u, std::true_type());
      } else {
#pragma unroll
        for (int u = 0; u < T; ++u) token(u, std::false_type());
      }
      out += T * D;
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int i = 0; i < V; ++i) row[j][i] = row[T + j][i];
    }
  }
  IO* behind = static_cast<IO*>(a.out) + it.b * a.L * D + it.d0;
  for (int64_t t = t0 > len ? t0 : len; t < t1; ++t) store_raw<IO, V, FULL>(behind + t * D, raw_t<IO, V>(0u), it.nv);
}

// FULL: rows of at least V channels.
template <typename IO, int V, int W, bool ACT, bool RESET, bool FULL>
__global__ __launch_bounds__(kBlock) void conv_fwd_kernel(ConvArgs a, int64_t nchunks, int64_t chunk) {
  // one more item per (row, channel group) than there are chunks: the window carried on
  const Item it = item_of<V, FULL>(a.batch, nchunks + 1, a.D);
  if (!it.in) return;
  int64_t len = a.L;
  if (a.lengths) {
    const int64_t l = a.lengths[it.b];
    len = l < 0 ? 0 : (l < a.L ? l : a.L);
  }
  if (it.chunk == nchunks) {
    if (a.last) conv_tail<IO, V, W, FULL>(a, it, len);
    return;
  }
  const int64_t t0 = it.chunk * chunk, t1 = t0 + chunk < a.L ? t0 + chunk : a.L;
  conv_chunk<IO, V, W, ACT, RESET, FULL>(a, it, t0, t1, len);
}

// ---------------------------------------------------------------- backward

// Part sums of dweight and dbias: (item row, W + 1, D), an item row per (batch row, chunk).  An item adds the
// sums of its tokens [t0, t1) and writes dx of the tokens that these complete, [t0 - (W - 1), t1 - (W - 1)),
// and the last of a row up to the sequence's end; the dc of the W - 1 tokens before t0 is formed again.
// Whole tiles that no reset cuts take the unrolled path, anything else goes token by token.
template <typename IO, int V, int W, bool ACT, bool RESET, bool FULL>
__device__ __forceinline__ void conv_bwd_chunk(const ConvBwdArgs& a, const Item& it, int64_t t0, int64_t t1,
                                               float* part) {
  constexpr int T = kTileBwd, H = W - 1;
  const ConvArgs& f = a.f;
  const int64_t D = f.D, base = it.b * f.L * D + it.d0;
  const IO* x = static_cast<const IO*>(f.x) + base;
  const IO* dout = static_cast<const IO*>(a.dout) + base;
  IO* dx = static_cast<IO*>(a.dx) + base;
  const uint8_t* reset = RESET ? f.reset + it.b * f.L : nullptr;
  float w[W][V], bias[V], dw[W][V], db[V];
  load_weights<V, W, FULL>(f.weight, f.bias, it.d0, it.nv, w, bias);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    db[i] = 0.0f;
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j][i] = 0.0f;
  }
  float row[H + T][V], g[H + T][V];  // inputs and dc of the W - 1 tokens before the tile, then the tile
  const int64_t first = t0 < H ? 0 : t0 - H;
#pragma unroll
  for (int j = 0; j < H; ++j) {
    widen<IO, V>(row_before<IO, V, W, FULL>(f, it, first - H + j), row[j]);
#pragma unroll
    for (int i = 0; i < V; ++i) g[j][i] = 0.0f;
  }
  uint32_t marks = RESET ? marks_before<W>(reset, first) : 0u;

  raw_t<IO, V> nx[T], nd[T];  // the next tokens' inputs and dout
  bytes_t<T> nr = 0;            // their reset bytes
  auto load = [&](int64_t t, int64_t to) {
    if (t + T <= to) {
#pragma unroll
      for (int u = 0; u < T; ++u) {
        nx[u] = load_raw<IO, V, FULL>(x + (t + u) * D, it.nv);
        nd[u] = load_raw<IO, V, FULL>(dout + (t + u) * D, it.nv);
      }
    } else {
#pragma unroll
      for (int u = 0; u < T; ++u) {
        nx[u] = nd[u] = raw_t<IO, V>(0u);
        if (t + u < to) {
          nx[u] = load_raw<IO, V, FULL>(x + (t + u) * D, it.nv);
          nd[u] = load_raw<IO, V, FULL>(dout + (t + u) * D, it.nv);
        }
      }
    }
    if (RESET) nr = reset_bytes<T>(reset, t, to);
  };
  // One token, whatever it is: before the chunk (only its dc counts), in it, or behind the sequence (only
  // what leaves).
  auto single = [&](int64_t t, raw_t<IO, V> rx, raw_t<IO, V> rd, bool mark) {
    widen<IO, V>(rx, row[H]);
    widen<IO, V>(rd, g[H]);
    marks = (marks << 1) | (RESET && mark ? 1u : 0u);
    if (t < t1) {
      if constexpr (ACT) {
        float c[V];
        conv_sum<V, W, RESET>(w, bias, &row[H], marks, c);
#pragma unroll
        for (int i = 0; i < V; ++i) g[H][i] *= silu_slope(c[i]);
      }
      if (t >= t0) {
#pragma unroll
        for (int o = 0; o < W; ++o)
          if (!RESET || sees(marks, o))
#pragma unroll
            for (int i = 0; i < V; ++i) dw[H - o][i] = __builtin_fmaf(g[H][i], row[H - o][i], dw[H - o][i]);
#pragma unroll
        for (int i = 0; i < V; ++i) db[i] += g[H][i];
      }
    }
    if (t >= t0) {
      // the token (or window entry) p = t - (W - 1) has all its gradients: token p + o sees p if none of
      // the marks of tokens p + 1 .. p + o is set
      const int64_t p = t - H;
      float acc[V];
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] = 0.0f;
#pragma unroll
      for (int o = 0; o < W; ++o)
        if (!RESET || sees(marks >> (H - o), o))
#pragma unroll
          for (int i = 0; i < V; ++i) acc[i] = __builtin_fmaf(w[H - o][i], g[o][i], acc[i]);
      if (t >= f.L && a.dlast && (!RESET || sees(marks, H))) {
        float v[V];
        widen<IO, V>(load_raw<IO, V, FULL>(static_cast<const IO*>(a.dlast) + (it.b * H + (t - f.L)) * D + it.d0, it.nv), v);
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] += v[i];
      }
      if (p >= 0) store_raw<IO, V, FULL>(dx + p * D, narrow<IO, V>(acc), it.nv);
      else if (a.dwindow)
        store_raw<IO, V, FULL>(static_cast<IO*>(a.dwindow) + (it.b * H + (p + H)) * D + it.d0, narrow<IO, V>(acc), it.nv);
    }
#pragma unroll
    for (int j = 0; j < H; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        row[j][i] = row[j + 1][i];
        g[j][i] = g[j + 1][i];
      }
  };

  // the first of those in flight
  auto pop = [&](int64_t t) {
    single(t, nx[0], nd[0], (nr & 0xffu) != 0);
    nr >>= 8;
#pragma unroll
    for (int u = 0; u + 1 < T; ++u) {
      nx[u] = nx[u + 1];
      nd[u] = nd[u + 1];
    }
  };
  {
    // a chunk that is not the first has the W - 1 tokens before it
    raw_t<IO, V> px[H], pd[H];
    uint32_t pm = 0;
#pragma unroll
    for (int u = 0; u < H; ++u) {
      px[u] = pd[u] = raw_t<IO, V>(0u);
      if (first + u < t0) {
        px[u] = load_raw<IO, V, FULL>(x + (first + u) * D, it.nv);
        pd[u] = load_raw<IO, V, FULL>(dout + (first + u) * D, it.nv);
        if (RESET) pm |= (uint32_t)reset[first + u] << (8 * u);
      }
    }
    load(t0, t1);
#pragma unroll 1
    for (int64_t t = first; t < t0; ++t) {
      single(t, px[0], pd[0], (pm & 0xffu) != 0);
      pm >>= 8;
#pragma unroll
      for (int u = 0; u + 1 < H; ++u) {
        px[u] = px[u + 1];
        pd[u] = pd[u + 1];
      }
    }
  }
  int64_t t = t0;
  for (; t + T <= t1; t += T) {
    if (__any(t < H || (RESET && (nr != 0 || !sees(marks, W - 2))))) {
#pragma unroll 1
      for (int u = 0; u < T; ++u) pop(t + u);
      load(t + T, t1);
      continue;
    }
#pragma unroll
    for (int u = 0; u < T; ++u) {
      widen<IO, V>(nx[u], row[H + u]);
      widen<IO, V>(nd[u], g[H + u]);
    }
    marks <<= T;
    load(t + T, t1);
#pragma unroll
    for (int u = 0; u < T; ++u) {
      if constexpr (ACT) {
        float c[V];
        conv_sum<V, W, false>(w, bias, &row[H + u], 0u, c);
#pragma unroll
        for (int i = 0; i < V; ++i) g[H + u][i] *= silu_slope(c[i]);
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        db[i] += g[H + u][i];
#pragma unroll
        for (int o = 0; o < W; ++o) dw[H - o][i] = __builtin_fmaf(g[H + u][i], row[H + u - o][i], dw[H - o][i]);
      }
    }
#pragma unroll
    for (int u = 0; u < T; ++u) {
      float acc[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        acc[i] = 0.0f;
#pragma unroll
        for (int o = 0; o < W; ++o) acc[i] = __builtin_fmaf(w[H - o][i], g[u + o][i], acc[i]);
      }
      store_raw<IO, V, FULL>(dx + (t + u - H) * D, narrow<IO, V>(acc), it.nv);
    }
#pragma unroll
    for (int j = 0; j < H; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        row[j][i] = row[T + j][i];
        g[j][i] = g[T + j][i];
      }
  }
  const int64_t end = t1 < f.L ? t1 : f.L + H;
#pragma unroll 1
  for (; t < end; ++t) pop(t);  // what is behind t1 was loaded as zeros and no marks
#pragma unroll
  for (int j = 0; j <= W; ++j)
    store_raw<float, V, FULL>(part + j * D + it.d0, narrow<float, V>(j < W ? dw[j < W ? j : 0] : db), it.nv);
}

template <typename IO, int V, int W, bool ACT, bool RESET, bool FULL>
__global__ __launch_bounds__(kBlock) void conv_bwd_kernel(ConvBwdArgs a, int64_t nchunks, int64_t chunk,
                                                             float* part) {
  const Item it = item_of<V, FULL>(a.f.batch, nchunks, a.f.D);
  if (!it.in) return;
  const int64_t t0 = it.chunk * chunk, t1 = t0 + chunk < a.f.L ? t0 + chunk : a.f.L;
  float* p = part + (it.b * nchunks + it.chunk) * (W + 1) * a.f.D;
  conv_bwd_chunk<IO, V, W, ACT, RESET, FULL>(a, it, t0, t1, p);
}

// dweight and dbias: the part sums of a column (one of (W + 1) D).
template <int C>
__global__ __launch_bounds__(1024) void conv_sum_kernel(const float* part, int64_t rows, int64_t D, int W,
                                                        float* dweight, float* dbias) {
  const int64_t col = (int64_t)blockIdx.x * C + threadIdx.x % C, cols = (W + 1) * D;
  const float v = column_sum<C>(part, rows, cols, col);
  if (threadIdx.x >= C || col >= cols) return;
  const int64_t j = col / D, d = col % D;
  if (j < W) dweight[d * W + j] = v;
  else if (dbias) dbias[d] = v;
}

// ---------------------------------------------------------------- one token

template <typename IO, int V, int W, bool FULL>
__device__ __forceinline__ void conv_step(const ConvStepArgs& a, const Item& it, int64_t slot) {
  IO* win = static_cast<IO*>(a.window) + slot * (W - 1) * a.D + it.d0;
  raw_t<IO, V> row[W];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) row[j] = load_raw<IO, V, FULL>(win + j * a.D, it.nv);
  row[W - 1] = load_raw<IO, V, FULL>(static_cast<const IO*>(a.x) + it.b * a.D + it.d0, it.nv);
  float w[W][V], bias[V], v[W][V], c[V];
  load_weights<V, W, FULL>(a.weight, a.bias, it.d0, it.nv, w, bias);
#pragma unroll
  for (int j = 0; j < W; ++j) widen<IO, V>(row[j], v[j]);
  conv_sum<V, W, false>(w, bias, &v[W - 1], 0u, c);
  if (a.silu)
#pragma unroll
    for (int i = 0; i < V; ++i) c[i] = silu(c[i]);
  store_raw<IO, V, FULL>(static_cast<IO*>(a.out) + it.b * a.D + it.d0, narrow<IO, V>(c), it.nv);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) store_raw<IO, V, FULL>(win + j * a.D, row[j + 1], it.nv);
}

template <typename IO, int V, int W>
__global__ __launch_bounds__(kBlock) void conv_step_kernel(ConvStepArgs a) {
  const Item it = item_of<V, false>(a.batch, 1, a.D);
  if (!it.in) return;
  const int64_t slot = a.slots ? a.slots[it.b] : it.b;
  if (slot < 0 || slot >= a.nslots) return;
  if (it.nv == V) conv_step<IO, V, W, true>(a, it, slot);
  else conv_step<IO, V, W, false>(a, it, slot);
}

// ---------------------------------------------------------------- plans and launches

struct ConvPlan {
  int64_t chunk, nchunks;
};

ConvPlan plan_fwd(int64_t batch, int64_t L, int64_t D) {
  const int64_t c = chunk_of(batch, L, D, kLeastFwd, kMostFwd);
  return {c, (L + c - 1) / c};
}

ConvPlan plan_conv_bwd(int64_t batch, int64_t L, int64_t D) {
  const int64_t c = chunk_of(batch, L, D, kLeastBwd, kMostBwd);
  const int64_t n = (L + c - 1) / c;
  return {c, n < 1 ? 1 : n};
}

unsigned blocks(int64_t batch, int64_t n, int64_t D) {
  return (unsigned)((batch * n * groups(D) + kBlock - 1) / kBlock);
}

template <typename F>
void by_flags(bool act, bool reset, bool full, F f) {
  using Yes = std::true_type;
  using No = std::false_type;
  if (!full) {  // rows of fewer channels than a thread has
    if (act) reset ? f(Yes(), Yes(), No()) : f(Yes(), No(), No());
    else reset ? f(No(), Yes(), No()) : f(No(), No(), No());
  } else {
    if (act) reset ? f(Yes(), Yes(), Yes()) : f(Yes(), No(), Yes());
    else reset ? f(No(), Yes(), Yes()) : f(No(), No(), Yes());
  }
}

template <typename IO, int W>
void fwd_w(const ConvArgs& a, const ConvPlan& p, unsigned grid, hipStream_t s) {
  constexpr int V = kGroup;
  by_flags(a.silu, a.reset, a.D >= V, [&](auto act, auto reset, auto full) {
    hipLaunchKernelGGL((conv_fwd_kernel<IO, V, W, decltype(act)::value, decltype(reset)::value, decltype(full)::value>),
                       dim3(grid), dim3(kBlock), 0, s, a, p.nchunks, p.chunk);
  });
}

template <typename IO, int W>
void bwd_w(const ConvBwdArgs& a, const ConvPlan& p, unsigned grid, float* part, hipStream_t s) {
  constexpr int V = kGroup;
  by_flags(a.f.silu, a.f.reset, a.f.D >= V, [&](auto act, auto reset, auto full) {
    hipLaunchKernelGGL((conv_bwd_kernel<IO, V, W, decltype(act)::value, decltype(reset)::value, decltype(full)::value>),
                       dim3(grid), dim3(kBlock), 0, s, a, p.nchunks, p.chunk, part);
  });
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
  // A launch counts its threads in 32 bits.  A thread has two channels, and fewer than 32 tokens only where
  // that makes no more than kThreads of them; the forward has one item more per row than it has chunks.
  return (double)batch * (double)groups(D) * (double)((L + 31) / 32 + 1) < 2147483648.0;
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
  const int64_t rows = f.L > 0 ? f.batch * p.nchunks : 0;  // of part sums
  if (f.L == 0) {
    // no tokens: what the forward did was to hand the window on, and so does dlast_window go; no weight is read
    if (f.batch > 0 && a.dwindow) {
      ConvArgs copy{};
      copy.window = a.dlast;
      copy.last = a.dwindow;
      copy.batch = f.batch;
      copy.D = f.D;
      copy.W = f.W;
      const hipError_t e = launch_conv_fwd(copy, io, s);
      if (e != hipSuccess) return e;
    }
  } else if (f.batch > 0) {
    const unsigned grid = blocks(f.batch, p.nchunks, f.D);
    const hipError_t e = by_type_and_width(
        io, f.W, [&](auto t, auto w) { bwd_w<decltype(t), decltype(w)::value>(a, p, grid, part, s); });
    if (e != hipSuccess) return e;
  }
  const int64_t cols = (f.W + 1) * f.D;
  by_columns(cols, [&](auto c) {
    constexpr int C = decltype(c)::value;
    hipLaunchKernelGGL((conv_sum_kernel<C>), dim3((unsigned)((cols + C - 1) / C)), dim3(1024), 0, s, part, rows,
                       f.D, f.W, a.dweight, a.dbias);
  });
  return hipGetLastError();
}

hipError_t launch_conv_step(const ConvStepArgs& a, int io, hipStream_t s) {
  const unsigned grid = blocks(a.batch, 1, a.D);
  return by_type_and_width(io, a.W, [&](auto t, auto w) {
    using T = decltype(t);
    hipLaunchKernelGGL((conv_step_kernel<T, kGroup, decltype(w)::value>), dim3(grid), dim3(kBlock), 0, s, a);
  });
}

}  // namespace s6
