// embed.hip -- embedding lookup and its gradient (include/mamba_mi355x_lm.h).
//
// Both are bound by memory traffic.  The lookup reads each named row and writes
// one row per token.  The gradient sorts the token positions by id (stable, so
// that every sum has one order), adds the rows of each id within fixed spans of
// the sorted list, and joins the spans of ids that cross them.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "lm_internal.h"
#include "s6_device.h"

namespace s6 {
namespace {

// VEC consecutive elements of a row: 16 bytes where rows stay 16-byte aligned, else one element.
template <typename IO, int VEC>
struct Piece {
  float v[VEC];
  __device__ __forceinline__ void load(const IO* p) {
    if constexpr (VEC == 1) {
      v[0] = load_io(p, 0);
    } else if constexpr (sizeof(IO) == 4) {
      const float4 w = *reinterpret_cast<const float4*>(p);
      v[0] = w.x, v[1] = w.y, v[2] = w.z, v[3] = w.w;
    } else {
      const uint4 w = *reinterpret_cast<const uint4*>(p);
      v[0] = bf16_lo(w.x), v[1] = bf16_hi(w.x), v[2] = bf16_lo(w.y), v[3] = bf16_hi(w.y);
      v[4] = bf16_lo(w.z), v[5] = bf16_hi(w.z), v[6] = bf16_lo(w.w), v[7] = bf16_hi(w.w);
    }
  }
  __device__ __forceinline__ void store(IO* p) const {
    if constexpr (VEC == 1) {
      store_io(p, 0, v[0]);
    } else if constexpr (sizeof(IO) == 4) {
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      uint4 w;
      w.x = f32_to_bf16(v[0]) | (uint32_t)f32_to_bf16(v[1]) << 16;
      w.y = f32_to_bf16(v[2]) | (uint32_t)f32_to_bf16(v[3]) << 16;
      w.z = f32_to_bf16(v[4]) | (uint32_t)f32_to_bf16(v[5]) << 16;
      w.w = f32_to_bf16(v[6]) | (uint32_t)f32_to_bf16(v[7]) << 16;
      *reinterpret_cast<uint4*>(p) = w;
    }
  }
};

template <typename IO>
constexpr int kVec = 16 / sizeof(IO);

// Workgroups of a launch at most (a grid holds fewer than 2^32 threads); the rest is looped over.
constexpr int64_t kMaxBlocks = int64_t(1) << 22;

// ---------------------------------------------------------------- lookup

// 1 << lpr_log2 lanes walk one row.
template <typename IO, int VEC>
__global__ __launch_bounds__(256) void embed_fwd_kernel(const int64_t* ids, const IO* W, IO* out, int64_t n, int64_t V,
                                                        int64_t D, float scale, int lpr_log2) {
  const int lpr = 1 << lpr_log2;
  const int64_t rows = 256 >> lpr_log2;
  for (int64_t i = (int64_t)blockIdx.x * rows + (threadIdx.x >> lpr_log2); i < n; i += gridDim.x * rows) {
    const int64_t id = ids[i];
    const bool ok = id >= 0 && id < V;
    const IO* src = W + (ok ? id : 0) * D;
    IO* dst = out + i * D;
    const float none = id < 0 ? 0.0f : __uint_as_float(0x7fc00000u);
    for (int64_t c = (int64_t)(threadIdx.x & (lpr - 1)) * VEC; c < D; c += (int64_t)lpr * VEC) {
      Piece<IO, VEC> p;
      if (ok) p.load(src + c);
#pragma unroll
      for (int k = 0; k < VEC; ++k) p.v[k] = ok ? p.v[k] * scale : none;
      p.store(dst + c);
    }
  }
}

// ---------------------------------------------------------------- sort of positions by id

constexpr int kSortWaves = 4;
constexpr int kMaxDigits = 1024;
constexpr int kMaxTiles = 128;

struct SortArgs {
  const int64_t* ids;     // first pass
  const uint32_t* key_in;  // later passes
  const uint32_t* pos_in;
  uint32_t* key_out;
  uint32_t* pos_out;
  uint32_t* hist;          // (tiles, digits)
  int64_t n, V;
  int64_t tile;            // positions per workgroup, a multiple of 256
  int tiles, shift, bits, first;
};

// Sort key of an id: itself, or V (after every row of the table) for ids outside it.
__device__ __forceinline__ uint32_t sort_key(const SortArgs& s, int64_t i) {
  if (!s.first) return s.key_in[i];
  const int64_t id = s.ids[i];
  return id >= 0 && id < s.V ? (uint32_t)id : (uint32_t)s.V;
}

// Lanes of the wave that hold the same digit, among the active ones.
__device__ __forceinline__ uint64_t same_digit(uint32_t digit, int bits, bool active) {
  uint64_t m = __ballot(active);
  for (int b = 0; b < bits; ++b) {
    const uint64_t one = __ballot((digit >> b) & 1u);
    m &= ((digit >> b) & 1u) ? one : ~one;
  }
  return m;
}

__device__ __forceinline__ int lanes_below(uint64_t m) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
}

// Count of each digit per wave: cnt[wave * digits + digit].  A wave owns a contiguous
// run of the tile, taken 64 positions at a time.
__device__ __forceinline__ void count_digits(const SortArgs& s, int64_t base, int64_t end, int digits, uint32_t* cnt) {
  const int lane = threadIdx.x & 63;
  for (int64_t i0 = base; i0 < end; i0 += 64) {
    const int64_t i = i0 + lane;
    const bool act = i < end;
    const uint32_t digit = act ? (sort_key(s, i) >> s.shift) & (digits - 1) : 0;
    const uint64_t m = same_digit(digit, s.bits, act);
    if (act && lanes_below(m) == 0) cnt[digit] += (uint32_t)__popcll(m);
    __builtin_amdgcn_wave_barrier();  // the wave's LDS accesses stay in this order
  }
}

__global__ __launch_bounds__(64 * kSortWaves) void sort_hist_kernel(SortArgs s) {
  __shared__ uint32_t cnt[kSortWaves * kMaxDigits];
  const int digits = 1 << s.bits, wave = threadIdx.x >> 6;
  for (int i = threadIdx.x; i < kSortWaves * digits; i += blockDim.x) cnt[i] = 0;
  __syncthreads();
  const int64_t per = s.tile / kSortWaves, t0 = (int64_t)blockIdx.x * s.tile;
  const int64_t end = t0 + s.tile < s.n ? t0 + s.tile : s.n;
  const int64_t b = t0 + wave * per, e = b + per < end ? b + per : end;
  count_digits(s, b, e, digits, cnt + wave * digits);
  __syncthreads();
  for (int i = threadIdx.x; i < digits; i += blockDim.x) {
    uint32_t c = 0;
    for (int w = 0; w < kSortWaves; ++w) c += cnt[w * digits + i];
    s.hist[(size_t)blockIdx.x * digits + i] = c;
  }
}

// Exclusive prefix sum of x over the workgroup (all threads call).
__device__ __forceinline__ uint32_t block_exclusive(uint32_t x, uint32_t* wsum) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  uint32_t v = x;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t y = __shfl_up(v, o, 64);
    if (lane >= o) v += y;
  }
  if (lane == 63) wsum[wave] = v;
  __syncthreads();
  uint32_t base = 0;
  for (int w = 0; w < wave; ++w) base += wsum[w];
  __syncthreads();
  return base + v - x;
}

// Stable scatter of one tile: a position's place is the number of smaller digits
// everywhere, plus its digit's count in earlier tiles and earlier waves, plus its
// rank in its own wave.
__global__ __launch_bounds__(64 * kSortWaves) void sort_scatter_kernel(SortArgs s) {
  __shared__ uint32_t cnt[kSortWaves * kMaxDigits];
  __shared__ uint32_t wsum[kSortWaves];
  constexpr int kPer = kMaxDigits / (64 * kSortWaves);
  const int digits = 1 << s.bits, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int i = threadIdx.x; i < kSortWaves * digits; i += blockDim.x) cnt[i] = 0;
  __syncthreads();
  const int64_t per = s.tile / kSortWaves, t0 = (int64_t)blockIdx.x * s.tile;
  const int64_t end = t0 + s.tile < s.n ? t0 + s.tile : s.n;
  const int64_t b = t0 + wave * per, e = b + per < end ? b + per : end;
  count_digits(s, b, e, digits, cnt + wave * digits);
  __syncthreads();
  // thread t owns digits t * kPer ... (consecutive, so that the prefix over threads is the prefix over digits)
  const int own = digits > (int)blockDim.x ? digits / (int)blockDim.x : 1;
  uint32_t total[kPer], before[kPer], sum = 0;
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    total[k] = before[k] = 0;
    const int d = threadIdx.x * own + k;
    if (k < own && d < digits)
      for (int t = 0; t < s.tiles; ++t) {
        const uint32_t c = s.hist[(size_t)t * digits + d];
        if (t < (int)blockIdx.x) before[k] += c;
        total[k] += c;
      }
    sum += total[k];
  }
  uint32_t base = block_exclusive(sum, wsum);
#pragma unroll
  for (int k = 0; k < kPer; ++k) {
    const int d = threadIdx.x * own + k;
    if (k < own && d < digits) {
      uint32_t at = base + before[k];
      for (int w = 0; w < kSortWaves; ++w) {
        const uint32_t c = cnt[w * digits + d];
        cnt[w * digits + d] = at;
        at += c;
      }
    }
    base += total[k];
  }
  __syncthreads();
  uint32_t* mine = cnt + wave * digits;
  for (int64_t i0 = b; i0 < e; i0 += 64) {
    const int64_t i = i0 + lane;
    const bool act = i < e;
    const uint32_t key = act ? sort_key(s, i) : 0;
    const uint32_t digit = (key >> s.shift) & (digits - 1);
    const uint64_t m = same_digit(digit, s.bits, act);
    const int rank = lanes_below(m);
    const uint32_t at = act ? mine[digit] + rank : 0;
    if (act) {
      s.key_out[at] = key;
      s.pos_out[at] = s.first ? (uint32_t)i : s.pos_in[i];
    }
    __builtin_amdgcn_wave_barrier();
    if (act && rank == 0) mine[digit] += (uint32_t)__popcll(m);
    __builtin_amdgcn_wave_barrier();
  }
}

// ---------------------------------------------------------------- sums over the sorted rows

struct SumArgs {
  const uint32_t* key;
  const uint32_t* pos;
  float* part;  // (spans, 2, D): of the run that enters the span, of the run that leaves it
  int64_t n, V, D;
  int span;     // sorted positions per span
  int spans;
  float scale;
};

// One wave per (span, block of columns).  A run of equal ids inside the span is
// finished here; the part of a run that crosses an end of the span goes to `part`.
template <typename IO, int VEC>
__global__ __launch_bounds__(64) void span_sum_kernel(SumArgs s, const IO* dout, IO* dW) {
  const int j = blockIdx.y;
  const int64_t col = ((int64_t)blockIdx.x * 64 + threadIdx.x) * VEC;
  const bool act = col < s.D;
  const int64_t b = (int64_t)j * s.span;
  const int64_t e = b + s.span < s.n ? b + s.span : s.n;
  uint32_t key = s.key[b];
  bool entered = b > 0 && s.key[b - 1] == key;
  float acc[VEC] = {};
  for (int64_t i = b; i < e && key < (uint32_t)s.V; ++i) {
    const uint32_t next = i + 1 < s.n ? s.key[i + 1] : (uint32_t)s.V;
    Piece<IO, VEC> p;
    if (act) p.load(dout + (size_t)s.pos[i] * s.D + col);
#pragma unroll
    for (int k = 0; k < VEC; ++k) acc[k] += act ? p.v[k] : 0.0f;
    const bool ends = next != key;
    if (ends || i + 1 == e) {
      if (act) {
        if (ends && !entered) {
#pragma unroll
          for (int k = 0; k < VEC; ++k) p.v[k] = acc[k] * s.scale;
          p.store(dW + (size_t)key * s.D + col);
        } else {
          float* q = s.part + ((size_t)j * 2 + (entered ? 0 : 1)) * s.D + col;
#pragma unroll
          for (int k = 0; k < VEC; ++k) q[k] = acc[k];
        }
      }
#pragma unroll
      for (int k = 0; k < VEC; ++k) acc[k] = 0.0f;
      entered = false;
    }
    key = next;
  }
}

// One wave per (span, block of columns): finishes the run that starts in the span
// and leaves it, if there is one.
template <typename IO, int VEC>
__global__ __launch_bounds__(64) void span_join_kernel(SumArgs s, IO* dW) {
  const int j = blockIdx.y;
  const int64_t b = (int64_t)j * s.span, next = b + s.span;
  if (next >= s.n) return;
  const uint32_t key = s.key[next];
  if (key >= (uint32_t)s.V || s.key[next - 1] != key) return;
  if (s.key[b] == key && b > 0 && s.key[b - 1] == key) return;  // entered the span already
  const int64_t col = ((int64_t)blockIdx.x * 64 + threadIdx.x) * VEC;
  if (col >= s.D) return;
  float acc[VEC];
  const float* q = s.part + ((size_t)j * 2 + 1) * s.D + col;
#pragma unroll
  for (int k = 0; k < VEC; ++k) acc[k] = q[k];
  for (int m = j + 1; m < s.spans && s.key[(int64_t)m * s.span] == key; ++m) {
    q = s.part + (size_t)m * 2 * s.D + col;
#pragma unroll
    for (int k = 0; k < VEC; ++k) acc[k] += q[k];
  }
  Piece<IO, VEC> p;
#pragma unroll
  for (int k = 0; k < VEC; ++k) p.v[k] = acc[k] * s.scale;
  p.store(dW + (size_t)key * s.D + col);
}

__global__ __launch_bounds__(256) void zero_bytes_kernel(uint8_t* p, size_t n) {
  const size_t step = (size_t)gridDim.x * 256 * 16;
  for (size_t i = ((size_t)blockIdx.x * 256 + threadIdx.x) * 16; i < n; i += step) {
    if (i + 16 <= n) *reinterpret_cast<uint4*>(p + i) = make_uint4(0, 0, 0, 0);
    else
      for (size_t k = i; k < n; ++k) p[k] = 0;
  }
}

// ---------------------------------------------------------------- plan

struct BwdPlanE {
  int passes, bits, tiles, span, spans;
  int64_t tile;
  size_t off_key[2], off_pos[2], off_hist, off_part, bytes;
};

BwdPlanE plan_embed_bwd(int64_t n, int64_t V, int64_t D) {
  BwdPlanE p{};
  int width = 1;
  while ((int64_t(1) << width) <= V) ++width;  // keys 0 ... V
  p.passes = (width + 9) / 10;
  p.bits = (width + p.passes - 1) / p.passes;
  p.tile = 1024;
  while ((n + p.tile - 1) / p.tile > kMaxTiles) p.tile *= 2;
  p.tiles = (int)((n + p.tile - 1) / p.tile);
  p.span = 32;
  while ((n + p.span - 1) / p.span > 4096) p.span *= 2;
  p.spans = (int)((n + p.span - 1) / p.span);
  auto al = [](size_t v) { return (v + 255) / 256 * 256; };
  size_t at = 0;
  for (int k = 0; k < 2; ++k) {
    p.off_key[k] = at;
    at += al((size_t)n * 4);
    p.off_pos[k] = at;
    at += al((size_t)n * 4);
  }
  p.off_hist = at;
  at += al((size_t)p.tiles * ((size_t)1 << p.bits) * 4);
  p.off_part = at;
  at += al((size_t)p.spans * 2 * D * 4);
  p.bytes = n > 0 && V > 0 && D > 0 ? at : 0;
  return p;
}

template <typename IO>
hipError_t fwd(int64_t n, int64_t V, int64_t D, const int64_t* ids, const void* W, float scale, void* out,
               hipStream_t st) {
  const bool vec = D % kVec<IO> == 0;
  const int64_t pieces = vec ? D / kVec<IO> : D;
  int lg = 0;
  while (lg < 6 && (int64_t(1) << lg) < pieces) ++lg;
  const dim3 grid((unsigned)std::min<int64_t>((n + (256 >> lg) - 1) / (256 >> lg), kMaxBlocks));
  if (vec)
    hipLaunchKernelGGL((embed_fwd_kernel<IO, kVec<IO>>), grid, dim3(256), 0, st, ids, (const IO*)W, (IO*)out, n, V, D,
                       scale, lg);
  else
    hipLaunchKernelGGL((embed_fwd_kernel<IO, 1>), grid, dim3(256), 0, st, ids, (const IO*)W, (IO*)out, n, V, D, scale,
                       lg);
  return hipGetLastError();
}

template <typename IO, int VEC>
void sums(const SumArgs& s, const void* dout, void* dW, hipStream_t st) {
  const dim3 grid((unsigned)((s.D + 64 * VEC - 1) / (64 * VEC)), (unsigned)s.spans);
  hipLaunchKernelGGL((span_sum_kernel<IO, VEC>), grid, dim3(64), 0, st, s, (const IO*)dout, (IO*)dW);
  hipLaunchKernelGGL((span_join_kernel<IO, VEC>), grid, dim3(64), 0, st, s, (IO*)dW);
}

}  // namespace

hipError_t launch_embed_fwd(int64_t n, int64_t V, int64_t D, int io, const int64_t* ids, const void* W, float scale,
                            void* out, hipStream_t st) {
  return io == kIoBF16 ? fwd<uint16_t>(n, V, D, ids, W, scale, out, st) : fwd<float>(n, V, D, ids, W, scale, out, st);
}

size_t embed_bwd_ws_bytes(int64_t n, int64_t V, int64_t D, int) { return plan_embed_bwd(n, V, D).bytes; }

hipError_t launch_embed_bwd(int64_t n, int64_t V, int64_t D, int io, const int64_t* ids, const void* dout, float scale,
                            void* dW, void* ws, hipStream_t st) {
  const size_t bytes = (size_t)V * D * (io == kIoBF16 ? 2 : 4);
  hipLaunchKernelGGL(zero_bytes_kernel, dim3((unsigned)std::min<size_t>((bytes + 4095) / 4096, kMaxBlocks)),
                     dim3(256), 0, st, (uint8_t*)dW,
                     bytes);
  if (n == 0) return hipGetLastError();
  const BwdPlanE p = plan_embed_bwd(n, V, D);
  uint8_t* w = static_cast<uint8_t*>(ws);
  SortArgs s{};
  s.ids = ids;
  s.hist = reinterpret_cast<uint32_t*>(w + p.off_hist);
  s.n = n;
  s.V = V;
  s.tile = p.tile;
  s.tiles = p.tiles;
  s.bits = p.bits;
  for (int k = 0; k < p.passes; ++k) {
    s.first = k == 0;
    s.shift = k * p.bits;
    s.key_in = reinterpret_cast<uint32_t*>(w + p.off_key[(k + 1) & 1]);
    s.pos_in = reinterpret_cast<uint32_t*>(w + p.off_pos[(k + 1) & 1]);
    s.key_out = reinterpret_cast<uint32_t*>(w + p.off_key[k & 1]);
    s.pos_out = reinterpret_cast<uint32_t*>(w + p.off_pos[k & 1]);
    hipLaunchKernelGGL(sort_hist_kernel, dim3(p.tiles), dim3(64 * kSortWaves), 0, st, s);
    hipLaunchKernelGGL(sort_scatter_kernel, dim3(p.tiles), dim3(64 * kSortWaves), 0, st, s);
  }
  SumArgs a{s.key_out, s.pos_out, reinterpret_cast<float*>(w + p.off_part), n, V, D, p.span, p.spans, scale};
  if (io == kIoBF16) {
    if (D % 8 == 0) sums<uint16_t, 8>(a, dout, dW, st);
    else sums<uint16_t, 1>(a, dout, dW, st);
  } else {
    if (D % 4 == 0) sums<float, 4>(a, dout, dW, st);
    else sums<float, 1>(a, dout, dW, st);
  }
  return hipGetLastError();
}

}  // namespace s6
