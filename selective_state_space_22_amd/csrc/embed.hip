// embed.hip -- embedding lookup and its gradient (include/mamba_mi355x_lm.h).
//
// Both are bound by memory traffic: the gradient by its zeros (50000 x 2560 bf16 with 16384
// positions, 340 MB: 74 us a call, a copy of as much 59; 32000 x 768 fp32 with 777, 101 MB:
// 20 us and 18).  The lookup reads each named row and writes
// one row per token.  The gradient sorts the token positions by id (stable, so
// that every sum has one order), adds the rows of each id within fixed spans of
// the sorted list, and joins the spans of ids that cross them.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "gated_device.h"
#include "lm_internal.h"

namespace s6 {
namespace {

// VEC consecutive elements of a row as they lie in memory (16 bytes where rows stay 16-byte
// aligned, else one element: lookup and gradient of 16384 rows of 2559 bf16 take 37 and 105 us,
// of 2560 22 and 74), and as numbers.
template <typename IO, int VEC>
struct Raw {
  uint32_t w[VEC == 1 ? 1 : 4];
  __device__ __forceinline__ void load(const IO* p) {
    if constexpr (VEC == 1) {
      if constexpr (sizeof(IO) == 4) w[0] = __float_as_uint(*p);
      else w[0] = (uint32_t)*p << 16;
    } else {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    }
  }
  __device__ __forceinline__ float at(int k) const {
    if constexpr (VEC == 8) return k & 1 ? bf16_hi(w[k / 2]) : bf16_lo(w[k / 2]);
    else return __uint_as_float(w[k]);
  }
};

template <typename IO, int VEC>
__device__ __forceinline__ void store_piece(IO* p, const float (&v)[VEC]) {
  if constexpr (VEC == 1) store_io(p, 0, v[0]);
  else if constexpr (sizeof(IO) == 4) *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  else
    *reinterpret_cast<uint4*>(p) = make_uint4(f32x2_to_bf16(v[0], v[1]), f32x2_to_bf16(v[2], v[3]),
                                              f32x2_to_bf16(v[4], v[5]), f32x2_to_bf16(v[6], v[7]));
}

template <typename IO>
constexpr int kVec = 16 / sizeof(IO);

// Workgroups of a launch at most (a grid holds fewer than 2^32 threads); the rest is looped over.
constexpr int64_t kMaxBlocks = int64_t(1) << 22;

// ---------------------------------------------------------------- lookup

// 1 << lpr_log2 lanes walk one row, four pieces of it at a time.  Bound by memory: 16384 rows
// of 2560 bf16 out of 50000, 168 MB read (most of the repeats from the last-level cache) and
// written: 22 us.
template <typename IO, int VEC>
__global__ __launch_bounds__(256) void embed_fwd_kernel(const int64_t* ids, const IO* W, IO* out, int64_t n, int64_t V,
                                                        int64_t D, float scale, int lpr_log2) {
  const int lpr = 1 << lpr_log2;
  const int64_t rows = 256 >> lpr_log2;
  const int64_t c0 = (int64_t)(threadIdx.x & (lpr - 1)) * VEC, step = (int64_t)lpr * VEC;
  for (int64_t i = (int64_t)blockIdx.x * rows + (threadIdx.x >> lpr_log2); i < n; i += gridDim.x * rows) {
    const int64_t id = ids[i];
    const bool ok = id >= 0 && id < V;
    const IO* src = W + (ok ? id : 0) * D;
    IO* dst = out + i * D;
    const float none = id < 0 ? 0.0f : __uint_as_float(0x7fc00000u);
    for (int64_t c = c0; c < D; c += 4 * step) {
      Raw<IO, VEC> p[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (ok && c + j * step < D) p[j].load(src + c + j * step);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (c + j * step >= D) continue;
        float v[VEC];
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[k] = ok ? p[j].at(k) * scale : none;
        store_piece<IO, VEC>(dst + c + j * step, v);
      }
    }
  }
}

// ---------------------------------------------------------------- zeros
//
// The table's gradient is mostly rows that no id names.  The whole of it is set to zero by
// the launches that sort: a sort leaves the memory idle, so it costs no time of its own.

// Zeros beyond what the last-level cache (256 MB) holds beside the rows are streamed past
// it: left in it they are written back while the sums read (when it was chosen, 50000 x 2560 bf16,
// 257 MB: 73 us against 84 for the whole gradient; 32000 x 768 fp32, 98 MB: 26 us cached, 30 streamed).

struct Zeros {
  uint8_t* p;       // 16-byte aligned
  size_t from, to;  // bytes, `from` a multiple of 16
  bool stream;
};

constexpr size_t kStreamZeros = size_t(128) << 20;

constexpr size_t kZeroChunk = 65536;

// Part of `blocks` workgroups of the launch, a chunk at a time.
template <bool STREAM>
__device__ __forceinline__ void zero_chunks(const Zeros& z, int64_t block, int64_t blocks) {
  typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
  const u32x4 zero = {0, 0, 0, 0};
  for (size_t c = z.from + block * kZeroChunk; c < z.to; c += blocks * kZeroChunk) {
    const size_t end = c + kZeroChunk < z.to ? c + kZeroChunk : z.to;
    for (size_t i = c + threadIdx.x * 16; i < end; i += blockDim.x * 16) {
      u32x4* q = reinterpret_cast<u32x4*>(z.p + i);
      if (i + 16 > end) {
        for (size_t k = i; k < end; ++k) z.p[k] = 0;
      } else if (STREAM) {
        __builtin_nontemporal_store(zero, q);
      } else {
        *q = zero;
      }
    }
  }
}

__device__ __forceinline__ void write_zeros(const Zeros& z, int64_t block, int64_t blocks) {
  if (z.stream) zero_chunks<true>(z, block, blocks);
  else zero_chunks<false>(z, block, blocks);
}

__global__ __launch_bounds__(1024) void zeros_kernel(Zeros z) { write_zeros(z, blockIdx.x, gridDim.x); }

// ---------------------------------------------------------------- sort of positions by id
//
// A stable radix sort.  A position's place is the number of smaller digits everywhere, plus
// its digit's count in earlier tiles and earlier waves of its tile (a wave owns consecutive
// positions), plus its rank in its own wave.

constexpr int kSortWaves = 16;
constexpr int kSortThreads = 64 * kSortWaves;
constexpr int kMaxDigits = 1024;  // of the sort over several workgroups
constexpr int kMaxTiles = 128;
constexpr int kSmallRounds = 4;   // positions per thread of the sort in one workgroup
constexpr int64_t kSmallCount = kSmallRounds * kSortThreads;
constexpr int kSmallDigits = 512;

struct SortArgs {
  const int64_t* ids;      // first pass
  const uint32_t* key_in;  // later passes
  const uint32_t* pos_in;
  uint32_t* key_out;
  uint32_t* pos_out;
  uint32_t* hist;          // (tiles, digits)
  int64_t n, V;
  int64_t tile;            // positions per workgroup, a multiple of kSortThreads
  int tiles, shift, bits, first, passes;
};

// Sort key of an id: itself, or V (after every row of the table) for ids outside it.
__device__ __forceinline__ uint32_t id_key(const SortArgs& s, int64_t i) {
  const int64_t id = s.ids[i];
  return id >= 0 && id < s.V ? (uint32_t)id : (uint32_t)s.V;
}
__device__ __forceinline__ uint32_t sort_key(const SortArgs& s, int64_t i) { return s.first ? id_key(s, i) : s.key_in[i]; }

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

// Rank of the lane's digit among those that the wave has counted into cnt so far, itself
// not included; counts the wave's 64 digits.  The wave's LDS accesses stay in order.
__device__ __forceinline__ uint32_t count_digit(uint32_t digit, int bits, bool active, uint32_t* cnt) {
  const uint64_t m = same_digit(digit, bits, active);
  const int below = lanes_below(m);
  const uint32_t before = active ? cnt[digit] : 0;
  __builtin_amdgcn_wave_barrier();
  if (active && below == 0) cnt[digit] = before + (uint32_t)__popcll(m);
  __builtin_amdgcn_wave_barrier();
  return before + below;
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

// cnt[wave][digit] from counts to places: `base` is the place of the thread's digit in the
// first wave.
__device__ __forceinline__ void counts_to_places(uint32_t* cnt, int digits, int digit, uint32_t base) {
  for (int w = 0; w < kSortWaves; ++w) {
    const uint32_t c = cnt[w * digits + digit];
    cnt[w * digits + digit] = base;
    base += c;
  }
}

// The whole sort in the first workgroup, positions in registers and LDS; the others write zeros.
struct SmallSort {
  uint32_t key[kSmallCount];
  uint16_t pos[kSmallCount];
  uint32_t cnt[kSortWaves * kSmallDigits];
  uint32_t wsum[kSortWaves];
};

__global__ __launch_bounds__(kSortThreads) void sort_small_kernel(SortArgs s, Zeros z) {
  __shared__ SmallSort sm;
  if (blockIdx.x != 0) {
    write_zeros(z, blockIdx.x - 1, gridDim.x - 1);
    return;
  }
  const int digits = 1 << s.bits, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int rounds = (int)((s.n + kSortThreads - 1) / kSortThreads), at0 = wave * rounds * 64 + lane, n = (int)s.n;
  uint32_t key[kSmallRounds];
  uint32_t pos[kSmallRounds], rank[kSmallRounds];
#pragma unroll
  for (int r = 0; r < kSmallRounds; ++r)
    if (r < rounds) {
      const int i = at0 + 64 * r;
      key[r] = i < n ? id_key(s, i) : 0;
      pos[r] = i;
    }
  for (int pass = 0, shift = 0; pass < s.passes; ++pass, shift += s.bits) {
    for (int i = threadIdx.x; i < kSortWaves * digits; i += kSortThreads) sm.cnt[i] = 0;
    __syncthreads();
    uint32_t* mine = sm.cnt + wave * digits;
#pragma unroll
    for (int r = 0; r < kSmallRounds; ++r)
      if (r < rounds) rank[r] = count_digit((key[r] >> shift) & (digits - 1), s.bits, at0 + 64 * r < n, mine);
    __syncthreads();
    uint32_t total = 0;
    if ((int)threadIdx.x < digits)
      for (int w = 0; w < kSortWaves; ++w) total += sm.cnt[w * digits + threadIdx.x];
    const uint32_t base = block_exclusive(total, sm.wsum);
    if ((int)threadIdx.x < digits) counts_to_places(sm.cnt, digits, threadIdx.x, base);
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kSmallRounds; ++r)
      if (r < rounds && at0 + 64 * r < n) {
        const uint32_t to = mine[(key[r] >> shift) & (digits - 1)] + rank[r];
        sm.key[to] = key[r];
        sm.pos[to] = (uint16_t)pos[r];
      }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kSmallRounds; ++r)
      if (r < rounds && at0 + 64 * r < n) key[r] = sm.key[at0 + 64 * r], pos[r] = sm.pos[at0 + 64 * r];
    __syncthreads();
  }
#pragma unroll
  for (int r = 0; r < kSmallRounds; ++r)
    if (r < rounds && at0 + 64 * r < n) s.key_out[at0 + 64 * r] = key[r], s.pos_out[at0 + 64 * r] = pos[r];
}

// Over several workgroups: the digits' counts of each tile, then the scatter of each tile.
__global__ __launch_bounds__(kSortThreads) void sort_hist_kernel(SortArgs s, Zeros z) {
  __shared__ uint32_t cnt[kSortWaves * kMaxDigits];
  if ((int)blockIdx.x >= s.tiles) {
    write_zeros(z, blockIdx.x - s.tiles, gridDim.x - s.tiles);
    return;
  }
  const int digits = 1 << s.bits, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int i = threadIdx.x; i < kSortWaves * digits; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
  const int64_t per = s.tile / kSortWaves, t0 = (int64_t)blockIdx.x * s.tile;
  const int64_t end = t0 + s.tile < s.n ? t0 + s.tile : s.n;
  const int64_t b = t0 + wave * per, e = b + per < end ? b + per : end;
  for (int64_t i = b + lane; i < e + lane; i += 64) {
    const uint32_t key = i < e ? sort_key(s, i) : 0;
    count_digit((key >> s.shift) & (digits - 1), s.bits, i < e, cnt + wave * digits);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < digits; i += kSortThreads) {
    uint32_t c = 0;
    for (int w = 0; w < kSortWaves; ++w) c += cnt[w * digits + i];
    s.hist[(size_t)blockIdx.x * digits + i] = c;
  }
}

__global__ __launch_bounds__(kSortThreads) void sort_scatter_kernel(SortArgs s, Zeros z) {
  __shared__ uint32_t cnt[kSortWaves * kMaxDigits];
  __shared__ uint32_t wsum[kSortWaves];
  if ((int)blockIdx.x >= s.tiles) {
    write_zeros(z, blockIdx.x - s.tiles, gridDim.x - s.tiles);
    return;
  }
  const int digits = 1 << s.bits, wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int i = threadIdx.x; i < kSortWaves * digits; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
  const int64_t per = s.tile / kSortWaves, t0 = (int64_t)blockIdx.x * s.tile;
  const int64_t end = t0 + s.tile < s.n ? t0 + s.tile : s.n;
  const int64_t b = t0 + wave * per, e = b + per < end ? b + per : end;
  uint32_t* mine = cnt + wave * digits;
  for (int64_t i = b + lane; i < e + lane; i += 64) {
    const uint32_t key = i < e ? sort_key(s, i) : 0;
    count_digit((key >> s.shift) & (digits - 1), s.bits, i < e, mine);
  }
  uint32_t total = 0, before = 0;
  if ((int)threadIdx.x < digits) {
#pragma unroll 8
    for (int t = 0; t < s.tiles; ++t) {
      const uint32_t c = s.hist[(size_t)t * digits + threadIdx.x];
      before += t < (int)blockIdx.x ? c : 0;
      total += c;
    }
  }
  __syncthreads();
  const uint32_t base = block_exclusive(total, wsum) + before;
  if ((int)threadIdx.x < digits) counts_to_places(cnt, digits, threadIdx.x, base);
  __syncthreads();
  for (int64_t i = b + lane; i < e + lane; i += 64) {
    const bool act = i < e;
    const uint32_t key = act ? sort_key(s, i) : 0;
    const uint32_t at = count_digit((key >> s.shift) & (digits - 1), s.bits, act, mine);
    if (act) {
      s.key_out[at] = key;
      s.pos_out[at] = s.first ? (uint32_t)i : s.pos_in[i];
    }
  }
}

// ---------------------------------------------------------------- sums over the sorted rows

struct SumArgs {
  const uint32_t* key;
  const uint32_t* pos;
  float* part;  // (spans, 2, D): of the run that enters the span, of the run that leaves it
  int64_t n, V, D;
  int span;     // sorted positions per span, a multiple of kRowsAhead
  int spans;
  float scale;
};

constexpr int kRowsAhead = 8;   // rows in flight per wave

// Rows are gathered eight to a wave at a time, so that their latency is paid once in eight:
// 16384 rows of 2560 bf16, 84 MB, 22 us.
// One wave per (block of columns, span).  A run of equal ids inside the span is finished
// here; the part of a run that crosses an end of the span goes to `part`.
template <typename IO, int VEC>
__global__ __launch_bounds__(64) void span_sum_kernel(SumArgs s, const IO* dout, IO* dW) {
  const int j = blockIdx.y, lane = threadIdx.x;
  const int64_t col = ((int64_t)blockIdx.x * 64 + lane) * VEC;
  const bool act = col < s.D;
  const int64_t b = (int64_t)j * s.span;
  const int64_t e = b + s.span < s.n ? b + s.span : s.n;
  const uint32_t V = (uint32_t)s.V;
  bool entered = b > 0 && s.key[b - 1] == s.key[b];
  float acc[VEC] = {};
  for (int64_t i0 = b; i0 < e; i0 += kRowsAhead) {
    // lane l holds the key of position i0 + l and its row (V past the end: no run)
    const int64_t il = i0 + (lane & 15);
    const uint32_t lkey = il < s.n ? s.key[il] : V;
    const uint32_t lpos = il < s.n ? s.pos[il] : 0;
    Raw<IO, VEC> p[kRowsAhead];  // rows that do not count are read all the same: no branches
#pragma unroll
    for (int r = 0; r < kRowsAhead; ++r)
      p[r].load(dout + (size_t)(uint32_t)__builtin_amdgcn_readlane(lpos, r) * s.D + (act ? col : 0));
#pragma unroll
    for (int r = 0; r < kRowsAhead; ++r) {
      const uint32_t key = __builtin_amdgcn_readlane(lkey, r), next = __builtin_amdgcn_readlane(lkey, r + 1);
      if (key >= V || i0 + r >= e) return;  // what follows is outside the table, or the span
#pragma unroll
      for (int k = 0; k < VEC; ++k) acc[k] += p[r].at(k);
      const bool ends = next != key;
      if (ends || i0 + r + 1 == e) {
        if (act) {
          if (ends && !entered) {
            float o[VEC];
#pragma unroll
            for (int k = 0; k < VEC; ++k) o[k] = acc[k] * s.scale;
            store_piece<IO, VEC>(dW + (size_t)key * s.D + col, o);
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
    }
  }
}

// One wave per (block of columns, span): finishes the run that starts in the span and
// leaves it, if there is one.
template <typename IO, int VEC>
__global__ __launch_bounds__(64) void span_join_kernel(SumArgs s, IO* dW) {
  const int j = blockIdx.y;
  const int64_t b = (int64_t)j * s.span, next = b + s.span;
  if (next >= s.n) return;
  const uint32_t key = s.key[next];
  if (key >= (uint32_t)s.V || s.key[next - 1] != key) return;
  if (s.key[b] == key && b > 0 && s.key[b - 1] == key) return;  // entered the span already
  int last = j + 1;  // the last span of the run; 64 are looked at at a time
  while (true) {
    const int m = last + 1 + (int)threadIdx.x;
    const uint64_t in = __ballot(m < s.spans && s.key[(int64_t)m * s.span] == key);
    const int more = in == ~0ull ? 64 : __ffsll((unsigned long long)~in) - 1;
    last += more;
    if (more < 64) break;
  }
  const int64_t col = ((int64_t)blockIdx.x * 64 + threadIdx.x) * VEC;
  if (col >= s.D) return;
  float acc[VEC];
  const float* q = s.part + ((size_t)j * 2 + 1) * s.D + col;
#pragma unroll
  for (int k = 0; k < VEC; ++k) acc[k] = q[k];
  for (int m = j + 1; m <= last; m += 8) {
    float v[8][VEC];
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      q = s.part + (size_t)(m + r <= last ? m + r : last) * 2 * s.D + col;
#pragma unroll
      for (int k = 0; k < VEC; ++k) v[r][k] = q[k];
    }
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int k = 0; k < VEC; ++k) acc[k] += m + r <= last ? v[r][k] : 0.0f;
  }
  float o[VEC];
#pragma unroll
  for (int k = 0; k < VEC; ++k) o[k] = acc[k] * s.scale;
  store_piece<IO, VEC>(dW + (size_t)key * s.D + col, o);
}

// ---------------------------------------------------------------- plan

struct EmbedBwdPlan {
  int passes, bits, tiles, span, spans;
  int64_t tile;
  bool small;
  size_t off_key[2], off_pos[2], off_hist, off_part, bytes;
};

EmbedBwdPlan plan_embed_bwd(int64_t n, int64_t V, int64_t D, int io) {
  EmbedBwdPlan p{};
  int width = 1;
  while ((int64_t(1) << width) <= V) ++width;  // keys 0 ... V
  // One workgroup sorts up to 4096 positions in one launch; beyond, its 60 us for 16384 would
  // show beside the zeros' 34 (50000 x 2560 bf16: 114 us against 92 with several workgroups, when
  // it was chosen).
  p.small = n <= kSmallCount;
  const int most = p.small ? 9 : 10;
  p.passes = (width + most - 1) / most;
  p.bits = (width + p.passes - 1) / p.passes;
  p.tile = kSortThreads;
  while ((n + p.tile - 1) / p.tile > kMaxTiles) p.tile *= 2;
  p.tiles = (int)((n + p.tile - 1) / p.tile);
  // Short spans spread few rows over more waves (777 rows of 768 fp32: 20.6 us with spans of
  // 8, 26 with 32); with waves enough, long ones leave less to join (16384 rows of 2560 bf16:
  // 84 us with 32, 91 with 8; both when it was chosen).
  const int64_t vec = io == kIoBF16 ? (D % 8 == 0 ? 8 : 1) : (D % 4 == 0 ? 4 : 1), blocks = (D + 64 * vec - 1) / (64 * vec);
  p.span = kRowsAhead;
  while (p.span < 32 && n * blocks / p.span > 4096) p.span *= 2;
  while ((n + p.span - 1) / p.span > 32768) p.span *= 2;
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

// Workgroups that write zeros beside a sort.
unsigned zero_blocks(const Zeros& z) {
  return (unsigned)std::min<size_t>((z.to - z.from + kZeroChunk - 1) / kZeroChunk, 1 << 16);
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

size_t embed_bwd_ws_bytes(int64_t n, int64_t V, int64_t D, int io) { return plan_embed_bwd(n, V, D, io).bytes; }

hipError_t launch_embed_bwd(int64_t n, int64_t V, int64_t D, int io, const int64_t* ids, const void* dout, float scale,
                            void* dW, void* ws, hipStream_t st) {
  const size_t bytes = (size_t)V * D * (io == kIoBF16 ? 2 : 4);
  Zeros z{(uint8_t*)dW, 0, bytes, bytes > kStreamZeros};
  if (n == 0) {
    hipLaunchKernelGGL(zeros_kernel, dim3(zero_blocks(z)), dim3(1024), 0, st, z);
    return hipGetLastError();
  }
  const EmbedBwdPlan p = plan_embed_bwd(n, V, D, io);
  uint8_t* w = static_cast<uint8_t*>(ws);
  SortArgs s{};
  s.ids = ids;
  s.hist = reinterpret_cast<uint32_t*>(w + p.off_hist);
  s.n = n;
  s.V = V;
  s.tile = p.tile;
  s.tiles = p.tiles;
  s.bits = p.bits;
  s.passes = p.passes;
  s.key_out = reinterpret_cast<uint32_t*>(w + p.off_key[0]);
  s.pos_out = reinterpret_cast<uint32_t*>(w + p.off_pos[0]);
  if (p.small) {
    hipLaunchKernelGGL(sort_small_kernel, dim3(1 + zero_blocks(z)), dim3(kSortThreads), 0, st, s, z);
  } else {
    for (int k = 0; k < p.passes; ++k) {
      s.first = k == 0;
      s.shift = k * p.bits;
      s.key_in = reinterpret_cast<uint32_t*>(w + p.off_key[(k + 1) & 1]);
      s.pos_in = reinterpret_cast<uint32_t*>(w + p.off_pos[(k + 1) & 1]);
      s.key_out = reinterpret_cast<uint32_t*>(w + p.off_key[k & 1]);
      s.pos_out = reinterpret_cast<uint32_t*>(w + p.off_pos[k & 1]);
      for (int half = 0; half < 2; ++half) {
        const int part = 2 * k + half, parts = 2 * p.passes;
        z.from = bytes / 16 * part / parts * 16;
        z.to = part + 1 == parts ? bytes : bytes / 16 * (part + 1) / parts * 16;
        const dim3 grid(p.tiles + zero_blocks(z));
        if (half == 0) hipLaunchKernelGGL(sort_hist_kernel, grid, dim3(kSortThreads), 0, st, s, z);
        else hipLaunchKernelGGL(sort_scatter_kernel, grid, dim3(kSortThreads), 0, st, s, z);
      }
    }
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
