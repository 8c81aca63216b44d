// sample.hip -- drawing a token per row of logits (include/mamba_mi355x_lm.h).
//
// One workgroup per row.  The filters keep a prefix of the row in falling order (equal
// logits: lower index first), so nothing has to be sorted: it is enough to find where the
// prefix ends.  A histogram over (m - x) / T, 64 bins to a unit, brackets the end; what
// lies above the bracket stays, and the few elements inside are listed in LDS and searched
// for the exact end by radix selection over (key, index), by counts (top_k) or by masses
// (top_p).  Rows that do not fit this (lists longer than LDS, logits spread over more than
// 32 units, temperatures near the end of fp32's range) take a radix selection over the whole row.
//
// Two or three passes: the largest logit, the bracket (top_p alone: in the same pass), the
// scores; what LDS holds of the row (114 KB) is read from memory once.  256 rows of 128000 fp32
// with top_p, a row to a compute unit, 131 MB of logits and up to as much noise: 71 us (40 up
// to the bracket, 20 for the scores, 10 for the exact end; a copy of logits and noise would
// take 46).  One row of 50000 bf16, all filters: 18 us, nearly all of it latency (passes 8,
// list 4, search and end 6); 64 rows of 50001 without filters 17, some 18 vector instructions
// to an element on 64 of the 256 compute units.  A list of more than kList elements costs a row's
// whole search: 64 rows of 50001 bf16 with a top_k of 50, 600 and 3000 take 19, 31 and 120 us.
//
// Masses that are added by atomics are integers (w 2^s, s = 62 - log2 of the row length),
// so that no sum depends on an order.
#include <hip/hip_runtime.h>

#include "lm_internal.h"
#include "s6_device.h"

namespace s6 {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr uint32_t kMasked = 0x007fffffu;  // key of -inf; NaN takes it too
constexpr int kBins = 2048;
constexpr float kBinsPerUnit = 64.0f;
// Bins above the reference of a histogram made before the maximum is known.  The reference is a
// logit of the row itself: no bin ends at it, where rounding would decide its bin.
constexpr float kAbove = 512.5f;
// Distances m - x end at kFarthest: those of masked logits, NaN and what lies past the row's end,
// which only a limit below it keeps out.  All limits are at most 90 units of the temperature, or
// kBins + 2 bins of it; below kLeastToBin bins to a logit (a temperature above 6.4e31) these could
// reach kFarthest, and the row takes the selection over the whole of it.
constexpr float kFarthest = 3.0e38f;
constexpr float kLeastToBin = 1.0e-30f;
static_assert((90.0f * kBinsPerUnit) / kLeastToBin < 1.0e-3f * kFarthest &&
                  (kBins + 2) / kLeastToBin < 1.0e-3f * kFarthest,
              "no limit comes near the farthest distance");
constexpr int kList = 2048;        // elements that the exact search holds
constexpr int kFew = 256;          // elements that it ranks in one go
constexpr int kCacheVecs = 7168;   // 16-byte pieces of the row kept in LDS
constexpr int kMaximaTopK = 512;   // top_k up to which the threads' maxima bracket the end

// Order-preserving key: larger logit, larger key; -0 and +0 are equal.
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  const uint32_t k = (b & 0x80000000u) ? ~b : b | 0x80000000u;
  return x != x ? kMasked : k;
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key ^ 0x80000000u : ~key);
}

// e^t to about an ulp for t <= 0: the product t log2(e) in two parts, the low one
// applied to first order.  Below -87 the result is 0 (such a weight never matters).
__device__ __forceinline__ float exp_accurate(float t) {
  constexpr float kLog2eLo = 1.925962991e-8f;  // log2(e) - float(log2(e))
  const float hi = t * kLog2e;
  const float lo = __builtin_fmaf(t, kLog2e, -hi) + t * kLog2eLo;
  const float r = ex2(hi);
  return t < -87.0f ? 0.0f : __builtin_fmaf(r, lo * kLn2, r);
}

struct Three {
  double a, b;
  unsigned long long c;
};

struct Shared {
  uint4 cache[kCacheVecs];
  uint32_t hist[kBins];
  unsigned long long list[kList];
  unsigned long long mass[256];
  uint32_t count[256];
  Three three[kWaves];
  unsigned long long sum[kWaves];
  uint32_t word[kWaves];
  float score[kWaves];
  unsigned long long before, found;
  uint32_t digit, listed, bound;
  int bin, cut_index;
};

// One row's logits, the first of them in LDS, and the weights relative to the largest.
template <typename IO>
struct Row {
  static constexpr int VEC = 16 / sizeof(IO);
  const IO* x;
  const uint4* vecs;  // the row's 16-byte aligned pieces
  const uint4* cache;
  int V, head, nvec, cached;
  uint32_t mkey;  // key of the largest logit
  float m, temperature, to_bin;
  float unit;     // masses are round(w * unit)
  int ibits;      // bits of an index

  __device__ __forceinline__ void set(const IO* row, int v) {
    x = row;
    V = v;
    const int off = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(IO));
    head = off ? (VEC - off < v ? VEC - off : v) : 0;
    nvec = (v - head) / VEC;
    vecs = reinterpret_cast<const uint4*>(row + head);
  }
  __device__ __forceinline__ float at(int i) const { return load_io(x, i); }
  __device__ __forceinline__ uint32_t key(int i) const { return key_of(at(i)); }
  static __device__ __forceinline__ float element(const uint4& v, int e) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (VEC == 8) return e & 1 ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
    else return __uint_as_float(w[e]);
  }
  // The thread's pieces of a batch of N times the workgroup's, from piece `base` on; -inf past
  // the last.
  template <int N>
  __device__ __forceinline__ void fetch(uint4 (&v)[N], int base) const {
    constexpr uint32_t kNone = VEC == 8 ? 0xff80ff80u : 0xff800000u;
#pragma unroll
    for (int q = 0; q < N; ++q) {
      const int first = base + q * kThreads, j = first + (int)threadIdx.x;
      v[q] = make_uint4(kNone, kNone, kNone, kNone);
      if (first < cached) {  // (a multiple of the workgroup, or the whole row)
        if (j < nvec) v[q] = cache[j];
      } else if (j < nvec) v[q] = vecs[j];
    }
  }
  // f(pieces, base, prefetch) for batch after batch of kElems elements to a thread; f calls
  // prefetch() behind its own loads.  The loops are rolled: a short row takes a few batches in
  // each pass, and fetching long code costs more than running it.  Eight elements, of what it cost
  // when they were chosen: 256 rows of 128000 f32, top_p, 83 us, with four 90, with sixteen 115
  // (registers spill); 64 rows of 50001 bf16 19.5 us, with sixteen 22.9.
  static constexpr int kElems = 8, kBatch = kElems / VEC;
  template <typename F>
  __device__ __forceinline__ void batches(F f) const {
    uint4 next[kBatch];
    fetch(next, 0);
#pragma unroll 1
    for (int base = 0; base < nvec; base += kBatch * kThreads) {
      uint4 v[kBatch];
#pragma unroll
      for (int q = 0; q < kBatch; ++q) v[q] = next[q];
      f(v, base, [&] { fetch(next, base + kBatch * kThreads); });
    }
  }
  // Index of element c of a batch.
  __device__ __forceinline__ int index(int base, int c) const {
    return head + (base + (int)threadIdx.x + c / VEC * kThreads) * VEC + c % VEC;
  }
  // f(logit, index) for the thread's elements: the batches', where some past the row's end come
  // with -inf, then those before the first and after the last piece, one to a thread.
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    batches([&](const uint4 (&v)[kBatch], int base, auto prefetch) {
      prefetch();
#pragma unroll
      for (int c = 0; c < kElems; ++c) f(element(v[c / VEC], c % VEC), index(base, c));
    });
    edges(f);
  }
  // f(piece, its number) for the thread's pieces, the next N in flight.
  template <int N, typename F>
  __device__ __forceinline__ void ahead(F f) const {
    uint4 v[N];
    int j = (int)threadIdx.x;
#pragma unroll
    for (int q = 0; q < N; ++q)
      if (j + q * kThreads < nvec) v[q] = vecs[j + q * kThreads];
    while (j < nvec) {
#pragma unroll
      for (int q = 0; q < N; ++q) {
        if (j + q * kThreads >= nvec) break;
        const uint4 now = v[q];
        if (j + (q + N) * kThreads < nvec) v[q] = vecs[j + (q + N) * kThreads];
        f(now, j + q * kThreads);
      }
      j += N * kThreads;
    }
  }
  template <typename F>
  __device__ __forceinline__ void edges(F f) const {
    const int rest = V - nvec * VEC;
    if ((int)threadIdx.x < rest) {
      const int i = (int)threadIdx.x < head ? (int)threadIdx.x : nvec * VEC + (int)threadIdx.x;
      f(at(i), i);
    }
  }
  // (x - m) / T, 0 where x equals the maximum (also an infinite one)
  __device__ __forceinline__ float scaled(float v) const { return v == m ? 0.0f : (v - m) / temperature; }
  __device__ __forceinline__ float weight(float v) const { return exp_accurate(scaled(v)); }
  __device__ __forceinline__ uint64_t mass(float w) const { return (uint64_t)__builtin_rintf(w * unit); }
  // Distance below the (finite) maximum in bins, monotone in the logit: infinite for -inf, a
  // NaN for a NaN; and the weight from it, to some 1e-6: for sums, and to tell whether an
  // element can matter.
  __device__ __forceinline__ float distance(float v) const { return (m - v) * to_bin; }
  // An element in the list: its key above the falling index, no bit more than they need, so
  // that the exact search takes few steps.
  static constexpr int kKeyShift = sizeof(IO) == 2 ? 16 : 0;  // a bf16's key has 16 bits
  __device__ __forceinline__ unsigned long long entry(float v, int i) const {
    return (unsigned long long)(key_of(v) >> kKeyShift) << ibits | (uint32_t)((1 << ibits) - 1 - i);
  }
  __device__ __forceinline__ float entry_logit(unsigned long long e) const {
    const float v = logit_of((uint32_t)(e >> ibits) << kKeyShift);
    return kKeyShift == 0 ? v : __uint_as_float(__float_as_uint(v) & 0xffff0000u);
  }
  __device__ __forceinline__ int entry_index(unsigned long long e) const {
    return (1 << ibits) - 1 - (int)((uint32_t)e & (uint32_t)((1 << ibits) - 1));
  }
  __device__ __forceinline__ uint64_t entry_mass(unsigned long long e) const { return mass(weight(entry_logit(e))); }
  static __device__ __forceinline__ float rough_weight(float d) { return ex2(d * (-kLog2e / kBinsPerUnit)); }
};

__device__ __forceinline__ bool masked(float v) { return !(v > -__builtin_inff()); }

// Reductions over the workgroup; slots: one to a wave, read again before it is written anew.
template <typename T, typename F>
__device__ __forceinline__ T block_all(T v, T* slots, F f) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = f(v, (T)__shfl_xor(v, o, 64));
  if (lane == 0) slots[threadIdx.x >> 6] = v;
  __syncthreads();
  v = slots[lane & (kWaves - 1)];
#pragma unroll
  for (int o = kWaves / 2; o > 0; o >>= 1) v = f(v, (T)__shfl_xor(v, o, 64));
  __syncthreads();
  return v;
}
__device__ __forceinline__ uint32_t block_max(uint32_t v, Shared& sm) {
  return block_all(v, sm.word, [](uint32_t a, uint32_t b) { return max(a, b); });
}
__device__ __forceinline__ uint64_t block_sum(uint64_t v, Shared& sm) {
  return block_all((unsigned long long)v, sm.sum, [](unsigned long long a, unsigned long long b) { return a + b; });
}
// Sums of two numbers and of an integer at once.
__device__ __forceinline__ Three block_sums(Three v, Shared& sm) {
  const int lane = threadIdx.x & 63;
  auto add = [&](int o) {
    v.a += __shfl_xor(v.a, o, 64);
    v.b += __shfl_xor(v.b, o, 64);
    v.c += __shfl_xor(v.c, o, 64);
  };
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) add(o);
  if (lane == 0) sm.three[threadIdx.x >> 6] = v;
  __syncthreads();
  v = sm.three[lane & (kWaves - 1)];
#pragma unroll
  for (int o = kWaves / 2; o > 0; o >>= 1) add(o);
  __syncthreads();
  return v;
}

// The best (score, lowest index) so far; a NaN score counts as -inf.
struct Best {
  float score = -__builtin_inff();
  uint32_t at = 0xffffffffu;  // none
  __device__ __forceinline__ void take(float s, uint32_t i) {
    if (i != 0xffffffffu && (at == 0xffffffffu || s > score || (s == score && i < at))) score = s, at = i;
  }
  __device__ __forceinline__ void offer(float w, float noise, uint32_t i) {
    const float s = w / noise;
    take(s != s ? -__builtin_inff() : s, i);
  }
  __device__ __forceinline__ void block(Shared& sm) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      const float s = __shfl_xor(score, o, 64);
      take(s, __shfl_xor(at, o, 64));
    }
    if (lane == 0) sm.score[threadIdx.x >> 6] = score, sm.word[threadIdx.x >> 6] = at;
    __syncthreads();
    score = sm.score[lane & (kWaves - 1)], at = sm.word[lane & (kWaves - 1)];
#pragma unroll
    for (int o = kWaves / 2; o > 0; o >>= 1) {
      const float s = __shfl_xor(score, o, 64);
      take(s, __shfl_xor(at, o, 64));
    }
    __syncthreads();
  }
};

// ---------------------------------------------------------------- bracketing by a histogram

__device__ __forceinline__ void clear_bins(Shared& sm) {
  __syncthreads();  // sm.bin has been read
  for (int i = threadIdx.x; i < kBins; i += kThreads) sm.hist[i] = 0;
  if (threadIdx.x == 0) sm.bin = 4 * kBins, sm.listed = 0;
  __syncthreads();
}

// The first bin up to which the bins' measure reaches `target` (kBins: none does).  MASS: a
// bin holds the sum of e^{(bin - 64 d) / 64} 2^14 of its elements, its mass but for a common
// factor of the bin; else their count.  before and after: whether the masses, whose rounding
// is some 4e-5 of the total, leave it open that it is the bin before or after.
template <bool MASS>
__device__ __forceinline__ int find_bin(float share, float target, int& before, int& after, Shared& sm) {
  constexpr float kSlack = 1.0e-4f;
  __syncthreads();
  const int b = 2 * threadIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const float scale = MASS ? ex2(-(float)b * (kLog2e / kBinsPerUnit)) : 1.0f;
  const float v0 = (float)sm.hist[b] * scale;
  const float v1 = (float)sm.hist[b + 1] * scale * (MASS ? 0.98449644f : 1.0f);  // e^{-1/64}
  float incl = v0 + v1;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const float y = __shfl_up(incl, o, 64);
    if (lane >= o) incl += y;
  }
  if (lane == 63) sm.score[wave] = incl;
  __syncthreads();
  float below = 0.0f, total = 0.0f;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    below += w < wave ? sm.score[w] : 0.0f;
    total += sm.score[w];
  }
  const float want = MASS ? share * total : target;
  const float end = below + incl, start = end - v0 - v1;
  if (end >= want) {
    const bool second = start + v0 < want;
    int bits = (second ? b + 1 : b) * 4;
    if (MASS) {
      const float from = second ? start + v0 : start, to = second ? end : start + v0;
      bits |= (want - from < kSlack * total ? 2 : 0) | (to - want < kSlack * total ? 1 : 0);
    }
    atomicMin(&sm.bin, bits);
  }
  __syncthreads();
  const int bits = sm.bin;
  before = bits >> 1 & 1, after = bits & 1;
  return bits >> 2;
}

// Appends an entry of each lane that has one to the list.
__device__ __forceinline__ void append(bool have, unsigned long long entry, Shared& sm) {
  const uint64_t m = __ballot(have);
  if (m == 0) return;
  const int lane = threadIdx.x & 63, first = __ffsll((unsigned long long)m) - 1;
  uint32_t base = 0;
  if (lane == first) base = atomicAdd(&sm.listed, (uint32_t)__popcll(m));
  base = __shfl(base, first, 64);
  const uint32_t at = base + __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
  if (have && at < kList) sm.list[at] = entry;
}

// Lists the elements of a batch that have their bit in `marks` (bit kElems - 1 - c: element c).
template <typename IO>
__device__ __forceinline__ void append_marked(const Row<IO>& row, const uint4 (&v)[Row<IO>::kBatch], int base,
                                              uint32_t marks, Shared& sm) {
  while (__any(marks != 0)) {
    const int c = __clz((int)(marks | 1u)) - (32 - Row<IO>::kElems);
    uint32_t word = 0;
#pragma unroll
    for (int k = 0; k < 4 * Row<IO>::kBatch; ++k) {
      const uint32_t u[4] = {v[k / 4].x, v[k / 4].y, v[k / 4].z, v[k / 4].w};
      word = c * (int)sizeof(IO) / 4 == k ? u[k % 4] : word;
    }
    float x = __uint_as_float(word);
    if constexpr (sizeof(IO) == 2) x = c & 1 ? bf16_hi(word) : bf16_lo(word);
    append(marks != 0, row.entry(x, row.index(base, c)), sm);
    marks &= ~((1u << (Row<IO>::kElems - 1)) >> c);
  }
}

// Lists the elements of the bins before `end`, by the distance that put them into their bins: a
// limit of m - x, end / to_bin, rounds otherwise and would leave out some of the last bin.
template <typename IO>
__device__ __forceinline__ void list_row(const Row<IO>& row, float end, Shared& sm) {
  row.batches([&](const uint4 (&v)[Row<IO>::kBatch], int base, auto prefetch) {
    prefetch();
    uint32_t marks = 0;
#pragma unroll
    for (int c = 0; c < Row<IO>::kElems; ++c)
      marks = marks + marks + (row.distance(Row<IO>::element(v[c / Row<IO>::VEC], c % Row<IO>::VEC)) < end ? 1u : 0u);
    append_marked(row, v, base, marks, sm);
  });
  row.edges([&](float x, int i) { append(row.distance(x) < end, row.entry(x, i), sm); });
}

// The element of the first n of the list at which the measure of the elements >= it first
// reaches target (1 <= target <= their total).  The measure is the count, or the mass of
// the elements >= from.  Eight bits a step, from the first bit in which the elements differ.
template <typename IO>
__device__ __forceinline__ unsigned long long select_listed(const Row<IO>& row, int n, unsigned long long from,
                                                            uint64_t target, bool by_mass, Shared& sm) {
  unsigned long long lo = ~0ull, hi = 0;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const unsigned long long e = sm.list[i];
    if (e >= from) lo = min(lo, e), hi = max(hi, e);
  }
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    lo = min(lo, (unsigned long long)__shfl_xor(lo, o, 64));
    hi = max(hi, (unsigned long long)__shfl_xor(hi, o, 64));
  }
  if ((threadIdx.x & 63) == 0) sm.sum[threadIdx.x >> 6] = lo, sm.mass[threadIdx.x >> 6] = hi;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; ++w) lo = min(lo, sm.sum[w]), hi = max(hi, sm.mass[w]);
  __syncthreads();
  if (lo == hi) return lo;
  int top = 64 - __clzll(lo ^ hi);  // bits below `top` are undecided
  unsigned long long prefix = top < 64 ? lo >> top : 0;
  uint64_t above = 0;
  while (true) {
    const int s = top > 8 ? top - 8 : 0, width = top - s;
    if (threadIdx.x < 256) sm.mass[threadIdx.x] = 0, sm.count[threadIdx.x] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const unsigned long long e = sm.list[i];
      if (e >= from && (top == 64 || e >> top == prefix)) {
        const uint32_t d = (uint32_t)(e >> s) & ((1u << width) - 1);
        atomicAdd(&sm.count[d], 1u);
        if (by_mass) atomicAdd(&sm.mass[d], (unsigned long long)row.entry_mass(e));
      }
    }
    __syncthreads();
    if (threadIdx.x < 64) {  // lane l: digits 255 - 4l downwards
      const int lane = threadIdx.x;
      unsigned long long h[4], incl = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int d = 255 - 4 * lane - j;
        incl += h[j] = by_mass ? sm.mass[d] : (unsigned long long)sm.count[d];
      }
      const unsigned long long mine = incl;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const unsigned long long y = __shfl_up(incl, o, 64);
        if (lane >= o) incl += y;
      }
      const uint64_t reach = __ballot(above + incl >= target);
      if (reach != 0 && lane == __ffsll((unsigned long long)reach) - 1) {
        unsigned long long b = above + incl - mine;
        int j = 0;
        while (j < 3 && b + h[j] < target) b += h[j++];
        sm.digit = 255 - 4 * lane - j;
        sm.before = b;
      }
      if (reach == 0 && lane == 0) sm.digit = 0, sm.before = above;  // (not where target <= total)
    }
    __syncthreads();
    const uint32_t d = sm.digit;
    above = sm.before;
    prefix = prefix << width | d;
    top = s;
    const bool last = top == 0 || sm.count[d] == 1;
    if (last) {
      if (top == 0) return prefix;
      for (int i = threadIdx.x; i < n; i += kThreads) {
        const unsigned long long e = sm.list[i];
        if (e >= from && e >> top == prefix) sm.found = e;
      }
      __syncthreads();
      return sm.found;
    }
    __syncthreads();
  }
}

// The same for a list of n <= kFew, without steps (1 x 50000, top_k 50 and top_p: 22 us a call in
// place of 31 when it came, 20 now): each entry's rank is counted, and the masses are summed in the
// ranks' order (by each wave for itself).  The element with which
// the first `most` entries end or, if that is asked for, at which their mass reaches target
// (0: the share p of it).  mass: that of the thread's first entry.
template <typename IO>
__device__ __forceinline__ unsigned long long end_of_few(const Row<IO>& row, int n, uint32_t most, bool by_mass,
                                                         uint64_t target, float p, uint64_t mass, Shared& sm) {
  constexpr int kParts = kThreads / kFew;
  unsigned long long* sorted = sm.list + kFew;
  const int i = threadIdx.x % kFew, part = threadIdx.x / kFew, lane = threadIdx.x & 63;
  if (threadIdx.x < kFew) sm.count[threadIdx.x] = 0, sm.mass[threadIdx.x] = 0;
  __syncthreads();
  const unsigned long long e = i < n ? sm.list[i] : 0;
  uint32_t rank = 0;
#pragma unroll 4
  for (int j = part; j < n; j += kParts) rank += sm.list[j] > e;
  if (i < n && rank) atomicAdd(&sm.count[i], rank);
  __syncthreads();
  if (part == 0 && i < n) {
    rank = sm.count[i];
    sorted[rank] = e;
    if (by_mass && rank < most) sm.mass[rank] = mass;
  }
  __syncthreads();
  const uint32_t last = min((uint32_t)n, most) - 1;
  if (!by_mass) return sorted[last];
  unsigned long long h[kFew / 64], incl = 0;
#pragma unroll
  for (int j = 0; j < kFew / 64; ++j) incl += h[j] = sm.mass[kFew / 64 * lane + j];
  const unsigned long long mine = incl;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const unsigned long long y = __shfl_up(incl, o, 64);
    if (lane >= o) incl += y;
  }
  if (target == 0) {
    const unsigned long long sum = __shfl(incl, 63, 64);
    target = (uint64_t)__builtin_ceil((double)p * (double)sum);
    target = target < 1 ? 1 : (target > sum ? sum : target);
  }
  const uint64_t reach = __ballot(incl >= target);
  const int at = reach == 0 ? 63 : __ffsll((unsigned long long)reach) - 1;
  unsigned long long b = incl - mine;
  int j = 0;
#pragma unroll
  for (int q = 0; q < kFew / 64 - 1; ++q) b += h[q], j += b < target;
  return sorted[min((uint32_t)__shfl(kFew / 64 * lane + j, at, 64), last)];
}

// ---------------------------------------------------------------- selection over the whole row

// The largest key K such that the measure of the keys >= K (those >= low and not
// masked) reaches target (1 <= target <= their total measure); before: the measure
// of the keys > K.  The measure is the count, or the mass.
template <bool MASS, typename IO>
__device__ __forceinline__ uint32_t select_key(const Row<IO>& row, uint32_t low, uint64_t target, uint64_t& before,
                                               Shared& sm) {
  uint32_t prefix = 0;
  uint64_t above = 0;
  for (int s = 24; s >= 0; s -= 8) {
    if (threadIdx.x < 256) sm.mass[threadIdx.x] = 0;
    __syncthreads();
    row.each([&](float v, int) {
      const uint32_t k = key_of(v);
      if (k >= low && k > kMasked && (s == 24 || k >> (s + 8) == prefix))
        atomicAdd(&sm.mass[(k >> s) & 255], MASS ? (unsigned long long)row.mass(row.weight(v)) : 1ull);
    });
    __syncthreads();
    if (threadIdx.x < 64) {  // lane l: digits 255 - 4l downwards
      const int lane = threadIdx.x;
      unsigned long long h[4], incl = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) incl += h[j] = sm.mass[255 - 4 * lane - j];
      const unsigned long long mine = incl;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const unsigned long long y = __shfl_up(incl, o, 64);
        if (lane >= o) incl += y;
      }
      const uint64_t reach = __ballot(above + incl >= target);
      if (reach != 0 && lane == __ffsll((unsigned long long)reach) - 1) {
        unsigned long long b = above + incl - mine;
        int j = 0;
        while (j < 3 && b + h[j] < target) b += h[j++];
        sm.digit = 255 - 4 * lane - j;
        sm.before = b;
      }
    }
    __syncthreads();
    prefix = prefix << 8 | sm.digit;
    above = sm.before;
    __syncthreads();
  }
  before = above;
  return prefix;
}

// What stays of a row, found without the histogram: the keys above `cut` and, of those equal
// to it, the ones up to index `last_tie`.
struct Cut {
  uint32_t key;
  int last_tie;
};

template <typename IO>
__device__ Cut cut_row(const Row<IO>& row, int64_t k, float p, Shared& sm) {
  uint32_t cut = kMasked + 1;
  uint64_t ties = ~0ull;
  if (k > 0 && k < row.V) {
    uint64_t n = 0, before;
    row.each([&](float v, int) { n += !masked(v); });
    n = block_sum(n, sm);
    if ((uint64_t)k < n) {
      cut = select_key<false>(row, cut, (uint64_t)k, before, sm);
      ties = (uint64_t)k - before;
    }
  }
  if (p < 1.0f) {
    uint64_t total = 0;
    row.each([&](float v, int) {
      const uint32_t key = key_of(v);
      if (key > cut || (key == cut && ties == ~0ull)) total += row.mass(row.weight(v));
    });
    total = block_sum(total, sm);
    if (ties != ~0ull) total += ties * row.mass(row.weight(logit_of(cut)));
    // before < p total for the integer `before` is before < ceil(p total)
    uint64_t target = (uint64_t)__builtin_ceil((double)p * (double)total), before;
    target = target < 1 ? 1 : (target > total ? total : target);
    const uint32_t at = select_key<true>(row, cut, target, before, sm);
    const uint64_t one = row.mass(row.weight(logit_of(at)));
    const uint64_t need = one > 0 ? (target - before + one - 1) / one : ~0ull;
    if (at != cut || need < ties) ties = need;
    cut = at;
  }
  // Index of the last equal logit that stays: threads own consecutive stretches.
  if (threadIdx.x == 0) sm.cut_index = 0x7fffffff;
  if (ties != ~0ull) {
    const int per = (row.V + kThreads - 1) / kThreads;
    const int i0 = threadIdx.x * per, i1 = min(i0 + per, row.V);
    uint32_t c = 0;
    for (int i = i0; i < i1; ++i) c += row.key(i) == cut;
    uint32_t incl = c;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const uint32_t y = __shfl_up(incl, o, 64);
      if (lane >= o) incl += y;
    }
    if (lane == 63) sm.word[wave] = incl;
    __syncthreads();
    for (int w = 0; w < wave; ++w) incl += sm.word[w];
    if (incl >= ties && incl - c < ties) {
      uint64_t left = ties - (incl - c);
      for (int i = i0; i < i1; ++i)
        if (row.key(i) == cut && --left == 0) {
          sm.cut_index = i;
          break;
        }
    }
  }
  __syncthreads();
  return Cut{cut, sm.cut_index};
}

// ---------------------------------------------------------------- scoring

// Limits of m - x for one pass over the row.  Below `sure` an element is scored, from there
// up to below `near` if its exact weight is large enough, from `lo` up to below `hi` it is
// listed (sure <= near <= lo <= hi; all but an infinite lo = hi far below kFarthest).
struct Limits {
  float sure, near, lo, hi;
  bool lists;
};
// Sums of rough weights: of what lies below lo, of the scored elements, of all.
struct Sums {
  float above = 0.0f, kept = 0.0f, all = 0.0f;
};

// kElems elements to a thread at a time: rough weights, then the noise of the pieces that
// have an element to be scored, the next pieces underway meanwhile, then the question whether
// a weight w exceeds its noise times a bound a little below the best rough score that any
// wave has published, one multiply-add to an element.  Where one does, rough scores are worked
// out, and the exact form (an exponential and a division) for the elements that pass the raised
// bound.  With a bound of the thread's own some lane of 64 passed it at nearly every element
// (256 rows of 128000, top_p: 132 us against 113).
template <typename IO>
__device__ __forceinline__ void score_row(const Row<IO>& row, const Limits& at, float minp, const float* noise,
                                          Sums& sums, Best& best, Shared& sm) {
  constexpr int VEC = Row<IO>::VEC, kBatch = Row<IO>::kBatch;
  typedef float Noise4 __attribute__((ext_vector_type(4), aligned(4)));
  const int tid = threadIdx.x;
  const float to_exponent = row.to_bin * (-kLog2e / kBinsPerUnit);
  const uint32_t lo_bits = __float_as_uint(at.lo), span = __float_as_uint(at.hi) - lo_bits;
  float bound = 0.0f, zone = 0.0f;
  Noise4 e[Row<IO>::kElems / 4];  // (that of pieces without an element to be scored: whatever was there)
#pragma unroll
  for (int c = 0; c < Row<IO>::kElems / 4; ++c) e[c] = Noise4{1.0f, 1.0f, 1.0f, 1.0f};
  auto exact = [&](float v, float n, int i, bool count) {
    const float w = row.weight(v);
    if (!(w > 0.0f && w >= minp)) return;
    zone += count ? w : 0.0f;
    best.offer(w, n, i);
  };
  row.batches([&](const uint4 (&v)[kBatch], int base, auto prefetch) {
    float w[Row<IO>::kElems], d[Row<IO>::kElems];
    float beyond = kFarthest;  // the least from `sure` on
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      float least = kFarthest;
#pragma unroll
      for (int c = 0; c < VEC; ++c) {
        const int k = q * VEC + c;
        d[k] = fminf(row.m - Row<IO>::element(v[q], c), kFarthest);  // (NaN: no weight)
        const float rough = ex2(d[k] * to_exponent);
        const bool in = d[k] < at.sure;
        least = fminf(least, d[k]);
        beyond = fminf(beyond, in ? kFarthest : d[k]);
        sums.all += rough;
        w[k] = in ? rough : 0.0f;
        sums.kept += w[k];
      }
      if (least < at.sure) {
        const int i = row.index(base, q * VEC);
#pragma unroll
        for (int c = 0; c < VEC / 4; ++c)
          e[q * (VEC / 4) + c] = *reinterpret_cast<const Noise4*>(noise + i + 4 * c);
      }
    }
    if (at.lists) {
      uint32_t listed = 0;  // marks of those to be listed
#pragma unroll
      for (int c = 0; c < Row<IO>::kElems; ++c)
        listed = listed + listed + (__float_as_uint(d[c]) - lo_bits < span ? 1u : 0u);
      append_marked(row, v, base, listed, sm);
      if (at.sure < at.lo) {
#pragma unroll
        for (int c = 0; c < Row<IO>::kElems; ++c)
          sums.above += d[c] >= at.sure && d[c] < at.lo ? ex2(d[c] * to_exponent) : 0.0f;
      }
    }
    prefetch();
    bound = fmaxf(bound, __uint_as_float(*(volatile uint32_t*)&sm.bound));
    float over = 0.0f;
#pragma unroll
    for (int c = 0; c < Row<IO>::kElems; ++c) over = fmaxf(over, __builtin_fmaf(-bound, e[c / 4][c % 4], w[c]));
    uint32_t which = 0, unsure = 0;
    if (__any(over > 0.0f)) {
      float score[Row<IO>::kElems], top = 0.0f;
#pragma unroll
      for (int c = 0; c < Row<IO>::kElems; ++c) {
        score[c] = w[c] > 0.0f ? w[c] * rcp(e[c / 4][c % 4]) : -__builtin_inff();
        top = fmaxf(top, score[c]);
      }
#pragma unroll 1
      for (int o = 32; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o, 64));
      // (an infinite score leaves the bound as it is)
      bound = fmaxf(bound, __builtin_fmaf(-1.0e-4f, top, top));
      if ((tid & 63) == 0) atomicMax(&sm.bound, __float_as_uint(bound));
#pragma unroll
      for (int c = 0; c < Row<IO>::kElems; ++c) which |= w[c] > 0.0f && !(score[c] < bound) ? 1u << c : 0u;
    }
    if (beyond < at.near) {
#pragma unroll
      for (int c = 0; c < Row<IO>::kElems; ++c) unsure |= d[c] >= at.sure && d[c] < at.near ? 1u << c : 0u;
    }
    for (uint32_t todo = which | unsure; todo != 0; todo &= todo - 1) {
      const int c = __ffs((int)todo) - 1, i = row.index(base, c);
      exact(row.at(i), noise[i], i, unsure >> c & 1);
    }
  });
  sums.above += sums.kept;
  row.edges([&](float x, int i) {
    const float d = fminf(row.m - x, kFarthest), rough = ex2(d * to_exponent);
    sums.all += rough;
    sums.above += d < at.lo ? rough : 0.0f;
    append(__float_as_uint(d) - lo_bits < span, row.entry(x, i), sm);
    if (d < at.near) exact(x, noise[i], i, true);
  });
  sums.kept += zone;
}

// ---------------------------------------------------------------- the row

template <typename IO>
__global__ __launch_bounds__(kThreads) void sample_row_kernel(SampleArgs a, float unit, int ibits) {
  __shared__ Shared sm;
  const int64_t r = blockIdx.x;
  Row<IO> row;
  row.set((const IO*)a.logits + r * a.V, (int)a.V);
  row.unit = unit;
  row.ibits = ibits;
  row.cache = sm.cache;
  row.cached = row.nvec < kCacheVecs ? row.nvec : kCacheVecs;
  const float* noise = a.noise + r * a.V;
  int64_t k = a.top_k ? a.top_k[r] : 0;
  const float t = a.temperature ? a.temperature[r] : 1.0f;
  const float p = a.top_p ? a.top_p[r] : 1.0f;
  const float minp = a.min_p && a.min_p[r] > 0.0f ? fminf(a.min_p[r], 1.0f) : 0.0f;  // NaN: off
  const bool greedy = !(t > 0.0f) || p <= 0.0f || k == 1;
  row.temperature = t > 0.0f ? t : 1.0f;
  row.to_bin = kBinsPerUnit / row.temperature;

  if (threadIdx.x == 0) sm.bound = 0;
  const bool want_k = k > 0 && k < row.V, want_p = p < 1.0f;
  // top_p alone: the histogram is filled in the same pass as the largest logit is found, its
  // distances taken from the largest of the row's first pieces, kAbove bins of it above that
  // (256 x 128000: 70 us in place of 82 with a pass for each).
  float ref = -__builtin_inff();
  if (!greedy && want_p && !want_k && row.to_bin >= kLeastToBin && row.to_bin <= 3.4028235e38f) {
    if ((int)threadIdx.x < row.nvec) {
      const uint4 v = row.vecs[threadIdx.x];
#pragma unroll
      for (int e = 0; e < Row<IO>::VEC; ++e) ref = fmaxf(ref, Row<IO>::element(v, e));
    }
    ref = logit_of(block_max(key_of(ref), sm));
  }
  const bool fused = fabsf(ref) < __builtin_inff();
  if (fused) clear_bins(sm);
  auto count = [&](float d) {  // d: a distance in bins
    if (!(d < (float)kBins)) return;
    d = fmaxf(d, 0.0f);  // (below 0: the counts are not used)
    const int b = (int)d;
    const float f = (d - (float)b) * (1.0f / kBinsPerUnit);
    // e^-f 2^14 for f <= 1/64 (a bin of more than 2^18 elements runs over: no list holds them
    // either, and a bracket that the end is not in is noticed when the list is searched)
    atomicAdd(&sm.hist[b], (uint32_t)__builtin_fmaf(f, __builtin_fmaf(f, 8192.0f, -16384.0f), 16384.5f));
  };
  auto count_from_ref = [&](float v) { count(__builtin_fmaf(ref - v, row.to_bin, kAbove)); };
  // the largest logit (a NaN is never the larger), the thread's and the row's
  float mine = -__builtin_inff();
  auto piece = [&](const uint4& v, int j) {
    if (j < kCacheVecs) sm.cache[j] = v;
#pragma unroll
    for (int e = 0; e < Row<IO>::VEC; ++e) mine = fmaxf(mine, Row<IO>::element(v, e));
  };
  if (fused) {
    row.template ahead<4>([&](const uint4& v, int j) {
      piece(v, j);
#pragma unroll
      for (int e = 0; e < Row<IO>::VEC; ++e) count_from_ref(Row<IO>::element(v, e));
    });
    row.edges([&](float v, int) { count_from_ref(v); });
  } else {
    row.template ahead<4>(piece);
  }
  row.edges([&](float v, int) { mine = fmaxf(mine, v); });
  row.mkey = block_max(key_of(mine), sm);
  row.m = logit_of(row.mkey);
  if (row.mkey <= kMasked) {
    if (threadIdx.x == 0) {
      a.tokens[r] = -1;
      if (a.logprob) a.logprob[r] = -__builtin_inff();
    }
    return;
  }

  Best best;
  double total = 1.0;  // mass of what stays
  float chosen = row.m;
  if (greedy) {
    uint32_t first = 0;
    row.each([&](float v, int i) {
      if (v == row.m) first = max(first, (uint32_t)~i);
    });
    best.at = ~block_max(first, sm);
  } else {
    int before, after;
    float lo = 0.0f, hi = -1.0f;  // distances below lo stay, those from lo up to below hi are listed
    // (an infinite maximum has no distances; its equals are all that has a weight)
    bool row_wide = row.m > 3.4028235e38f || row.to_bin > 3.4028235e38f || row.to_bin < kLeastToBin;
    if (row_wide) {
      clear_bins(sm);
    } else if (want_k) {
      clear_bins(sm);
      int b = kBins;
      if (k <= kMaximaTopK) {  // k threads' maxima, so k elements, lie up to the bin
        const float d = row.distance(mine);
        if (d < (float)kBins) atomicAdd(&sm.hist[(int)d], 1u);
        b = find_bin<false>(0.0f, (float)k, before, after, sm);
      }
      if (b == kBins) {
        clear_bins(sm);
        row.each([&](float v, int) {
          const float d = row.distance(v);
          if (d < (float)kBins) atomicAdd(&sm.hist[(int)d], 1u);
        });
        b = find_bin<false>(0.0f, (float)k, before, after, sm);
      }
      // fewer than k within the histogram's range: all that is not masked
      hi = b == kBins ? __builtin_inff() : (float)(b + 1);
    } else if (want_p) {
      const float shift = (row.m - ref) * row.to_bin - kAbove;  // from bins of ref to those of m
      const bool counted = fused && shift <= 0.0f;
      if (!counted) {
        clear_bins(sm);
        row.each([&](float v, int) { count(row.distance(v)); });
      }
      const int b = find_bin<true>(p, 0.0f, before, after, sm);
      lo = fmaxf((float)(b - before) + (counted ? shift : 0.0f), 0.0f);
      // (at least lo: counts that run over to nothing leave the first bin, above the maximum's)
      hi = fmaxf((float)(b + 1 + after) + (counted ? shift : 0.0f), lo);
      row_wide = b == kBins;
    }
    if (!want_k && !want_p && !row_wide) lo = hi = __builtin_inff();
    Sums sums;
    uint64_t listed = 0;  // mass of the listed elements that stay
    if (!row_wide) {
      if (want_k) list_row(row, hi, sm);
      else {
        // the exact test of min_p for what lies a hundredth of a bin about its limit; weights
        // below e^-80 are worked out exactly too, and those below e^-87 are 0
        const float limit = fminf(-logf(minp) * kBinsPerUnit, 83.5f * kBinsPerUnit);
        const float margin = minp > 0.0f && limit < 83.5f * kBinsPerUnit ? 0.01f : 4.0f * kBinsPerUnit;
        const float one = 1.0f / row.to_bin, end = lo * one;
        score_row(row, {fminf((limit - margin) * one, end), fminf((limit + margin) * one, end), end, hi * one, want_p},
                  minp, noise, sums, best, sm);
      }
    }
    if (want_k || want_p || row_wide) {
      __syncthreads();
      const int n = (int)sm.listed;
      row_wide |= n > kList;
      unsigned long long from = 0;  // listed elements >= from stay
      const bool few = n <= kFew;
      // the thread's first entry, its noise underway during the search
      const int i0 = threadIdx.x;
      const unsigned long long e0 = i0 < n && !row_wide ? sm.list[i0] : 0;
      const float n0 = i0 < n && !row_wide ? noise[row.entry_index(e0)] : 1.0f;
      const float w0 = row.weight(row.entry_logit(e0));
      uint64_t target = (uint64_t)k;
      // by counts, then (or only) by masses
      for (bool by_mass = !want_k; !row_wide; by_mass = true) {
        if (by_mass && !(few && want_k)) {
          Three sum = {(double)sums.above, (double)sums.all, 0};
          for (int i = threadIdx.x; i < n; i += kThreads)
            if (sm.list[i] >= from) sum.c += row.entry_mass(sm.list[i]);
          sum = block_sums(sum, sm);
          const double mass = (double)sum.c;
          double need = __builtin_ceil(want_k ? (double)p * mass : ((double)p * sum.b - sum.a) * (double)unit);
          if (want_k) need = fmin(fmax(need, 1.0), mass);
          if (!(need >= 1.0 && need <= mass)) row_wide = true;  // the end is not in the list
          target = min((uint64_t)need, (uint64_t)sum.c);  // (`mass` may have been rounded up)
        }
        if (row_wide) break;
        if (few) {
          from = end_of_few(row, n, want_k ? (uint32_t)min(k, (int64_t)kFew) : kFew, want_p, want_k ? 0 : target, p,
                            row.mass(w0), sm);
          break;
        }
        if (by_mass || n > k) from = select_listed(row, n, from, target, by_mass, sm);
        if (by_mass || !want_p) break;
      }
      if (!row_wide) {
        for (int i = threadIdx.x; i < n; i += kThreads) {
          const unsigned long long e = i == i0 ? e0 : sm.list[i];
          if (e < from) continue;
          const float w = i == i0 ? w0 : row.weight(row.entry_logit(e));
          if (!(w > 0.0f && w >= minp)) continue;
          listed += row.mass(w);  // an integer: the list's order is no fixed one
          best.offer(w, i == i0 ? n0 : noise[row.entry_index(e)], row.entry_index(e));
        }
      }
    }
    while (true) {
      if (row_wide) {
        best = Best();
        sums.kept = 0.0f;
        listed = 0;
        const Cut cut = cut_row(row, k, p, sm);
        row.each([&](float v, int i) {
          const uint32_t key = key_of(v);
          if (!(key > cut.key || (key == cut.key && i <= cut.last_tie))) return;
          const float w = row.weight(v);
          if (!(w > 0.0f && w >= minp)) return;
          sums.kept += w;
          best.offer(w, noise[i], i);
        });
      }
      best.block(sm);
      if (best.at != 0xffffffffu) chosen = row.at(best.at);
      const Three sum = block_sums(Three{(double)sums.kept, 0.0, listed}, sm);
      total = sum.a + (double)sum.c / (double)unit;
      if (best.score > 0.0f || row_wide) break;
      row_wide = true;  // scores of 0 and less, and those that are no numbers, are not among the sure ones
    }
  }
  if (threadIdx.x == 0) {
    a.tokens[r] = best.at;
    if (a.logprob) a.logprob[r] = row.scaled(chosen) - logf((float)total);
  }
}

}  // namespace

hipError_t launch_sample(const SampleArgs& a, int io, hipStream_t st) {
  int bits = 0;
  while ((int64_t(1) << bits) < a.V) ++bits;
  const float unit = __builtin_ldexpf(1.0f, 62 - bits);  // a row's masses sum to 2^62 at most
  if (io == kIoBF16) hipLaunchKernelGGL(sample_row_kernel<uint16_t>, dim3((unsigned)a.rows), dim3(kThreads), 0, st, a, unit, bits);
  else hipLaunchKernelGGL(sample_row_kernel<float>, dim3((unsigned)a.rows), dim3(kThreads), 0, st, a, unit, bits);
  return hipGetLastError();
}

}  // namespace s6
