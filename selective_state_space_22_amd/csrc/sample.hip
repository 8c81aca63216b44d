// sample.hip -- drawing a token per row of logits (include/mamba_mi355x_lm.h).
//
// One workgroup per row.  The three filters keep a prefix of the row in falling
// order (equal logits: lower index first), so what stays is everything above a
// cut key, the first few logits equal to it, and of those what min_p leaves.  The
// cut is found by radix selection over an order-preserving 32-bit key, by counts
// (top_k) or by masses (top_p).  Masses are summed as integers (w 2^s, s = 62 -
// log2 of the row length), so that their sums do not depend on an order.
#include <hip/hip_runtime.h>

#include "lm_internal.h"
#include "s6_device.h"

namespace s6 {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr uint32_t kMasked = 0x007fffffu;  // key of -inf; NaN takes it too

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

// One row's logits as keys, and the weights relative to its largest logit.
template <typename IO>
struct Row {
  const IO* x;
  int V;
  uint32_t mkey;  // key of the largest logit
  float m, temperature;
  float unit;     // masses are round(w * unit)
  __device__ __forceinline__ uint32_t key(int i) const { return key_of(load_io(x, i)); }
  // (x - m) / T, 0 where x equals the maximum (also an infinite one)
  __device__ __forceinline__ float scaled(uint32_t k) const {
    return k == mkey ? 0.0f : (logit_of(k) - m) / temperature;
  }
  __device__ __forceinline__ float weight(uint32_t k) const { return k == mkey ? 1.0f : exp_accurate(scaled(k)); }
  __device__ __forceinline__ uint64_t mass(uint32_t k) const {
    return (uint64_t)__builtin_rintf(weight(k) * unit);
  }
};

struct Shared {
  unsigned long long hist[256];
  unsigned long long sum[kWaves];
  uint32_t word[kWaves];
  float score[kWaves];
  uint32_t digit;
  unsigned long long before;
  int cut_index;
};

__device__ __forceinline__ uint32_t block_max(uint32_t v, Shared& sm) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = max(v, (uint32_t)__shfl_xor(v, o, 64));
  if ((threadIdx.x & 63) == 0) sm.word[threadIdx.x >> 6] = v;
  __syncthreads();
  uint32_t r = 0;
  for (int w = 0; w < kWaves; ++w) r = max(r, sm.word[w]);
  __syncthreads();
  return r;
}

__device__ __forceinline__ uint64_t block_sum(uint64_t v, Shared& sm) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += (uint64_t)__shfl_xor((unsigned long long)v, o, 64);
  if ((threadIdx.x & 63) == 0) sm.sum[threadIdx.x >> 6] = v;
  __syncthreads();
  uint64_t r = 0;
  for (int w = 0; w < kWaves; ++w) r += sm.sum[w];
  __syncthreads();
  return r;
}

// The largest key K such that the measure of the keys >= K (those >= low and not
// masked) reaches target (1 <= target <= their total measure); before: the measure
// of the keys > K.  The measure is the count, or the mass.
template <bool MASS, typename IO>
__device__ __forceinline__ uint32_t select_key(const Row<IO>& row, uint32_t low, uint64_t target, uint64_t& before,
                                               Shared& sm) {
  uint32_t prefix = 0;
  uint64_t above = 0;
  for (int s = 24; s >= 0; s -= 8) {
    for (int i = threadIdx.x; i < 256; i += kThreads) sm.hist[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < row.V; i += kThreads) {
      const uint32_t k = row.key(i);
      if (k >= low && k > kMasked && (s == 24 || k >> (s + 8) == prefix))
        atomicAdd(&sm.hist[(k >> s) & 255], MASS ? (unsigned long long)row.mass(k) : 1ull);
    }
    __syncthreads();
    if (threadIdx.x < 64) {  // lane l: digits 255 - 4l downwards
      const int lane = threadIdx.x;
      unsigned long long h[4], incl = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) incl += h[j] = sm.hist[255 - 4 * lane - j];
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

template <typename IO>
__global__ __launch_bounds__(kThreads) void sample_row_kernel(SampleArgs a, float unit) {
  __shared__ Shared sm;
  const int64_t r = blockIdx.x;
  Row<IO> row;
  row.x = (const IO*)a.logits + r * a.V;
  row.V = (int)a.V;
  row.unit = unit;
  const float* noise = a.noise + r * a.V;
  int64_t k = a.top_k ? a.top_k[r] : 0;
  const float t = a.temperature ? a.temperature[r] : 1.0f;
  const float p = a.top_p ? a.top_p[r] : 1.0f;
  const float minp = a.min_p && a.min_p[r] > 0.0f ? fminf(a.min_p[r], 1.0f) : 0.0f;  // NaN: off
  const bool greedy = !(t > 0.0f) || p <= 0.0f;
  row.temperature = t > 0.0f ? t : 1.0f;
  if (greedy) k = 1;

  uint32_t mk = 0;
  for (int i = threadIdx.x; i < row.V; i += kThreads) mk = max(mk, row.key(i));
  row.mkey = block_max(mk, sm);
  row.m = logit_of(row.mkey);
  if (row.mkey <= kMasked) {
    if (threadIdx.x == 0) {
      a.tokens[r] = -1;
      if (a.logprob) a.logprob[r] = -__builtin_inff();
    }
    return;
  }

  // What stays: keys above cut, and the first `ties` of those equal to it.
  uint32_t cut = kMasked + 1;
  uint64_t ties = ~0ull;
  if (k > 0 && k < row.V) {
    uint64_t n = 0, before;
    for (int i = threadIdx.x; i < row.V; i += kThreads) n += row.key(i) > kMasked;
    n = block_sum(n, sm);
    if ((uint64_t)k < n) {
      cut = select_key<false>(row, cut, (uint64_t)k, before, sm);
      ties = (uint64_t)k - before;
    }
  }
  if (p < 1.0f && k != 1) {
    uint64_t total = 0;
    for (int i = threadIdx.x; i < row.V; i += kThreads) {
      const uint32_t key = row.key(i);
      if (key > cut || (key == cut && ties == ~0ull)) total += row.mass(key);
    }
    total = block_sum(total, sm);
    if (ties != ~0ull) total += ties * row.mass(cut);
    // before < p total for the integer `before` is before < ceil(p total)
    uint64_t target = (uint64_t)__builtin_ceil((double)p * (double)total), before;
    target = target < 1 ? 1 : (target > total ? total : target);
    const uint32_t at = select_key<true>(row, cut, target, before, sm);
    const uint64_t one = row.mass(at);
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
  const int last_tie = sm.cut_index;

  uint64_t total = 0;
  float best = -__builtin_inff();
  uint32_t at = 0xffffffffu;
  for (int i = threadIdx.x; i < row.V; i += kThreads) {
    const uint32_t key = row.key(i);
    if (!(key > cut || (key == cut && i <= last_tie))) continue;
    const float w = row.weight(key);
    if (!(w > 0.0f && w >= minp)) continue;
    total += (uint64_t)__builtin_rintf(w * row.unit);
    float sc = w / noise[i];
    if (sc != sc) sc = -__builtin_inff();
    if (at == 0xffffffffu || sc > best) best = sc, at = i;
  }
  total = block_sum(total, sm);
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    const float sc = __shfl_xor(best, o, 64);
    const uint32_t i = __shfl_xor(at, o, 64);
    if (i != 0xffffffffu && (at == 0xffffffffu || sc > best || (sc == best && i < at))) best = sc, at = i;
  }
  if ((threadIdx.x & 63) == 0) sm.score[threadIdx.x >> 6] = best, sm.word[threadIdx.x >> 6] = at;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kWaves; ++w) {
      const float sc = sm.score[w];
      const uint32_t i = sm.word[w];
      if (i != 0xffffffffu && (at == 0xffffffffu || sc > best || (sc == best && i < at))) best = sc, at = i;
    }
    a.tokens[r] = at;
    if (a.logprob) a.logprob[r] = row.scaled(row.key(at)) - logf((float)((double)total / (double)row.unit));
  }
}

}  // namespace

size_t sample_ws_bytes(int64_t, int64_t, int) { return 0; }

hipError_t launch_sample(const SampleArgs& a, int io, void*, hipStream_t st) {
  int bits = 0;
  while ((int64_t(1) << bits) < a.V) ++bits;
  const float unit = __builtin_ldexpf(1.0f, 62 - bits < 44 ? 62 - bits : 44);
  if (io == kIoBF16) hipLaunchKernelGGL(sample_row_kernel<uint16_t>, dim3((unsigned)a.rows), dim3(kThreads), 0, st, a, unit);
  else hipLaunchKernelGGL(sample_row_kernel<float>, dim3((unsigned)a.rows), dim3(kThreads), 0, st, a, unit);
  return hipGetLastError();
}

}  // namespace s6
