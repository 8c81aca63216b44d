// verify.hip -- verification of drafted tokens against the target's probabilities, on gfx950.
//
// Per row with drafts d_0 .. d_{n-1}: draft k stays while uniform_k q_k(d_k) < p_k(d_k) and all before it
// stayed (a draft of probability q is kept with probability min(1, p / q)).  With a drafts kept, one token
// more is drawn: the argmax over i of w_i / noise_i, w = max(p_a - q_a, 0) where draft a was refused (w = p_a
// if that is zero everywhere), w = p_a where none was; with Exp(1) noise it has the distribution w / sum(w).
//
// What a row needs is one row of p, of q and of the noise, and a handful of single values: memory bounds it.
// A row is split over workgroups where there are few; each finds the number of kept drafts for itself (a
// gather of n values) and the best (score, index) of its part, and a second launch joins the parts.  A score
// and its index are one 64-bit key, the index inverted, so that the largest key is the first of the best.
// Measured (a streaming copy reaches 6.1 TB/s): 64 rows of 128000 fp32, 8 drafts, 18 us for 98 MB at the most (84 MB
// read) and 4 us the join; one row of 50000, 4 drafts, 5.3 and 2.5 us, latency of the drafts' gathers, then of the row.
#include "layer_device.h"
#include "layer_internal.h"

namespace s6 {
namespace {

constexpr int kBlock = 256;            // threads of a row's part
constexpr int kWide = 1024;            // threads of a row that is a workgroup's alone
constexpr int V = 4;                   // elements per load
constexpr int kAhead = 4;              // loads in flight
constexpr int64_t kPart = 2048;        // fewest elements of a row's part
constexpr int64_t kFill = 1024;        // workgroups that fill the chip (64 x 128000: 512 20.4 us, 1024 19.1, 2048 20.7)
// A row that kWide threads read in one round of loads ahead is one workgroup of its own and needs no join, as
// long as there is a compute unit for each (bf16, 4 drafts: 1 x 8000 in parts 9.2 us a call, alone 7.4; 32 x 12000
// 8.9, 7.8; beyond the round 1 x 20000 9.3, 10.2 and 32 x 20000 8.8, 11.0; more rows than compute units 1000 x 30000
// 42, 46).
constexpr int64_t kAlone = kWide * V * kAhead;
constexpr int64_t kUnits = 256;

// Ordered bits of a score (larger float, larger integer), then the inverted index; 0: no candidate.
__device__ __forceinline__ uint64_t key_of(float score, int32_t index) {
  const uint32_t b = __float_as_uint(score);
  const uint32_t o = b & 0x80000000u ? ~b : b | 0x80000000u;
  return ((uint64_t)o << 32) | (uint32_t)(0xffffffffu - (uint32_t)index);
}

template <int BLOCK>
__device__ __forceinline__ uint64_t block_max(uint64_t v, uint64_t* lds) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) {
    const uint64_t o = __shfl_xor((unsigned long long)v, m, 64);
    v = o > v ? o : v;
  }
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < BLOCK / 64; ++w) v = lds[w] > v ? lds[w] : v;
  return v;
}

// Drafts kept of a row, the same in every wave that asks.
template <typename IO>
__device__ __forceinline__ int64_t kept_drafts(const VerifyArgs& a, int64_t row, int64_t count) {
  const int lane = threadIdx.x & 63;
  for (int64_t k0 = 0; k0 < count; k0 += 64) {
    const int64_t k = k0 + lane;
    bool stays = false;
    if (k < count) {
      const int64_t id = a.drafted[row * a.K + k];
      if (id >= 0 && id < a.V) {
        const float p = load_io(static_cast<const IO*>(a.target), (size_t)((row * (a.K + 1) + k) * a.V + id));
        const float q = load_io(static_cast<const IO*>(a.draft), (size_t)((row * a.K + k) * a.V + id));
        stays = a.uniform[row * a.K + k] * q < p;
      }
    }
    const uint64_t no = ~__ballot(stays);
    if (no) return k0 + __builtin_ctzll(no);
  }
  return count;
}

struct Best {
  float score = 0.0f;
  int32_t index = -1;
  __device__ __forceinline__ void offer(float w, float noise, int32_t i) {
    // negative noise and NaN lose against everything, a noise of +-0 wins
    float s = noise >= 0.0f ? w / __builtin_fabsf(noise) : -__builtin_inff();
    s = s == s ? s : -__builtin_inff();
    if (w > 0.0f && (index < 0 || s > score)) {
      score = s;
      index = i;
    }
  }
  __device__ __forceinline__ uint64_t key() const { return index < 0 ? 0u : key_of(score, index); }
};

// The best of elements [lo, hi) of a row, over the workgroup's threads.  q null: weights p.
template <typename IO, int BLOCK>
__device__ __forceinline__ uint64_t best_of(const IO* p, const IO* q, const float* noise, int64_t lo, int64_t hi,
                                            uint64_t* lds) {
  Best best;
  for (int64_t i0 = lo + threadIdx.x * V; i0 < hi; i0 += BLOCK * V * kAhead) {
    raw_t<IO, V> rp[kAhead], rq[kAhead];
    raw_t<float, V> rn[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t i = i0 + u * BLOCK * V;
      const int nv = hi - i < V ? (int)(hi - i) : V;
      rq[u] = raw_t<IO, V>(0u);
      if (nv == V) {
        rp[u] = load_raw<IO, V, true>(p + i, V);
        if (q) rq[u] = load_raw<IO, V, true>(q + i, V);
        rn[u] = load_raw<float, V, true>(noise + i, V);
      } else {
        rp[u] = load_raw<IO, V, false>(p + i, nv);
        if (q) rq[u] = load_raw<IO, V, false>(q + i, nv);
        rn[u] = load_raw<float, V, false>(noise + i, nv);
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      float fp[V], fq[V], fn[V];
      widen<IO, V>(rp[u], fp);
      widen<IO, V>(rq[u], fq);
      widen<float, V>(rn[u], fn);
#pragma unroll
      for (int k = 0; k < V; ++k) best.offer(fp[k] - fq[k], fn[k], (int32_t)(i0 + u * BLOCK * V + k));
    }
  }
  return block_max<BLOCK>(best.key(), lds);
}

// Writes a row's tokens, given the best key of the weights that its drafts leave.
template <typename IO, int BLOCK>
__device__ __forceinline__ void finish_row(const VerifyArgs& a, int64_t row, int64_t kept, bool refused, uint64_t key,
                                           uint64_t* lds) {
  if (refused && key == 0) {  // p is nowhere above q: from p itself (a row that rounding alone can make)
    key = best_of<IO, BLOCK>(static_cast<const IO*>(a.target) + (row * (a.K + 1) + kept) * a.V, static_cast<const IO*>(nullptr),
                      a.noise + row * a.V, 0, a.V, lds);
  }
  const int64_t token = key == 0 ? -1 : (int64_t)(0xffffffffu - (uint32_t)key);
  for (int64_t k = threadIdx.x; k <= a.K; k += BLOCK)
    a.tokens[row * (a.K + 1) + k] = k < kept ? a.drafted[row * a.K + k] : (k == kept ? token : -1);
  if (threadIdx.x == 0) a.accepted[row] = (int32_t)kept;
}

__device__ __forceinline__ int64_t count_of(const VerifyArgs& a, int64_t row) {
  if (!a.counts) return a.K;
  const int64_t c = a.counts[row];
  return c < 0 ? 0 : (c < a.K ? c : a.K);
}

template <typename IO, int BLOCK>
__global__ __launch_bounds__(BLOCK) void verify_kernel(VerifyArgs a, int parts, int64_t part, uint64_t* keys) {
  __shared__ uint64_t lds[BLOCK / 64];
  const int64_t row = blockIdx.x / (uint32_t)parts;
  const int s = blockIdx.x % (uint32_t)parts;
  const int64_t count = count_of(a, row), kept = kept_drafts<IO>(a, row, count);
  const bool refused = kept < count;
  const int64_t lo = s * part, hi = lo + part < a.V ? lo + part : a.V;
  const uint64_t key = best_of<IO, BLOCK>(static_cast<const IO*>(a.target) + (row * (a.K + 1) + kept) * a.V,
                                   refused ? static_cast<const IO*>(a.draft) + (row * a.K + kept) * a.V : nullptr,
                                   a.noise + row * a.V, lo, hi, lds);
  if (parts == 1) finish_row<IO, BLOCK>(a, row, kept, refused, key, lds);
  else if (threadIdx.x == 0) keys[blockIdx.x] = key;
}

template <typename IO>
__global__ __launch_bounds__(kBlock) void verify_join_kernel(VerifyArgs a, int parts, const uint64_t* keys) {
  __shared__ uint64_t lds[kBlock / 64];
  const int64_t row = blockIdx.x;
  uint64_t key = 0;
  for (int s = threadIdx.x; s < parts; s += kBlock) {
    const uint64_t k = keys[row * parts + s];
    key = k > key ? k : key;
  }
  key = block_max<kBlock>(key, lds);
  const int64_t count = count_of(a, row), kept = kept_drafts<IO>(a, row, count);
  finish_row<IO, kBlock>(a, row, kept, kept < count, key, lds);
}

bool alone(int64_t rows, int64_t vocab) { return rows <= kUnits && vocab > kPart && vocab <= kAlone; }

int parts_of(int64_t rows, int64_t vocab) {
  if (alone(rows, vocab)) return 1;
  int64_t n = (kFill + rows - 1) / (rows < 1 ? 1 : rows);
  const int64_t most = (vocab + kPart - 1) / kPart;
  n = n < most ? n : most;
  return (int)(n < 1 ? 1 : n);
}

template <typename IO>
hipError_t launch_t(const VerifyArgs& a, uint64_t* keys, hipStream_t s) {
  const int parts = parts_of(a.rows, a.V);
  const int64_t part = ((a.V + parts - 1) / parts + V - 1) / V * V;
  if (alone(a.rows, a.V))
    hipLaunchKernelGGL((verify_kernel<IO, kWide>), dim3((unsigned)a.rows), dim3(kWide), 0, s, a, 1, part, keys);
  else
    hipLaunchKernelGGL((verify_kernel<IO, kBlock>), dim3((unsigned)(a.rows * parts)), dim3(kBlock), 0, s, a, parts, part,
                       keys);
  if (parts > 1)
    hipLaunchKernelGGL((verify_join_kernel<IO>), dim3((unsigned)a.rows), dim3(kBlock), 0, s, a, parts, keys);
  return hipGetLastError();
}

}  // namespace

size_t verify_ws_bytes(int64_t rows, int64_t vocab) {
  const int parts = parts_of(rows, vocab);
  return parts > 1 ? (size_t)rows * parts * sizeof(uint64_t) : 0;
}

hipError_t launch_verify(const VerifyArgs& a, int io, void* workspace, hipStream_t s) {
  uint64_t* keys = static_cast<uint64_t*>(workspace);
  return io == kIoBF16 ? launch_t<uint16_t>(a, keys, s) : launch_t<float>(a, keys, s);
}

}  // namespace s6
