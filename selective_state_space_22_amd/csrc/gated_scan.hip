// gated_scan.hip -- the gated linear recurrence of include/mamba_mi355x_lm.h:
// forward over sequences, backward, and the one-token step.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "gated_device.h"
#include "lm_internal.h"

namespace s6 {
namespace {

// ---------------------------------------------------------------- rows of a wave's tokens
//
// A lane owns C channels (two where bf16 pairs share a 32-bit word, else one).  The rows of
// a wave's tokens are reached through bounds-checked buffer resources: a load outside (a
// token past the end, a lane past the last channel, an absent tensor of 0 bytes) returns 0
// and a store is dropped, with no branch around either.

constexpr int kBufferDword3 = 0x00027000;   // raw, 32-bit data format
constexpr int kStreamed = 2;                // non-temporal: every row is used once (2 to 4% of the time)
constexpr uint32_t kNowhere = 0x80000000u;  // a lane offset beyond every resource here

// One resource of n rows, row i by the scalar offset at(i).  A token past the end gets the
// offset n * stride, the resource's size, so that nothing of it is in range (the offset
// never exceeds the size).
struct Rows {
  __amdgpu_buffer_rsrc_t r;
  uint32_t stride;  // 0 where the tensor is absent (and the resource empty)
  int n;
  __device__ __forceinline__ Rows(const void* p, size_t skip, uint32_t stride_, int n_)
      : r(__builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(static_cast<const uint8_t*>(p) + (p ? skip : 0)),
                                            (short)0, (int)(p ? n_ * stride_ : 0u), kBufferDword3)),
        stride(p ? stride_ : 0u),
        n(n_) {}
  __device__ __forceinline__ uint32_t at(int i) const { return (uint32_t)(i < n ? i : n) * stride; }
};

// C channels of one token as loaded, and as numbers.
template <typename IO, int C>
__device__ __forceinline__ uint32_t fetch(const Rows& w, int i, uint32_t off) {
  if constexpr (sizeof(IO) * C == 2) return (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(w.r, off, w.at(i), kStreamed) << 16;
  else return __builtin_amdgcn_raw_buffer_load_b32(w.r, off, w.at(i), kStreamed);
}
template <int C>
__device__ __forceinline__ float value(uint32_t raw, int c) {
  return C == 2 && c == 0 ? bf16_lo(raw) : C == 2 ? bf16_hi(raw) : __uint_as_float(raw);
}
template <typename IO, int C>
__device__ __forceinline__ void put(const Rows& w, int i, uint32_t off, const float (&v)[C]) {
  if constexpr (C == 2) __builtin_amdgcn_raw_buffer_store_b32(f32x2_to_bf16(v[0], v[1]), w.r, off, w.at(i), kStreamed);
  else if constexpr (sizeof(IO) == 2) __builtin_amdgcn_raw_buffer_store_b16(f32_to_bf16(v[0]), w.r, off, w.at(i), kStreamed);
  else __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[0]), w.r, off, w.at(i), kStreamed);
}
template <typename IO>
__device__ __forceinline__ void put1(const Rows& w, int i, uint32_t off, float v) {
  const float a[1] = {v};
  put<IO, 1>(w, i, off, a);
}
template <int C>
__device__ __forceinline__ void put_state(const Rows& w, int i, uint32_t off, const float (&v)[C]) {
#pragma unroll
  for (int c = 0; c < C; ++c) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[c]), w.r, off + 4 * c, w.at(i), 0);
}

// Has a value formed at this point.  A token's raw values are taken when its turn comes and
// its results are fixed when it ends: otherwise the compiler starts on all tokens at once,
// or moves the forming of a result to its use beyond the look back, where everything it is
// formed from stays alive, and spills either way.
template <typename V>
__device__ __forceinline__ void fix(V& v) { asm volatile("" : "+v"(v)); }

// ---------------------------------------------------------------- the split over the sequence
//
// A workgroup has W waves that compute (fewer for a short sequence) and one that keeps the
// order.  It takes
// work items of 64 * C channels and some tokens per computing wave (wave after wave).
// Each wave scans its tokens from zero and leaves their affine map h -> A h + H in LDS.
// The other wave publishes the map of all of them, looks back at its predecessors' to one
// that depends on nothing older, takes the state through them, publishes the end state as
// such a map (A = 0) in the place of the first, and hands the state that enters to the
// others, which run their recurrence from decays and inputs still in registers: every
// input is read once.  Meanwhile the computing waves have the next item's loads in flight;
// a wave's loads return in order, which is why one that looks back must not load.
//
// Which of a level's two maps a reader meets depends on timing, so maps of levels are
// never composed with each other: the state is taken through them one by one, oldest
// first, which gives the bits that the chain of end states has wherever it starts.
//
// A published {A, H} is one 64-bit word and its own flag: the workspace starts as all
// ones, and an A of all ones is a NaN that no publisher writes (its NaNs are replaced by
// the standard one), so a reader needs no separate flag and no cache write-back.  Items
// are handed out by a counter, level after level.  A workgroup holds one item that it
// works on and the next one that it only loads; the unfinished item that was handed out
// first is one that its holder works on (the holder's present item came before), and it
// waits for nothing unfinished: every wait ends.
// A decay of exactly 0 drops the older state, whatever it is; only a reset has one (run_decay).

constexpr int kRead = 4;      // predecessors read at once
// Predecessors looked back at; the last of them is waited for to its end.  Two channels a
// lane is a plan of many blocks, so that few levels of one are in flight.
template <int C>
constexpr int kDepth = C == 2 ? 32 : 128;
constexpr uint32_t kEmpty = 0xffffffffu;

// x / d for x < 2^31 by a multiplication: m = floor(2^(31 + s) / d) + 1, 2^s >= d.
struct Divisor {
  uint32_t m;
  int s;
  __device__ __forceinline__ uint32_t of(uint32_t x) const { return (uint32_t)(((uint64_t)x * m) >> (31 + s)); }
};

struct Link {
  unsigned long long* map;  // (levels, blocks, 64 * C) of {A, H}
  uint32_t* ticket;
  uint32_t* err;
  uint32_t spin_limit;
  int levels, blocks, row_blocks;
  Divisor by_blocks, by_row;
};

template <int C, int W>
struct ScanShared {
  float S[W][64 * C], A[W][64 * C], H[W][64 * C];  // the waves' log decays and maps
  float in[64 * C];                                    // the state that enters the item
  float backA[kDepth<C>][64 * C], backH[kDepth<C>][64 * C];  // the predecessors' maps, nearest first
  uint32_t first, item;                                // the workgroup's first item, and its next one
};

__device__ __forceinline__ uint32_t published(float v) { return v != v ? 0x7fc00000u : __float_as_uint(v); }
__device__ __forceinline__ float apply(float A, float H, float h) { return A == 0.0f ? H : __builtin_fmaf(A, h, H); }

// (A, H) of the waves before `wave`, in order.  A wave with a reset (S of -inf) starts A anew: added
// to it, a NaN gate of the waves before would pass the reset.
template <int C, int W>
__device__ __forceinline__ void maps_before(int wave, uint32_t lane, float (&A)[C], float (&H)[C],
                                            const ScanShared<C, W>& sm) {
#pragma unroll
  for (int c = 0; c < C; ++c) A[c] = 0.0f, H[c] = 0.0f;
#pragma unroll
  for (int w = 0; w < W; ++w)
    if (w < wave) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        H[c] = apply(sm.A[w][lane * C + c], sm.H[w][lane * C + c], H[c]);
        const float S = sm.S[w][lane * C + c];
        A[c] = S == -__builtin_inff() ? S : A[c] + S;
      }
    }
#pragma unroll
  for (int c = 0; c < C; ++c) A[c] = run_decay(A[c]);
}

// Leaves a wave's map in sm.
template <int C, int W>
__device__ __forceinline__ void leave_map(int wave, uint32_t lane, const float (&S)[C], const float (&H)[C],
                                          ScanShared<C, W>& sm) {
#pragma unroll
  for (int c = 0; c < C; ++c) {
    sm.S[wave][lane * C + c] = S[c];
    sm.A[wave][lane * C + c] = run_decay(S[c]);
    sm.H[wave][lane * C + c] = H[c];
  }
}

template <int C>
__device__ __forceinline__ void read_map(const Link& k, int level, int blk, uint32_t lane, unsigned long long (&m)[C]) {
  const unsigned long long* from = k.map + ((size_t)level * k.blocks + blk) * 64 * C;
#pragma unroll
  for (int c = 0; c < C; ++c) m[c] = __hip_atomic_load(from + (lane * C + c), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <int C>
__device__ __forceinline__ void write_map(const Link& k, int level, int blk, uint32_t lane, const float (&A)[C],
                                          const float (&H)[C]) {
  unsigned long long* to = k.map + ((size_t)level * k.blocks + blk) * 64 * C;
#pragma unroll
  for (int c = 0; c < C; ++c)
    __hip_atomic_store(to + (lane * C + c), published(A[c]) | (unsigned long long)published(H[c]) << 32,
                       __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// State entering `level` of a block (state: the one entering level 0, on entry).
template <int C, int W>
__device__ __forceinline__ void look_back(const Link& k, int level, int blk, uint32_t lane, float (&state)[C],
                                          ScanShared<C, W>& sm) {
  int slot = 0;
  bool closed = level == 0;
  while (!closed) {
    unsigned long long m[kRead][C];
#pragma unroll
    for (int j = 0; j < kRead; ++j) {
      const int e = level - 1 - slot - j;
      read_map<C>(k, e > 0 ? e : 0, blk, lane, m[j]);
    }
#pragma unroll
    for (int j = 0; j < kRead; ++j) {
      const int e = level - 1 - slot;
      if (closed) continue;
      if (e < 0) {  // before level 0: the initial state
        closed = true;
        continue;
      }
      for (uint32_t polls = 0;; ++polls) {
        bool there = true, end = true;
#pragma unroll
        for (int c = 0; c < C; ++c) there &= (uint32_t)m[j][c] != kEmpty, end &= __uint_as_float((uint32_t)m[j][c]) == 0.0f;
        closed = __all(end);
        if (closed || (__all(there) && slot + 1 < kDepth<C>)) break;
        if (polls >= k.spin_limit) {  // never expected: report, and go on from NaN
          if (lane == 0) __hip_atomic_store(k.err, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
          for (int c = 0; c < C; ++c) m[j][c] = 0x7fc0000000000000ull;
          closed = true;
          break;
        }
        __builtin_amdgcn_s_sleep(1);
        read_map<C>(k, e, blk, lane, m[j]);
      }
      if (closed) {
#pragma unroll
        for (int c = 0; c < C; ++c) state[c] = __uint_as_float((uint32_t)(m[j][c] >> 32));
      } else {
#pragma unroll
        for (int c = 0; c < C; ++c) {
          sm.backA[slot][lane * C + c] = __uint_as_float((uint32_t)m[j][c]);
          sm.backH[slot][lane * C + c] = __uint_as_float((uint32_t)(m[j][c] >> 32));
        }
        ++slot;
      }
    }
  }
#pragma unroll 8
  for (int j = slot - 1; j >= 0; --j) {
#pragma unroll
    for (int c = 0; c < C; ++c) state[c] = apply(sm.backA[j][lane * C + c], sm.backH[j][lane * C + c], state[c]);
  }
}

// Where an item's wave stands.  REVERSE: level 0 is the end of the sequence and the first
// wave holds a level's last tokens.
struct Place {
  int level, blk, n;  // n: tokens of the wave's run inside the sequence
  int64_t bt, run, t0, row;
  uint32_t d;    // the lane's first channel (0 where it is past the last)
  uint32_t off;  // the same as an offset in elements, or kNowhere
  template <int T, int C, bool REVERSE>
  __device__ __forceinline__ void set(const Link& k, uint32_t item, bool real, int wave, uint32_t lane, int64_t L,
                                      int64_t D) {
    const int waves = (int)(blockDim.x >> 6) - 1;
    level = (int)k.by_blocks.of(item);
    blk = (int)(item - (uint32_t)level * (uint32_t)k.blocks);
    const uint32_t b = k.by_row.of((uint32_t)blk);
    bt = b;
    const uint32_t c = ((uint32_t)(blk - b * k.row_blocks) * 64 + lane) * C;
    const bool act = c < (uint32_t)D;
    d = act ? c : 0;
    off = act ? c : kNowhere;
    run = REVERSE ? (int64_t)(k.levels - 1 - level) * waves + (waves - 1 - wave) : (int64_t)level * waves + wave;
    const int64_t left = real ? L - run * T : 0;
    n = __builtin_amdgcn_readfirstlane((int)(left < T ? (left > 0 ? left : 0) : T));
    if (n == 0) run = 0;  // (nothing is read or written there)
    t0 = run * T;
    row = bt * L + t0;
  }
};

template <typename IO>
__device__ __forceinline__ uint32_t bytes(uint32_t off) { return off == kNowhere ? kNowhere : off * (uint32_t)sizeof(IO); }

// The items of a workgroup, one after the other (one level: from the grid, no order).
__device__ __forceinline__ uint32_t take_item(const Link& k, uint32_t item) {
  if (k.levels == 1) return item == kEmpty ? blockIdx.x : item + gridDim.x;
  const uint32_t t = (threadIdx.x & 63) == 0 ? atomicAdd(k.ticket, 1u) : 0u;
  return __builtin_amdgcn_readfirstlane(t);
}

// The order-keeping wave's part, item after item.  init: (batch, D) states entering level 0,
// or null (zero); end_state: (batch, D) states leaving the last level, or null.  SUMS: after
// each item, the sum over the waves of each lane's value in sums goes to pl.
template <typename IO, int T, int C, int W, bool REVERSE, bool SUMS>
__device__ __forceinline__ void keep_order(const Link& k, uint32_t item, uint32_t lane, int64_t L, int64_t D,
                                           const float* init, float* end_state, float* pl, const float (*sums)[64],
                                           ScanShared<C, W>& sm) {
  const int waves = (int)(blockDim.x >> 6) - 1;
  const uint32_t items = (uint32_t)k.levels * (uint32_t)k.blocks, sstride = (uint32_t)D * 4;
  uint32_t last_off = kNowhere;
  size_t last_row = 0;
  bool more = true, first = true;
  while (true) {
    const uint32_t next = more ? take_item(k, item) : kEmpty;
    Place p;
    if (more) {
      p.set<T, C, REVERSE>(k, item, true, 0, lane, L, D);
      if (lane == 0) sm.item = next;
    }
    float state[C];
#pragma unroll
    for (int c = 0; c < C; ++c) state[c] = more && init && p.level == 0 ? init[p.bt * D + p.d + c] : 0.0f;
    __syncthreads();  // the waves' maps, and the sums of the item before
    if (SUMS && !first) {
      float v = 0.0f;
      for (int w = 0; w < waves; ++w) v += sums[w][lane];
      const float vs[1] = {v};
      put_state<1>(Rows(pl, last_row * sstride, sstride, 1), 0, last_off, vs);
    }
    if (!more) return;
    float A[C], H[C];
    maps_before<C, W>(waves, lane, A, H, sm);
    if (p.level > 0 && p.level + 1 < k.levels) write_map<C>(k, p.level, p.blk, lane, A, H);
    look_back<C, W>(k, p.level, p.blk, lane, state, sm);
    float end[C], none[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      sm.in[lane * C + c] = state[c];
      end[c] = apply(A[c], H[c], state[c]);  // the bits that a reader of the level's map gets
      none[c] = 0.0f;
    }
    if (p.level + 1 < k.levels) write_map<C>(k, p.level, p.blk, lane, none, end);
    else if (end_state) put_state<C>(Rows(end_state, (size_t)p.bt * sstride, sstride, 1), 0, bytes<float>(p.off), end);
    __syncthreads();  // the state that enters
    first = false;
    if (SUMS) last_row = (size_t)(p.bt * k.levels + p.level), last_off = bytes<float>(p.off);
    more = next < items;
    if (!more && !SUMS) return;
    item = next;
  }
}

__global__ __launch_bounds__(256) void gated_clear_kernel(uint32_t* ticket, uint32_t* words, int64_t n) {
  if (blockIdx.x == 0 && threadIdx.x == 0) __hip_atomic_store(ticket, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    __hip_atomic_store(words + i, kEmpty, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// ---------------------------------------------------------------- forward

// Tokens per wave: 16 elements a lane (decays and inputs, 32 registers, and the next run's
// raw values beside them) is what 128 registers hold.
template <int C>
constexpr int kTokF = 16 / C;
constexpr int kWavesF = 15;  // computing waves

// A run as loaded (z, which is needed last, is loaded when the run's turn comes).
template <typename IO, int C, bool HASR, int T>
struct FwdRaw {
  uint32_t ra[T], rx[T], u[T], reset;
  float lam[C];
  __device__ __forceinline__ void load(const GatedArgs& g, const Place& p, uint32_t lane) {
    const uint32_t stride = (uint32_t)g.D * sizeof(IO), off = bytes<IO>(p.off);
    const size_t skip = (size_t)p.row * stride;
    const Rows r_ra(g.ra, skip, stride, p.n), r_rx(g.rx, skip, stride, p.n), r_u(g.u, skip, stride, p.n);
#pragma unroll
    for (int i = 0; i < T; ++i) {
      ra[i] = fetch<IO, C>(r_ra, i, off);
      rx[i] = fetch<IO, C>(r_rx, i, off);
      u[i] = fetch<IO, C>(r_u, i, off);
    }
    if (HASR) reset = (int)lane < p.n ? g.reset[p.row + lane] : 0;
#pragma unroll
    for (int c = 0; c < C; ++c) lam[c] = g.lam[p.d + c];
  }
};

// Bound by memory: every input and the output pass once, and nothing else of that size.
// (4, 4096, 5120) bf16 with z, 839 MB: 206 us a call, 4.1 TB/s, where the same loads and
// stores without the arithmetic and the looking back take 179 and a copy of the bytes 146.
// With decays from 0.5 to 0.999 (two waves in five take the exponential) 213 us, with channels that
// all forget within a token 219.
// (1, 1048576, 256) fp32, 4.3 GB, 4 blocks of channels, so all of the parallelism is in the
// split: 720 us, 6.0 TB/s.
template <typename IO, int C, bool HASZ, bool HASR>
__global__ __launch_bounds__(64 * (kWavesF + 1), 4) void gated_fwd_kernel(GatedArgs g, Link k) {
  constexpr int T = kTokF<C>, W = kWavesF;
  __shared__ ScanShared<C, W> sm;
  const uint32_t lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = (int)(blockDim.x >> 6) - 1;
  const uint32_t items = (uint32_t)k.levels * (uint32_t)k.blocks;
  if (wave == waves) {
    const uint32_t first = take_item(k, kEmpty);
    if (lane == 0) sm.first = first;
  }
  __syncthreads();
  uint32_t item = __builtin_amdgcn_readfirstlane(sm.first);
  if (item >= items) return;
  if (wave == waves) {
    keep_order<IO, T, C, W, false, false>(k, item, lane, g.L, g.D, g.h0, nullptr, nullptr, nullptr, sm);
    return;
  }
  const int64_t nst = (g.L + kGatedStateChunk - 1) / kGatedStateChunk;
  const uint32_t stride = (uint32_t)g.D * sizeof(IO), sstride = (uint32_t)g.D * 4;
  Place p;
  p.set<T, C, false>(k, item, true, wave, lane, g.L, g.D);
  FwdRaw<IO, C, HASR, T> raw;
  raw.load(g, p, lane);
  while (true) {
    const uint32_t off = bytes<IO>(p.off), soff = bytes<float>(p.off);
    uint32_t z[T];
    if (HASZ) {
      const Rows r_z(g.z, (size_t)p.row * stride, stride, p.n);
#pragma unroll
      for (int i = 0; i < T; ++i) z[i] = fetch<IO, C>(r_z, i, off);
    }
    float kappa[C], S[C], H[C], a[T][C], b[T][C];
    bool slow = true;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      kappa[c] = g.c * softplus(raw.lam[c]);
      slow &= kappa[c] < kNearExp;
      S[c] = 0.0f, H[c] = 0.0f;
    }
    slow = __all(slow);
    const uint32_t reset = HASR ? (uint32_t)__ballot(raw.reset != 0) : 0;
    // Decays and inputs, and the run's map from zero.  A token past the end has loaded
    // zeros: it adds nothing, and no token after it is kept.
#pragma unroll
    for (int i = 0; i < T; ++i) {
      const bool cut = HASR && ((reset >> i) & 1);
      fix(raw.ra[i]), fix(raw.rx[i]), fix(raw.u[i]);
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float l;
        gated_token(value<C>(raw.ra[i], c), value<C>(raw.rx[i], c), value<C>(raw.u[i], c), kappa[c], slow, cut,
                    a[i][c], b[i][c], l);
        fix(a[i][c]), fix(b[i][c]);
        H[c] = cut ? b[i][c] : __builtin_fmaf(a[i][c], H[c], b[i][c]);
        S[c] = cut ? -__builtin_inff() : S[c] + l;
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    leave_map<C, W>(wave, lane, S, H, sm);
    __syncthreads();
    const uint32_t next = __builtin_amdgcn_readfirstlane(sm.item);
    const bool more = next < items;  // (else the loads below are of no tokens)
    Place q;
    q.set<T, C, false>(k, more ? next : item, more, wave, lane, g.L, g.D);
    raw.load(g, q, lane);
    float Ap[C], Hp[C], h[C];
    maps_before<C, W>(wave, lane, Ap, Hp, sm);
    __syncthreads();
#pragma unroll
    for (int c = 0; c < C; ++c) h[c] = apply(Ap[c], Hp[c], sm.in[lane * C + c]);

    // the recurrence from the state that enters
    const Rows r_out(g.out, (size_t)p.row * stride, stride, p.n);
    const Rows r_st(g.states, (size_t)(p.bt * nst + p.t0 / kGatedStateChunk) * sstride, sstride,
                    (p.n + kGatedStateChunk - 1) / kGatedStateChunk);
    const int last_token = g.last && p.t0 + T >= g.L ? p.n - 1 : -1;
    const Rows r_last(g.last, (size_t)p.bt * sstride, sstride, 1);
#pragma unroll
    for (int i = 0; i < T; ++i) {
      const bool cut = HASR && ((reset >> i) & 1);
      if (i % kGatedStateChunk == 0) put_state<C>(r_st, i / kGatedStateChunk, soff, h);
      if (HASZ) fix(z[i]);
      float o[C];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        h[c] = cut ? b[i][c] : __builtin_fmaf(a[i][c], h[c], b[i][c]);
        o[c] = HASZ ? h[c] * silu(value<C>(z[i], c)) : h[c];
      }
      put<IO, C>(r_out, i, off, o);
      if (i == last_token) put_state<C>(r_last, 0, soff, h);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (!more) return;
    p = q;
    item = next;
  }
}

// seqlen 0: the final state is the initial one.
__global__ __launch_bounds__(256) void gated_copy_state_kernel(const float* h0, float* last, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    last[i] = h0 ? h0[i] : 0.0f;
}

// ---------------------------------------------------------------- backward
//
// With G_t = dL/dh_t, the gradient that leaves token t for the one before is
// c_t = a_t (dy_t + c_{t+1}), dy = dout SiLU(z): the same kind of scan, from the last
// token to the first, split in the same way (level 0 is the end of the sequence).  A
// wave owns the 8 tokens after one saved state, so the states are recomputed in
// registers with no exchange; what does not depend on G (dz, and the factors that G
// multiplies) is formed on the way forward through the 8 tokens:
//   du = G s sx,  dgate_x = G b (1 - sx),  e = G (a h_{t-1} l - q sx u),
//   dgate_a = e (1 - sa),  dlam = dlam_factor * sum e.

constexpr int kTokB = kGatedStateChunk;  // tokens per wave
// Computing waves: two workgroups of 7 share a compute unit, which overlaps them better
// where there are blocks enough ((8, 2048, 1536) bf16, 192 blocks: 128 us against 137 with
// one of 15).  With few blocks more levels of one are in flight, and longer levels mean
// less looking back ((3, 1537, 1101) fp32, 54 blocks: 48 us with 15 and 56 with 7).
constexpr int kWavesB = 7, kWavesBFew = 15;
constexpr int64_t kFewBlocks = 128;

template <typename IO, bool HASZ, bool HASR, int T>
struct BwdRaw {
  uint32_t ra[T], rx[T], u[T], z[T], dout[T], reset;
  float lam, dlast, h;
  int last_token;  // the run's token where dlast enters, -1: none
  __device__ __forceinline__ void load(const GatedBwdArgs& g, const Place& p, uint32_t lane) {
    const GatedArgs& f = g.f;
    const uint32_t stride = (uint32_t)f.D * sizeof(IO), off = bytes<IO>(p.off);
    const size_t skip = (size_t)p.row * stride;
    const Rows r_ra(f.ra, skip, stride, p.n), r_rx(f.rx, skip, stride, p.n), r_u(f.u, skip, stride, p.n),
        r_do(g.dout, skip, stride, p.n);
#pragma unroll
    for (int i = 0; i < T; ++i) {
      ra[i] = fetch<IO, 1>(r_ra, i, off);
      rx[i] = fetch<IO, 1>(r_rx, i, off);
      u[i] = fetch<IO, 1>(r_u, i, off);
      dout[i] = fetch<IO, 1>(r_do, i, off);
    }
    if (HASZ) {
      const Rows r_z(f.z, skip, stride, p.n);
#pragma unroll
      for (int i = 0; i < T; ++i) z[i] = fetch<IO, 1>(r_z, i, off);
    }
    if (HASR) reset = (int)lane < p.n ? f.reset[p.row + lane] : 0;
    lam = f.lam[p.d];
    h = f.states[(p.bt * ((f.L + T - 1) / T) + p.run) * f.D + p.d];
    last_token = g.dlast && p.t0 + T >= f.L ? p.n - 1 : -1;
    dlast = last_token >= 0 ? g.dlast[p.bt * f.D + p.d] : 0.0f;
  }
};

// Reads five arrays and writes four, with 96 vector instructions to an element beside them.
// (8, 2048, 1536) bf16 with z and resets, 465 MB: 125 us, 3.7 TB/s (a copy: 81 us).  Odd widths
// leave rows of bf16 on 2-byte boundaries: forward and backward take 360 us with 1535 channels, 208
// with 1536.
template <typename IO, int W, bool HASZ, bool HASR>
__global__ __launch_bounds__(64 * (W + 1), 4) void gated_bwd_kernel(GatedBwdArgs g, Link k, float* pl) {
  constexpr int T = kTokB;
  const GatedArgs& f = g.f;
  __shared__ ScanShared<1, W> sm;
  __shared__ float sums[W][64];
  const uint32_t lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = (int)(blockDim.x >> 6) - 1;
  const uint32_t items = (uint32_t)k.levels * (uint32_t)k.blocks;
  if (wave == waves) {
    const uint32_t first = take_item(k, kEmpty);
    if (lane == 0) sm.first = first;
  }
  __syncthreads();
  uint32_t item = __builtin_amdgcn_readfirstlane(sm.first);
  if (item >= items) return;
  if (wave == waves) {
    keep_order<IO, T, 1, W, true, true>(k, item, lane, f.L, f.D, nullptr, g.dh0, pl, sums, sm);
    return;
  }
  const uint32_t stride = (uint32_t)f.D * sizeof(IO);
  Place p;
  p.set<T, 1, true>(k, item, true, wave, lane, f.L, f.D);
  BwdRaw<IO, HASZ, HASR, T> raw;
  raw.load(g, p, lane);
  while (true) {
    const float kappa = f.c * softplus(raw.lam);
    const bool slow = __all(kappa < kNearExp);
    // (past the end every token is a reset: whatever the state there is, its share of dlam is 0)
    const uint32_t reset = HASR ? ((uint32_t)__ballot(raw.reset != 0) | ~0u << p.n) & ((1u << T) - 1) : 0;
    const Rows r_dz(g.dz, (size_t)p.row * stride, stride, p.n);
    const uint32_t off = bytes<IO>(p.off);
    // The way forward.  A token past the end has loaded zeros: its gradient is 0 and
    // stays 0 up to the last token, where dlast enters.
    float a[T], dy[T], p1[T], p2[T], e0[T], oa[T], h = raw.h, S[1] = {0.0f}, H[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < T; ++i) {
      const bool cut = HASR && ((reset >> i) & 1);
      fix(raw.ra[i]), fix(raw.rx[i]), fix(raw.u[i]), fix(raw.dout[i]);
      if (HASZ) fix(raw.z[i]);
      const GatedGrad q = gated_grad(value<1>(raw.ra[i], 0), value<1>(raw.rx[i], 0), kappa, slow, cut);
      const float x = q.sx * value<1>(raw.u[i], 0), b = q.s * x;
      const float ah = cut ? 0.0f : q.a * h;
      h = ah + b;
      a[i] = q.a;
      p1[i] = q.s * q.sx;
      p2[i] = b * q.ox;
      e0[i] = __builtin_fmaf(ah, q.l, -q.q * x);
      oa[i] = q.oa;
      S[0] += q.l;
      dy[i] = value<1>(raw.dout[i], 0);
      if (HASZ) {
        float sz, dsz;
        silu_pair(value<1>(raw.z[i], 0), sz, dsz);
        put1<IO>(r_dz, i, off, dy[i] * h * dsz);
        dy[i] *= sz;
      }
      fix(a[i]), fix(p1[i]), fix(p2[i]), fix(e0[i]), fix(oa[i]), fix(dy[i]);
      __builtin_amdgcn_sched_barrier(0);
    }
    // (in whatever place: a NaN before the reset is in H, one behind it does not leave the run)
    if (HASR && reset != 0) S[0] = -__builtin_inff();
    if (raw.last_token >= 0) {
#pragma unroll
      for (int i = 0; i < T; ++i) dy[i] += i == raw.last_token ? raw.dlast : 0.0f;
    }
#pragma unroll
    for (int i = T - 1; i >= 0; --i) {
      const bool cut = HASR && ((reset >> i) & 1);
      H[0] = cut ? 0.0f : a[i] * (dy[i] + H[0]);
    }
    leave_map<1, W>(wave, lane, S, H, sm);
    __syncthreads();
    const uint32_t next = __builtin_amdgcn_readfirstlane(sm.item);
    const bool more = next < items;  // (else the loads below are of no tokens)
    Place q;
    q.set<T, 1, true>(k, more ? next : item, more, wave, lane, f.L, f.D);
    raw.load(g, q, lane);
    float Ap[1], Hp[1];
    maps_before<1, W>(wave, lane, Ap, Hp, sm);
    __syncthreads();
    float cg = apply(Ap[0], Hp[0], sm.in[lane]), sum = 0.0f;

    // the way back from the gradient that enters
    const Rows r_du(g.du, (size_t)p.row * stride, stride, p.n), r_drx(g.drx, (size_t)p.row * stride, stride, p.n),
        r_dra(g.dra, (size_t)p.row * stride, stride, p.n);
#pragma unroll
    for (int i = T - 1; i >= 0; --i) {
      const bool cut = HASR && ((reset >> i) & 1);
      const float G = dy[i] + cg;
      const float e = cut ? 0.0f : G * e0[i];
      sum += e;
      cg = cut ? 0.0f : a[i] * G;
      put1<IO>(r_du, i, off, G * p1[i]);
      put1<IO>(r_drx, i, off, G * p2[i]);
      put1<IO>(r_dra, i, off, e * oa[i]);
      __builtin_amdgcn_sched_barrier(0);
    }
    sums[wave][lane] = sum;
    if (!more) break;
    p = q;
    item = next;
  }
  __syncthreads();  // the order-keeping wave adds the last sums
}

// Column sums of `rows` consecutive rows of in (n, D) per blockIdx.y, each of four waves
// over a quarter of them in order; the last pass multiplies by the channel's factor.
__global__ __launch_bounds__(256) void gated_dlam_kernel(const float* in, const float* lam, float* out, int64_t n,
                                                         int64_t rows, int64_t D) {
  __shared__ float part_sum[4][64];
  const int64_t d = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63);
  const int wave = threadIdx.x >> 6;
  const int64_t quarter = (rows + 3) / 4, end = (blockIdx.y + 1) * rows < n ? (blockIdx.y + 1) * rows : n;
  const int64_t r0 = blockIdx.y * rows + wave * quarter;
  const int64_t r1 = r0 + quarter < end ? r0 + quarter : end;
  float s = 0.0f;
  if (d < D)
    for (int64_t i = r0; i < r1; ++i) s += in[i * D + d];
  part_sum[wave][threadIdx.x & 63] = s;
  __syncthreads();
  if (wave != 0 || d >= D) return;
  s = (s + part_sum[1][threadIdx.x]) + (part_sum[2][threadIdx.x] + part_sum[3][threadIdx.x]);
  out[blockIdx.y * D + d] = lam ? (n > 0 ? s * dlam_factor(lam[d]) : 0.0f) : s;
}

// ---------------------------------------------------------------- one token

// A thread to a channel, the forward's arithmetic: (256, 5120) bf16, 23.6 MB, 6 us in the
// kernel, 3.9 TB/s; (1, 2560) 2.9 us, a launch.
template <typename IO>
__global__ __launch_bounds__(256) void gated_step_kernel(GatedStepArgs g) {
  const int64_t d = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t bt = blockIdx.y;
  if (d >= g.D) return;
  const size_t i = (size_t)bt * g.D + d;
  const bool reset = g.reset && g.reset[bt] != 0;
  float a, b, l;
  gated_token(load_io((const IO*)g.ra, i), load_io((const IO*)g.rx, i), load_io((const IO*)g.u, i),
              g.c * softplus(g.lam[d]), false, reset, a, b, l);
  const float h = reset ? b : __builtin_fmaf(a, g.state[i], b);
  g.state[i] = h;
  store_io((IO*)g.out, i, g.z ? h * silu(load_io((const IO*)g.z, i)) : h);
}

size_t al256(size_t v) { return (v + 255) / 256 * 256; }

// How a sequence is cut: levels of waves * tok tokens (`waves` computing ones), blocks of 64 * vec channels.
struct GatedPlan {
  int vec, waves, row_blocks;
  int64_t levels, blocks;
  size_t words, bytes;  // workspace: the ticket in 256 bytes, then the map's words (none for one level)
};

GatedPlan plan_gated(int64_t batch, int64_t L, int64_t D, int tok, int vec, int waves) {
  GatedPlan p{};
  if (batch == 0 || L == 0 || D == 0) return p;
  p.vec = vec;
  p.row_blocks = (int)((D + 64 * vec - 1) / (64 * vec));
  p.blocks = batch * p.row_blocks;
  const int64_t runs = (L + tok - 1) / tok;
  p.waves = (int)std::min<int64_t>(runs, waves);
  p.levels = (runs + p.waves - 1) / p.waves;
  if (p.levels > 1) {
    const size_t n = (size_t)p.levels * p.blocks * 64 * vec;
    p.words = n * 2;
    p.bytes = 256 + al256(n * 8);
  }
  return p;
}

// The forward's plan: pairs of bf16 channels where rows stay 4-byte aligned and there are
// blocks enough that few levels of one are in flight (the look back is shallower there).
GatedPlan plan_gated_fwd(int64_t batch, int64_t L, int64_t D, int io) {
  const GatedPlan two = plan_gated(batch, L, D, kTokF<2>, 2, kWavesF);
  return io == kIoBF16 && D % 2 == 0 && two.blocks >= 64 ? two : plan_gated(batch, L, D, kTokF<1>, 1, kWavesF);
}

GatedPlan plan_gated_bwd_link(int64_t batch, int64_t L, int64_t D) {
  const GatedPlan p = plan_gated(batch, L, D, kTokB, 1, kWavesB);
  return p.blocks < kFewBlocks ? plan_gated(batch, L, D, kTokB, 1, kWavesBFew) : p;
}

Divisor divisor(int64_t d) {
  Divisor r{0, 0};
  while ((int64_t(1) << r.s) < d) ++r.s;
  r.m = (uint32_t)((uint64_t(1) << (31 + r.s)) / (uint64_t)d + 1);
  return r;
}

// Workgroups of a launch: as many as the chip's 256 compute units hold (more where they
// have fewer waves), each going from item to item.
unsigned grid_of(const GatedPlan& p) {
  return (unsigned)std::min<int64_t>(p.levels * p.blocks, 256 * 16 / (p.waves + 1));
}

// The link of a launch: clears the workspace's words (one level: nothing).
hipError_t prepare_link(const GatedPlan& p, void* ws, Link& k, hipStream_t st) {
  k = Link{};
  k.levels = (int)p.levels;
  k.blocks = (int)p.blocks;
  k.row_blocks = p.row_blocks;
  k.by_blocks = divisor(p.blocks);
  k.by_row = divisor(p.row_blocks);
  if (p.levels == 1) return hipSuccess;
  uint8_t* w = static_cast<uint8_t*>(ws);
  k.ticket = reinterpret_cast<uint32_t*>(w);
  k.map = reinterpret_cast<unsigned long long*>(w + 256);
  k.err = wait_status_ptr();
  if (k.err == nullptr) return hipErrorInvalidSymbol;
  k.spin_limit = (uint32_t)option(kOptSpinLimit);
  hipLaunchKernelGGL(gated_clear_kernel, dim3((unsigned)std::min<size_t>((p.words + 1023) / 1024, 4096)), dim3(256), 0,
                     st, k.ticket, reinterpret_cast<uint32_t*>(w + 256), (int64_t)p.words);
  return hipGetLastError();
}

size_t states_bytes(int64_t batch, int64_t L, int64_t D) {
  return al256((size_t)batch * ((L + kGatedStateChunk - 1) / kGatedStateChunk) * D * 4);
}

template <typename IO, int C>
auto* pick_fwd(const GatedArgs& a) {
  return a.z ? (a.reset ? gated_fwd_kernel<IO, C, true, true> : gated_fwd_kernel<IO, C, true, false>)
             : (a.reset ? gated_fwd_kernel<IO, C, false, true> : gated_fwd_kernel<IO, C, false, false>);
}
template <typename IO, int W>
auto* pick_bwd(const GatedArgs& a) {
  return a.z ? (a.reset ? gated_bwd_kernel<IO, W, true, true> : gated_bwd_kernel<IO, W, true, false>)
             : (a.reset ? gated_bwd_kernel<IO, W, false, true> : gated_bwd_kernel<IO, W, false, false>);
}

}  // namespace

// Work items are counted in 32 bits.
bool gated_fits(int64_t batch, int64_t L, int64_t D) {
  const GatedPlan p = plan_gated(batch, L, D, kTokB, 1, kWavesB);
  return p.levels < (int64_t(1) << 31) && p.blocks < (int64_t(1) << 31) &&
         (double)p.levels * (double)p.blocks < 2147483648.0;
}

size_t gated_fwd_ws_bytes(int64_t batch, int64_t L, int64_t D, int io) {
  return plan_gated_fwd(batch, L, D, io).bytes;
}

hipError_t launch_gated_fwd(const GatedArgs& a, int io, void* ws, hipStream_t st) {
  if (a.L == 0) {
    const int64_t n = a.batch * a.D;
    if (a.last) hipLaunchKernelGGL(gated_copy_state_kernel, dim3((unsigned)std::min<int64_t>((n + 255) / 256, 65536)),
                                   dim3(256), 0, st, a.h0, a.last, n);
    return hipGetLastError();
  }
  const GatedPlan p = plan_gated_fwd(a.batch, a.L, a.D, io);
  Link k;
  const hipError_t e = prepare_link(p, ws, k, st);
  if (e != hipSuccess) return e;
  const dim3 grid(grid_of(p)), block(64 * (p.waves + 1));
  auto* kernel = p.vec == 2 ? pick_fwd<uint16_t, 2>(a) : io == kIoBF16 ? pick_fwd<uint16_t, 1>(a) : pick_fwd<float, 1>(a);
  hipLaunchKernelGGL(kernel, grid, block, 0, st, a, k);
  return hipGetLastError();
}

namespace {

// Workspace of the backward: the link's words (the forward's too, where it has to be
// run for the states: first, in the same place), then the partial sums of dlam in two
// stages, then the states.
struct GatedBwdPlan {
  GatedPlan link;
  int64_t rows, stages;  // rows of the first sums, and per second sum
  size_t off_sum, off_sum2, off_states, bytes;
};

GatedBwdPlan plan_gated_bwd(int64_t batch, int64_t L, int64_t D, int io) {
  GatedBwdPlan p{};
  if (batch == 0 || D == 0 || L == 0) return p;
  p.link = plan_gated_bwd_link(batch, L, D);
  const int64_t n = batch * p.link.levels;
  p.rows = std::max<int64_t>(64, (n + 255) / 256);
  p.stages = (n + p.rows - 1) / p.rows;
  p.off_sum = al256(std::max(p.link.bytes, plan_gated_fwd(batch, L, D, io).bytes));
  p.off_sum2 = p.off_sum + al256((size_t)n * D * 4);
  p.off_states = p.off_sum2 + al256((size_t)p.stages * D * 4);
  p.bytes = p.off_states + states_bytes(batch, L, D);
  return p;
}

// Copies the final gradient to dh0 and zeros dlam where there are no tokens.
hipError_t empty_bwd(const GatedBwdArgs& a, hipStream_t st) {
  const GatedArgs& f = a.f;
  const int64_t n = f.batch * f.D;
  if (a.dh0 && n > 0)
    hipLaunchKernelGGL(gated_copy_state_kernel, dim3((unsigned)std::min<int64_t>((n + 255) / 256, 65536)), dim3(256), 0,
                       st, a.dlast, a.dh0, n);
  hipLaunchKernelGGL(gated_copy_state_kernel, dim3((unsigned)((f.D + 255) / 256)), dim3(256), 0, st,
                     (const float*)nullptr, a.dlam, f.D);
  return hipGetLastError();
}

}  // namespace

size_t gated_bwd_ws_bytes(int64_t batch, int64_t L, int64_t D, int io) {
  return plan_gated_bwd(batch, L, D, io).bytes;
}

hipError_t launch_gated_bwd(const GatedBwdArgs& a, int io, void* ws, hipStream_t st) {
  const GatedArgs& f = a.f;
  if (f.batch == 0 || f.L == 0) return empty_bwd(a, st);
  const GatedBwdPlan p = plan_gated_bwd(f.batch, f.L, f.D, io);
  uint8_t* w = static_cast<uint8_t*>(ws);
  GatedBwdArgs g = a;
  hipError_t e;
  if (!f.states) {
    GatedArgs s = f;
    s.out = nullptr;
    s.last = nullptr;
    s.z = nullptr;
    s.states = reinterpret_cast<float*>(w + p.off_states);
    if ((e = launch_gated_fwd(s, io, ws, st)) != hipSuccess) return e;
    g.f.states = s.states;
  }
  Link k;
  if ((e = prepare_link(p.link, ws, k, st)) != hipSuccess) return e;
  float* pl = reinterpret_cast<float*>(w + p.off_sum);
  float* pl2 = reinterpret_cast<float*>(w + p.off_sum2);
  const dim3 grid(grid_of(p.link)), block(64 * (p.link.waves + 1));
  const bool few = p.link.blocks < kFewBlocks;
  auto* kernel = io == kIoBF16 ? (few ? pick_bwd<uint16_t, kWavesBFew>(f) : pick_bwd<uint16_t, kWavesB>(f))
                               : (few ? pick_bwd<float, kWavesBFew>(f) : pick_bwd<float, kWavesB>(f));
  hipLaunchKernelGGL(kernel, grid, block, 0, st, g, k, pl);
  const int64_t n = f.batch * p.link.levels;
  const unsigned cols = (unsigned)((f.D + 63) / 64);
  if (p.stages > 1) {
    hipLaunchKernelGGL(gated_dlam_kernel, dim3(cols, (unsigned)p.stages), dim3(256), 0, st, pl, (const float*)nullptr,
                       pl2, n, p.rows, f.D);
    hipLaunchKernelGGL(gated_dlam_kernel, dim3(cols), dim3(256), 0, st, pl2, f.lam, a.dlam, p.stages, p.stages, f.D);
  } else {
    hipLaunchKernelGGL(gated_dlam_kernel, dim3(cols), dim3(256), 0, st, pl, f.lam, a.dlam, n, n, f.D);
  }
  return hipGetLastError();
}

hipError_t launch_gated_step(const GatedStepArgs& a, int io, hipStream_t st) {
  const dim3 grid((unsigned)((a.D + 255) / 256), (unsigned)a.batch);
  if (io == kIoBF16) hipLaunchKernelGGL(gated_step_kernel<uint16_t>, grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL(gated_step_kernel<float>, grid, dim3(256), 0, st, a);
  return hipGetLastError();
}

}  // namespace s6
