// gated_scan.hip -- the gated linear recurrence of include/mamba_mi355x_lm.h:
// forward over sequences, backward, and the one-token step.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "gated_device.h"
#include "lm_internal.h"

namespace s6 {
namespace {

// ---------------------------------------------------------------- loads and stores of C channels
//
// The rows of a wave's tokens are reached through bounds-checked buffer resources: a
// load outside (a token past the end, a lane past the last channel, an absent tensor
// of 0 bytes) returns 0 and a store is dropped, with no branch around either.

using Buffer = __amdgpu_buffer_rsrc_t;
constexpr int kBufferDword3 = 0x00027000;  // raw, 32-bit data format
constexpr uint32_t kNowhere = 0x80000000u;  // an offset beyond every resource here

__device__ __forceinline__ Buffer bytes_of(const void* p, size_t skip, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(static_cast<const uint8_t*>(p) + (p ? skip : 0)), (short)0,
                                           (int)(p ? bytes : 0u), kBufferDword3);
}

// The rows of a wave's n tokens of one tensor: one resource of n rows, row i by the scalar
// offset at(i).  A token past the end gets the offset n * stride, the resource's size, so
// that nothing of it is in range (the offset never exceeds the size).
struct Rows {
  Buffer r;
  uint32_t stride;  // 0 where the tensor is absent (and the resource empty)
  int n;
  __device__ __forceinline__ Rows(const void* p, size_t skip, uint32_t stride_, int n_)
      : r(bytes_of(p, skip, n_ * stride_)), stride(p ? stride_ : 0u), n(n_) {}
  __device__ __forceinline__ uint32_t at(int i) const { return (uint32_t)(i < n ? i : n) * stride; }
};

// C channels of one token as loaded: bf16 pairs stay packed until they are used.
template <typename IO, int C>
__device__ __forceinline__ uint32_t fetch(const Rows& w, int i, uint32_t off) {
  if constexpr (sizeof(IO) * C == 2) return (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(w.r, off, w.at(i), 0);
  else return __builtin_amdgcn_raw_buffer_load_b32(w.r, off, w.at(i), 0);
}
template <typename IO>
__device__ __forceinline__ float part(uint32_t raw, int c) {
  if constexpr (sizeof(IO) == 4) return __uint_as_float(raw);
  else return c ? bf16_hi(raw) : bf16_lo(raw);
}
// Has a value formed at this point.  A token's raw values are taken when its turn comes and
// its results are fixed when it ends: otherwise the compiler starts on all tokens at once,
// or moves the forming of a result to its use beyond the look back, where everything it is
// formed from stays alive, and spills either way.
template <typename V>
__device__ __forceinline__ void fix(V& v) { asm volatile("" : "+v"(v)); }

template <typename IO, int C>
__device__ __forceinline__ void put(const Rows& w, int i, uint32_t off, const float (&v)[C]) {
  if constexpr (sizeof(IO) == 4) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[0]), w.r, off, w.at(i), 0);
  else if constexpr (C == 1) __builtin_amdgcn_raw_buffer_store_b16(f32_to_bf16(v[0]), w.r, off, w.at(i), 0);
  else
    __builtin_amdgcn_raw_buffer_store_b32(f32_to_bf16(v[0]) | (uint32_t)f32_to_bf16(v[1]) << 16, w.r, off, w.at(i), 0);
}
template <int C>
__device__ __forceinline__ void put_state(const Rows& w, int i, uint32_t off, const float (&v)[C]) {
#pragma unroll
  for (int c = 0; c < C; ++c) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[c]), w.r, off + 4 * c, w.at(i), 0);
}

// ---------------------------------------------------------------- the split over the sequence
//
// A workgroup owns kTok tokens per wave (wave after wave) of 64 * C channels.  Each
// wave scans its tokens from zero and leaves their affine map h -> A h + H in LDS.
// The workgroup publishes the map of all its tokens, composes the maps of its
// predecessors back to one whose end state is known (or to the initial state),
// publishes its own end state, and only then runs its recurrence from the state
// that enters, from decays and inputs still in registers: every input is read once.
//
// A published word is its own flag: the workspace starts as all ones, a NaN that no
// publisher writes (its NaNs are replaced by the standard one), so a reader needs no
// separate flag and no cache write-back orders the two.  Work items are handed out by
// a counter, level after level: whoever waits waits for items handed out before.
// A decay of exactly 0 (a reset) drops the older state, whatever it is.

constexpr int kMaxWaves = 8;
constexpr int kLook = 2;  // predecessors per wave and round of the look back
constexpr uint32_t kEmpty = 0xffffffffu;

struct Link {
  unsigned long long* map;  // (levels, blocks, 64 * C) of {A, H}
  uint32_t* end;            // (levels, blocks, 64 * C)
  uint32_t* ticket;
  uint32_t* err;
  uint32_t spin_limit;
  int levels, blocks, row_blocks;
};

template <int C>
struct ScanShared {
  float A[kMaxWaves][64 * C], H[kMaxWaves][64 * C];
  int closed[kMaxWaves];
  uint32_t item;
};

__device__ __forceinline__ uint32_t published(float v) { return v != v ? 0x7fc00000u : __float_as_uint(v); }

// (A, H) after (a, h): the older map applied first.
__device__ __forceinline__ void compose(float& A, float& H, float a, float h) {
  H = A == 0.0f ? H : __builtin_fmaf(A, h, H);
  A = A == 0.0f ? 0.0f : A * a;
}
__device__ __forceinline__ float apply(float A, float H, float h) { return A == 0.0f ? H : __builtin_fmaf(A, h, H); }

template <int C>
__device__ __forceinline__ void read_words(const Link& k, int level, int blk, int lane, uint32_t (&end)[C],
                                           unsigned long long (&map)[C]) {
  const size_t row = ((size_t)level * k.blocks + blk) * 64 * C;
  const uint32_t* e = k.end + row;
  const unsigned long long* m = k.map + row;
#pragma unroll
  for (int c = 0; c < C; ++c) {
    end[c] = __hip_atomic_load(e + (uint32_t)(lane * C + c), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    map[c] = __hip_atomic_load(m + (uint32_t)(lane * C + c), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
}

// State entering `level` of a block (init: the one entering level 0).  All waves call.
template <int C>
__device__ __forceinline__ void look_back(const Link& k, int level, int blk, int wave, const float (&init)[C],
                                          float (&carry)[C], ScanShared<C>& sm) {
  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  float A[C], H[C];
#pragma unroll
  for (int c = 0; c < C; ++c) A[c] = 1.0f, H[c] = 0.0f;
  for (int newest = level - 1;; newest -= waves * kLook) {
    float a[C], h[C];
#pragma unroll
    for (int c = 0; c < C; ++c) a[c] = 1.0f, h[c] = 0.0f;
    int closed = 0;
    const int e0 = newest - wave * kLook;
    unsigned long long m[kLook][C];
    uint32_t x[kLook][C];
#pragma unroll
    for (int j = 0; j < kLook; ++j) {
      read_words<C>(k, e0 - j > 0 ? e0 - j : 0, blk, lane, x[j], m[j]);
    }
#pragma unroll
    for (int j = 0; j < kLook; ++j) {
      if (closed || e0 - j < -1) continue;
      if (e0 - j == -1) {
#pragma unroll
        for (int c = 0; c < C; ++c) h[c] = apply(a[c], h[c], init[c]);
        closed = 1;
        continue;
      }
      for (uint32_t polls = 0;; ++polls) {
        bool end = true, map = true;
#pragma unroll
        for (int c = 0; c < C; ++c) end &= x[j][c] != kEmpty, map &= (uint32_t)m[j][c] != kEmpty;
        if (__all(end)) {
#pragma unroll
          for (int c = 0; c < C; ++c) h[c] = apply(a[c], h[c], __uint_as_float(x[j][c]));
          closed = 1;
          break;
        }
        if (__all(map)) {
#pragma unroll
          for (int c = 0; c < C; ++c)
            compose(a[c], h[c], __uint_as_float((uint32_t)m[j][c]), __uint_as_float((uint32_t)(m[j][c] >> 32)));
          break;
        }
        if (polls >= k.spin_limit) {  // never expected: report, and go on from NaN
          if (lane == 0) __hip_atomic_store(k.err, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
          for (int c = 0; c < C; ++c) h[c] = __uint_as_float(0x7fc00000u);
          closed = 1;
          break;
        }
        __builtin_amdgcn_s_sleep(1);
        read_words<C>(k, e0 - j, blk, lane, x[j], m[j]);
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) sm.A[wave][lane * C + c] = a[c], sm.H[wave][lane * C + c] = h[c];
    if (lane == 0) sm.closed[wave] = closed;
    __syncthreads();
    bool done = false;
#pragma unroll 1
    for (int w = 0; w < waves && !done; ++w) {
#pragma unroll
      for (int c = 0; c < C; ++c) compose(A[c], H[c], sm.A[w][lane * C + c], sm.H[w][lane * C + c]);
      done = sm.closed[w] != 0;
    }
    __syncthreads();
    if (done) break;
  }
#pragma unroll
  for (int c = 0; c < C; ++c) carry[c] = H[c];
}

// The workgroup's next work item (previous: -1 for the first): from the counter, or
// from the grid where there is one level and so no order.
__device__ __forceinline__ int64_t take_item(const Link& k, int64_t previous, uint32_t* shared_item) {
  if (k.levels == 1) return previous < 0 ? blockIdx.x : previous + gridDim.x;
  if (threadIdx.x == 0) *shared_item = atomicAdd(k.ticket, 1u);
  __syncthreads();
  return (uint32_t)__builtin_amdgcn_readfirstlane(*shared_item);
}

// State entering each wave's tokens, from the waves' maps in sm and the level's
// predecessors.  The last wave publishes the level's map and its end state, which it
// returns in `end`.
template <int C>
__device__ __forceinline__ void enter(const Link& k, int level, int blk, int wave, const float (&A)[C],
                                      const float (&H)[C], const float (&init)[C], float (&carry)[C], float (&end)[C],
                                      ScanShared<C>& sm) {
  const int lane = threadIdx.x & 63, waves = blockDim.x >> 6;
  float Ap[C], Hp[C];  // the map of the waves before this one
#pragma unroll
  for (int c = 0; c < C; ++c) Ap[c] = 1.0f, Hp[c] = 0.0f;
#pragma unroll 1
  for (int w = 0; w < wave; ++w)
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float a = sm.A[w][lane * C + c];
      Hp[c] = apply(a, sm.H[w][lane * C + c], Hp[c]);
      Ap[c] = a == 0.0f ? 0.0f : Ap[c] * a;
    }
  float in[C];
  if (k.levels == 1) {
#pragma unroll
    for (int c = 0; c < C; ++c) in[c] = init[c];
  } else {
    const size_t at = ((size_t)level * k.blocks + blk) * 64 * C + lane * C;
    const bool publish = wave == waves - 1 && level + 1 < k.levels;
    if (publish && level > 0)
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const float m = A[c] == 0.0f ? 0.0f : Ap[c] * A[c];
        __hip_atomic_store(k.map + at + c, published(m) | (unsigned long long)published(apply(A[c], H[c], Hp[c])) << 32,
                           __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
    __syncthreads();  // sm.A and sm.H are reused
    look_back<C>(k, level, blk, wave, init, in, sm);
    if (publish)
#pragma unroll
      for (int c = 0; c < C; ++c)
        __hip_atomic_store(k.end + at + c, published(apply(A[c], H[c], apply(Ap[c], Hp[c], in[c]))), __ATOMIC_RELAXED,
                           __HIP_MEMORY_SCOPE_AGENT);
  }
#pragma unroll
  for (int c = 0; c < C; ++c) {
    carry[c] = apply(Ap[c], Hp[c], in[c]);
    end[c] = apply(A[c], H[c], carry[c]);
  }
}

__global__ __launch_bounds__(256) void gated_clear_kernel(uint32_t* ticket, uint32_t* words, int64_t n) {
  if (blockIdx.x == 0 && threadIdx.x == 0) __hip_atomic_store(ticket, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    __hip_atomic_store(words + i, kEmpty, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// ---------------------------------------------------------------- forward

constexpr int kTokF = 16;  // tokens per wave

// Decays and inputs of a wave's tokens, and their map from zero.  A token past the end
// has loaded zeros: it adds nothing, and no token after it is kept.
template <bool HASR, int T, int C, typename IO>
__device__ __forceinline__ void gated_local(uint32_t (&ra)[T], uint32_t (&rx)[T], uint32_t (&u)[T],
                                            const float (&kappa)[C], uint32_t reset, float (&a)[T][C],
                                            float (&b)[T][C], float (&A)[C], float (&H)[C]) {
#pragma unroll
  for (int c = 0; c < C; ++c) A[c] = 1.0f, H[c] = 0.0f;
#pragma unroll
  for (int i = 0; i < T; ++i) {
    const bool cut = HASR && ((reset >> i) & 1);
    fix(ra[i]), fix(rx[i]), fix(u[i]);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      gated_token(part<IO>(ra[i], c), part<IO>(rx[i], c), part<IO>(u[i], c), kappa[c], cut, a[i][c], b[i][c]);
      H[c] = cut ? b[i][c] : __builtin_fmaf(a[i][c], H[c], b[i][c]);
      A[c] = cut ? 0.0f : A[c] * a[i][c];
      fix(a[i][c]), fix(b[i][c]);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
}

template <typename IO, int C, bool HASZ, bool HASR>
__global__ __launch_bounds__(64 * kMaxWaves, 4) void gated_fwd_kernel(GatedArgs g, Link k) {
  constexpr int T = kTokF, ES = sizeof(IO);
  __shared__ ScanShared<C> sm;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int64_t items = (int64_t)k.levels * k.blocks;
  const int64_t nst = (g.L + kGatedStateChunk - 1) / kGatedStateChunk;
  const uint32_t stride = (uint32_t)g.D * ES, sstride = (uint32_t)g.D * 4;
  for (int64_t item = take_item(k, -1, &sm.item); item < items; item = take_item(k, item, &sm.item)) {
    const int level = (int)((uint32_t)item / (uint32_t)k.blocks), blk = (int)((uint32_t)item % (uint32_t)k.blocks);
    const int64_t bt = blk / k.row_blocks;
    const int64_t d0 = (int64_t)(blk % k.row_blocks) * 64 * C + lane * C;
    const bool act = d0 < g.D;
    const uint32_t d = act ? (uint32_t)d0 : 0;
    const int64_t t0 = ((int64_t)level * waves + wave) * T;
    const int n = __builtin_amdgcn_readfirstlane((int)(g.L - t0 < T ? (g.L - t0 > 0 ? g.L - t0 : 0) : T));
    const int64_t row = bt * g.L + (n > 0 ? t0 : 0);
    const size_t skip = (size_t)row * g.D * ES;
    const uint32_t off = act ? (uint32_t)d0 * ES : kNowhere, soff = act ? (uint32_t)d0 * 4 : kNowhere;

    const Rows r_ra(g.ra, skip, stride, n), r_rx(g.rx, skip, stride, n), r_u(g.u, skip, stride, n);
    uint32_t ra[T], rx[T], u[T], z[T];
#pragma unroll
    for (int i = 0; i < T; ++i) {
      ra[i] = fetch<IO, C>(r_ra, i, off);
      rx[i] = fetch<IO, C>(r_rx, i, off);
      u[i] = fetch<IO, C>(r_u, i, off);
    }
    if (HASZ) {
      const Rows r_z(g.z, skip, stride, n);
#pragma unroll
      for (int i = 0; i < T; ++i) z[i] = fetch<IO, C>(r_z, i, off);
    }
    uint32_t reset = 0;
    if (HASR) reset = (uint32_t)__ballot(lane < n && g.reset[row + (lane < n ? lane : 0)] != 0);
    float kappa[C], init[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      kappa[c] = g.c * softplus(g.lam[d + c]);
      init[c] = g.h0 ? g.h0[bt * g.D + d + c] : 0.0f;
    }
    float a[T][C], b[T][C], A[C], H[C];
    gated_local<HASR, T, C, IO>(ra, rx, u, kappa, reset, a, b, A, H);
#pragma unroll
    for (int c = 0; c < C; ++c) sm.A[wave][lane * C + c] = A[c], sm.H[wave][lane * C + c] = H[c];
    __syncthreads();
    float h[C], end[C];
    enter<C>(k, level, blk, wave, A, H, init, h, end, sm);

    // the recurrence from the state that enters
    const Rows r_out(g.out, skip, stride, n);
    const Rows r_st(g.states, (size_t)(bt * nst + (n > 0 ? t0 : 0) / kGatedStateChunk) * sstride, sstride,
                    (n + kGatedStateChunk - 1) / kGatedStateChunk);
    const int last_token = g.last && t0 + T >= g.L ? n - 1 : -1;
#pragma unroll
    for (int i = 0; i < T; ++i) {
      const bool cut = HASR && ((reset >> i) & 1);
      if (i % kGatedStateChunk == 0) put_state<C>(r_st, i / kGatedStateChunk, soff, h);
      float o[C];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        h[c] = cut ? b[i][c] : __builtin_fmaf(a[i][c], h[c], b[i][c]);
        o[c] = HASZ ? h[c] * silu(part<IO>(z[i], c)) : h[c];
      }
      put<IO, C>(r_out, i, off, o);
      __builtin_amdgcn_sched_barrier(0);
      if (i == last_token) put_state<C>(Rows(g.last, (size_t)bt * sstride, sstride, 1), 0, soff, h);
    }
    __syncthreads();  // sm is reused by the next item
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

// What the way back needs of each token.
template <int T, int C>
struct BwdRun {
  float a[T][C], dy[T][C], p1[T][C], p2[T][C], e0[T][C], oa[T][C];
};

// A run's way forward: dz, the factors, and the map of the gradient through the run.  A
// token past the end has loaded zeros: its gradient is 0 and stays 0 up to the last token,
// where dlast enters (`last_token`; -1 where the run does not hold it).
template <bool HASZ, bool HASR, int T, int C, typename IO>
__device__ __forceinline__ void gated_bwd_local(uint32_t (&ra)[T], uint32_t (&rx)[T], uint32_t (&u)[T],
                                                uint32_t (&z)[T], uint32_t (&dout)[T], const float (&kappa)[C],
                                                uint32_t reset, int last_token, const float (&dlast)[C], Rows dz,
                                                uint32_t off, float (&h)[C], BwdRun<T, C>& w,
                                                float (&A)[C], float (&H)[C]) {
#pragma unroll
  for (int i = 0; i < T; ++i) {
    const bool cut = HASR && ((reset >> i) & 1);
    float dzv[C];
    fix(ra[i]), fix(rx[i]), fix(u[i]), fix(dout[i]);
    if (HASZ) fix(z[i]);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const GatedGrad q = gated_grad(part<IO>(ra[i], c), part<IO>(rx[i], c), kappa[c], cut);
      const float x = q.sx * part<IO>(u[i], c), b = q.s * x;
      const float ah = cut ? 0.0f : q.a * h[c];
      h[c] = ah + b;
      w.a[i][c] = q.a;
      w.p1[i][c] = q.s * q.sx;
      w.p2[i][c] = b * q.ox;
      w.e0[i][c] = __builtin_fmaf(ah, q.l, -q.q * x);
      w.oa[i][c] = q.oa;
      w.dy[i][c] = part<IO>(dout[i], c);
      if (HASZ) {
        float sz, dsz;
        silu_pair(part<IO>(z[i], c), sz, dsz);
        dzv[c] = w.dy[i][c] * h[c] * dsz;
        w.dy[i][c] *= sz;
      }
      w.dy[i][c] += i == last_token ? dlast[c] : 0.0f;
      fix(w.a[i][c]), fix(w.p1[i][c]), fix(w.p2[i][c]), fix(w.e0[i][c]), fix(w.oa[i][c]), fix(w.dy[i][c]);
    }
    if (HASZ) put<IO, C>(dz, i, off, dzv);
    __builtin_amdgcn_sched_barrier(0);
  }
#pragma unroll
  for (int c = 0; c < C; ++c) A[c] = 1.0f, H[c] = 0.0f;
#pragma unroll
  for (int i = T - 1; i >= 0; --i) {
    const bool cut = HASR && ((reset >> i) & 1);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      H[c] = cut ? 0.0f : w.a[i][c] * (w.dy[i][c] + H[c]);
      A[c] = cut ? 0.0f : A[c] * w.a[i][c];
    }
  }
}

template <typename IO, int C, bool HASZ, bool HASR>
__global__ __launch_bounds__(64 * kMaxWaves, 4) void gated_bwd_kernel(GatedBwdArgs g, Link k, float* pl) {
  constexpr int T = kTokB, ES = sizeof(IO);
  const GatedArgs& f = g.f;
  __shared__ ScanShared<C> sm;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), waves = blockDim.x >> 6;
  const int64_t items = (int64_t)k.levels * k.blocks;
  const uint32_t stride = (uint32_t)f.D * ES, sstride = (uint32_t)f.D * 4;
  for (int64_t item = take_item(k, -1, &sm.item); item < items; item = take_item(k, item, &sm.item)) {
    const int level = (int)((uint32_t)item / (uint32_t)k.blocks), blk = (int)((uint32_t)item % (uint32_t)k.blocks);
    const int64_t bt = blk / k.row_blocks;
    const int64_t d0 = (int64_t)(blk % k.row_blocks) * 64 * C + lane * C;
    const bool act = d0 < f.D;
    const uint32_t d = act ? (uint32_t)d0 : 0;
    const int64_t run = (int64_t)(k.levels - 1 - level) * waves + (waves - 1 - wave);
    const int64_t t0 = run * T;
    const int n = __builtin_amdgcn_readfirstlane((int)(f.L - t0 < T ? (f.L - t0 > 0 ? f.L - t0 : 0) : T));
    const int64_t row = bt * f.L + (n > 0 ? t0 : 0);
    const size_t skip = (size_t)row * f.D * ES;
    const uint32_t off = act ? (uint32_t)d0 * ES : kNowhere, soff = act ? (uint32_t)d0 * 4 : kNowhere;

    const Rows r_ra(f.ra, skip, stride, n), r_rx(f.rx, skip, stride, n), r_u(f.u, skip, stride, n),
        r_do(g.dout, skip, stride, n);
    uint32_t ra[T], rx[T], u[T], dout[T], z[T];
#pragma unroll
    for (int i = 0; i < T; ++i) {
      ra[i] = fetch<IO, C>(r_ra, i, off);
      rx[i] = fetch<IO, C>(r_rx, i, off);
      u[i] = fetch<IO, C>(r_u, i, off);
      dout[i] = fetch<IO, C>(r_do, i, off);
    }
    if (HASZ) {
      const Rows r_z(f.z, skip, stride, n);
#pragma unroll
      for (int i = 0; i < T; ++i) z[i] = fetch<IO, C>(r_z, i, off);
    }
    uint32_t reset = 0;
    if (HASR) reset = (uint32_t)__ballot(lane < n && f.reset[row + (lane < n ? lane : 0)] != 0);
    float kappa[C], dlast[C], h[C];
    const int64_t state_row = bt * ((f.L + T - 1) / T) + (n > 0 ? run : 0);
    const int last_token = g.dlast && t0 + T >= f.L ? n - 1 : -1;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      kappa[c] = f.c * softplus(f.lam[d + c]);
      dlast[c] = last_token >= 0 ? g.dlast[bt * f.D + d + c] : 0.0f;
      h[c] = f.states[state_row * f.D + d + c];
    }
    BwdRun<T, C> w;
    float A[C], H[C];
    gated_bwd_local<HASZ, HASR, T, C, IO>(ra, rx, u, z, dout, kappa, reset, last_token, dlast,
                                          Rows(g.dz, skip, stride, n), off, h, w, A, H);
#pragma unroll
    for (int c = 0; c < C; ++c) sm.A[wave][lane * C + c] = A[c], sm.H[wave][lane * C + c] = H[c];
    __syncthreads();
    float cg[C], end[C], sum[C], zero[C];
#pragma unroll
    for (int c = 0; c < C; ++c) sum[c] = zero[c] = 0.0f;
    enter<C>(k, level, blk, wave, A, H, zero, cg, end, sm);
    if (g.dh0 && level == k.levels - 1 && wave == waves - 1)
      put_state<C>(Rows(g.dh0, (size_t)bt * sstride, sstride, 1), 0, soff, end);

    // the way back from the gradient that enters
    const Rows r_du(g.du, skip, stride, n), r_drx(g.drx, skip, stride, n), r_dra(g.dra, skip, stride, n);
#pragma unroll
    for (int i = T - 1; i >= 0; --i) {
      const bool cut = HASR && ((reset >> i) & 1);
      float du[C], dra[C], drx[C];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const float G = w.dy[i][c] + cg[c];
        const float e = cut ? 0.0f : G * w.e0[i][c];
        du[c] = G * w.p1[i][c];
        drx[c] = G * w.p2[i][c];
        dra[c] = e * w.oa[i][c];
        sum[c] += e;
        cg[c] = cut ? 0.0f : w.a[i][c] * G;
      }
      put<IO, C>(r_du, i, off, du);
      put<IO, C>(r_drx, i, off, drx);
      put<IO, C>(r_dra, i, off, dra);
      __builtin_amdgcn_sched_barrier(0);
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < C; ++c) sm.H[wave][lane * C + c] = sum[c];
    __syncthreads();
    if (wave == 0) {
      float v[C];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        v[c] = 0.0f;
#pragma unroll 1
        for (int q = 0; q < waves; ++q) v[c] += sm.H[q][lane * C + c];
      }
      put_state<C>(Rows(pl, (size_t)(bt * k.levels + level) * sstride, sstride, 1), 0, soff, v);
    }
    __syncthreads();
  }
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

template <typename IO>
__global__ __launch_bounds__(256) void gated_step_kernel(GatedStepArgs g) {
  const int64_t d = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t bt = blockIdx.y;
  if (d >= g.D) return;
  const size_t i = (size_t)bt * g.D + d;
  const bool reset = g.reset && g.reset[bt] != 0;
  float a, b;
  gated_token(load_io((const IO*)g.ra, i), load_io((const IO*)g.rx, i), load_io((const IO*)g.u, i),
              g.c * softplus(g.lam[d]), reset, a, b);
  const float h = reset ? b : __builtin_fmaf(a, g.state[i], b);
  g.state[i] = h;
  store_io((IO*)g.out, i, g.z ? h * silu(load_io((const IO*)g.z, i)) : h);
}

size_t al256(size_t v) { return (v + 255) / 256 * 256; }

// How a sequence is cut: levels of waves * tok tokens, blocks of 64 * vec channels.
struct GatedPlan {
  int vec, waves, row_blocks;
  int64_t levels, blocks;
  size_t words, off_end, off_map, bytes;  // workspace: the ticket, `end` and `map` words (none for one level)
};

GatedPlan plan_gated(int64_t batch, int64_t L, int64_t D, int tok, int io) {
  GatedPlan p{};
  if (batch == 0 || L == 0 || D == 0) return p;
  p.vec = io == kIoBF16 && D % 2 == 0 ? 2 : 1;
  p.row_blocks = (int)((D + 64 * p.vec - 1) / (64 * p.vec));
  p.blocks = batch * p.row_blocks;
  const int64_t runs = (L + tok - 1) / tok;
  p.waves = (int)std::min<int64_t>(runs, kMaxWaves);
  p.levels = (runs + p.waves - 1) / p.waves;
  if (p.levels > 1) {
    const size_t n = (size_t)p.levels * p.blocks * 64 * p.vec;
    p.off_end = 256;
    p.off_map = p.off_end + al256(n * 4);
    p.bytes = p.off_map + al256(n * 8);
    p.words = (p.bytes - p.off_end) / 4;
  }
  return p;
}

// One workgroup per item, up to 2^20 (a grid holds fewer than 2^32 threads); the rest is looped over.
unsigned grid_of(const GatedPlan& p) { return (unsigned)std::min<int64_t>((int64_t)p.levels * p.blocks, 1 << 20); }

// The link of a launch: clears the workspace's words (one level: nothing).
hipError_t prepare_link(const GatedPlan& p, void* ws, Link& k, hipStream_t st) {
  k = Link{};
  k.levels = (int)p.levels;
  k.blocks = (int)p.blocks;
  k.row_blocks = p.row_blocks;
  if (p.levels == 1) return hipSuccess;
  uint8_t* w = static_cast<uint8_t*>(ws);
  k.ticket = reinterpret_cast<uint32_t*>(w);
  k.end = reinterpret_cast<uint32_t*>(w + p.off_end);
  k.map = reinterpret_cast<unsigned long long*>(w + p.off_map);
  k.err = wait_status_ptr();
  if (k.err == nullptr) return hipErrorInvalidSymbol;
  k.spin_limit = (uint32_t)option(kOptSpinLimit);
  hipLaunchKernelGGL(gated_clear_kernel, dim3((unsigned)std::min<size_t>((p.words + 1023) / 1024, 4096)), dim3(256), 0,
                     st, k.ticket, k.end, (int64_t)p.words);
  return hipGetLastError();
}

size_t states_bytes(int64_t batch, int64_t L, int64_t D) {
  return al256((size_t)batch * ((L + kGatedStateChunk - 1) / kGatedStateChunk) * D * 4);
}

#define S6_PICK_GATED(name)                                                                      \
  template <typename IO, int C>                                                                  \
  auto* pick_##name(const void* z, const void* reset) {                                          \
    return z ? (reset ? name##_kernel<IO, C, true, true> : name##_kernel<IO, C, true, false>)    \
             : (reset ? name##_kernel<IO, C, false, true> : name##_kernel<IO, C, false, false>); \
  }                                                                                              \
  auto* pick_##name(int vec, int io, const void* z, const void* reset) {                         \
    return vec == 2        ? pick_##name<uint16_t, 2>(z, reset)                                  \
           : io == kIoBF16 ? pick_##name<uint16_t, 1>(z, reset)                                  \
                           : pick_##name<float, 1>(z, reset);                                    \
  }
S6_PICK_GATED(gated_fwd)
S6_PICK_GATED(gated_bwd)
#undef S6_PICK_GATED

}  // namespace

// Work items are counted in 32 bits.
bool gated_fits(int64_t batch, int64_t L, int64_t D) {
  const GatedPlan p = plan_gated(batch, L, D, kTokB, kIoF32);
  return p.levels < (int64_t(1) << 31) && p.blocks < (int64_t(1) << 31) &&
         (double)p.levels * (double)p.blocks < 2147483648.0;
}

size_t gated_fwd_ws_bytes(int64_t batch, int64_t L, int64_t D, int io) {
  return plan_gated(batch, L, D, kTokF, io).bytes;
}

hipError_t launch_gated_fwd(const GatedArgs& a, int io, void* ws, hipStream_t st) {
  if (a.L == 0) {
    const int64_t n = a.batch * a.D;
    if (a.last) hipLaunchKernelGGL(gated_copy_state_kernel, dim3((unsigned)std::min<int64_t>((n + 255) / 256, 65536)),
                                   dim3(256), 0, st, a.h0, a.last, n);
    return hipGetLastError();
  }
  const GatedPlan p = plan_gated(a.batch, a.L, a.D, kTokF, io);
  Link k;
  const hipError_t e = prepare_link(p, ws, k, st);
  if (e != hipSuccess) return e;
  const dim3 grid(grid_of(p)), block(64 * p.waves);
  auto* kernel = pick_gated_fwd(p.vec, io, a.z, a.reset);
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
  p.link = plan_gated(batch, L, D, kTokB, io);
  const int64_t n = batch * p.link.levels;
  p.rows = std::max<int64_t>(64, (n + 255) / 256);
  p.stages = (n + p.rows - 1) / p.rows;
  p.off_sum = al256(std::max(p.link.bytes, plan_gated(batch, L, D, kTokF, io).bytes));
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
  const dim3 grid(grid_of(p.link)), block(64 * p.link.waves);
  auto* kernel = pick_gated_bwd(p.link.vec, io, f.z, f.reset);
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
