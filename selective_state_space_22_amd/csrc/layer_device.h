// layer_device.h -- device helpers shared by the layer operators (include/mamba_mi355x_layer.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "s6_device.h"

namespace s6 {

// V elements of an I/O type as raw 32-bit words.
template <typename T, int V>
using raw_t = uint32_t __attribute__((ext_vector_type(V * (int)sizeof(T) / 4)));

// V elements of a row from p on, of which the first nv exist (FULL: all); the others are zero bits and
// are not read.  p is aligned to its element only (rows of an odd length): global memory takes 8- and
// 16-byte accesses at any byte address on gfx950, so one code path serves every row length.
template <typename T, int V, bool FULL>
__device__ __forceinline__ raw_t<T, V> load_raw(const T* p, int nv) {
  raw_t<T, V> v;
  if constexpr (FULL) {
    __builtin_memcpy(&v, p, V * sizeof(T));
  } else {
#pragma unroll
    for (int i = 0; i < V * (int)sizeof(T) / 4; ++i) v[i] = 0u;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (i < nv) {
        if constexpr (sizeof(T) == 2) v[i / 2] |= (uint32_t)p[i] << (16 * (i & 1));
        else v[i] = __float_as_uint(p[i]);
      }
    }
  }
  return v;
}

template <typename T, int V, bool FULL>
__device__ __forceinline__ void store_raw(T* p, raw_t<T, V> v, int nv) {
  if constexpr (FULL) {
    __builtin_memcpy(p, &v, V * sizeof(T));
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (i < nv) {
        if constexpr (sizeof(T) == 2) p[i] = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
        else p[i] = __uint_as_float(v[i]);
      }
    }
  }
}

// Raw words <-> fp32 values.
template <typename T, int V>
__device__ __forceinline__ void widen(raw_t<T, V> v, float (&f)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if constexpr (sizeof(T) == 2) f[i] = i & 1 ? bf16_hi(v[i / 2]) : bf16_lo(v[i / 2]);
    else f[i] = __uint_as_float(v[i]);
  }
}

template <typename T, int V>
__device__ __forceinline__ raw_t<T, V> narrow(const float (&f)[V]) {
  raw_t<T, V> v;
#pragma unroll
  for (int i = 0; i < V * (int)sizeof(T) / 4; ++i) {
    if constexpr (sizeof(T) == 2) v[i] = (uint32_t)f32_to_bf16(f[2 * i]) | ((uint32_t)f32_to_bf16(f[2 * i + 1]) << 16);
    else v[i] = __float_as_uint(f[i]);
  }
  return v;
}

// sigma(v) = 1 / (1 + e^-v), and SiLU'(v) = sigma (1 + v (1 - sigma)).  The slope is no number at either infinity, SiLU
// itself only at -infinity.
__device__ __forceinline__ float sigmoid(float v) { return rcp(1.0f + ex2(-v * kLog2e)); }
__device__ __forceinline__ float silu_slope(float v) {
  const float s = sigmoid(v);
  return s * __builtin_fmaf(v, 1.0f - s, 1.0f);
}

// Sums of the columns of part (rows, cols), a column per threadIdx.x % C of a 1024-thread block: K = 1024 / C
// threads add every K-th row each, in the order of the rows, then the K sums are added in their order.
// Returns the sum in the block's first C threads (col < cols).
template <int C>
__device__ __forceinline__ float column_sum(const float* part, int64_t rows, int64_t cols, int64_t col) {
  constexpr int K = 1024 / C, S = K / 32;
  static_assert(K % 32 == 0, "the K sums are added in 32 groups");
  __shared__ float s[K][C + 1];
  const int c = threadIdx.x % C, k = threadIdx.x / C;
  float v = 0.0f;
  if (col < cols) {
    const float* p = part + col;
    int64_t r = k;
    for (; r + 7 * K < rows; r += 8 * K) {  // eight loads in flight
      float q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = p[(r + K * i) * cols];
#pragma unroll
      for (int i = 0; i < 8; ++i) v += q[i];
    }
    for (; r < rows; r += K) v += p[r * cols];
  }
  s[k][c] = v;
  __syncthreads();
  if constexpr (S > 1) {
    v = 0.0f;
    if (k < 32)
#pragma unroll
      for (int i = 0; i < S; ++i) v += s[k * S + i][c];
    __syncthreads();
    if (k < 32) s[k][c] = v;
    __syncthreads();
  }
  v = 0.0f;
  if (k == 0)
    for (int i = 0; i < 32; ++i) v += s[i][c];
  return v;
}

// Columns of a block of column_sum: 8 as long as every such block has a compute unit of its own, so that more threads share
// a column's rows (8869 rows of 240 columns: 11.3 us so, 14.0 with 32), else 32 (forward and gradients of 3 x 1537 x 1101
// fp32, 4404 columns: 28.7 us so, 31.6 with 8).
template <typename F>
void by_columns(int64_t cols, F f) {
  if (cols <= 8 * 256) f(std::integral_constant<int, 8>());
  else f(std::integral_constant<int, 32>());
}

}  // namespace s6
