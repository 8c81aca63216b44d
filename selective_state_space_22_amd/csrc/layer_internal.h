// layer_internal.h -- host-side plans and launchers of the layer operators
// (include/mamba_mi355x_layer.h), shared by api_layer.cpp and the kernel files.  Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "s6_internal.h"

namespace s6 {

// ---------------------------------------------------------------- short convolution (conv.hip)

// Tokens of the chunk [t0, t1) that a row of len tokens has.  Clamped in 64 bits: the row may end more than 2^31
// tokens before the chunk.
__host__ __device__ constexpr int chunk_tokens(int64_t t0, int64_t t1, int64_t len) {
  const int64_t n = (t1 < len ? t1 : len) - t0;
  return n > 0 ? (int)n : 0;
}

struct ConvArgs {
  const void* x;
  const float* weight;     // (D, W)
  const float* bias;       // may be null
  const void* window;      // (batch, W - 1, D), may be null
  const uint8_t* reset;    // (batch, L), may be null
  const int32_t* lengths;  // (batch), may be null
  void* out;
  void* last;              // (batch, W - 1, D), may be null
  int64_t batch, L, D;
  int32_t W, silu;
};

struct ConvBwdArgs {
  ConvArgs f;              // inputs of the forward; lengths, out, last unused
  const void* dout;
  const void* dlast;       // may be null
  void* dx;
  float* dweight;          // (D, W)
  float* dbias;            // may be null
  void* dwindow;           // may be null
};

struct ConvStepArgs {
  void* window;            // (nslots, W - 1, D)
  const void* x;
  const float* weight;
  const float* bias;       // may be null
  const int32_t* slots;    // (batch), may be null: row b has place b
  void* out;
  int64_t batch, D, nslots;
  int32_t W, silu;
};

bool conv_fits(int64_t batch, int64_t L, int64_t D);  // false: more work items than a launch can count
hipError_t launch_conv_fwd(const ConvArgs& a, int io, hipStream_t stream);
size_t conv_bwd_ws_bytes(int64_t batch, int64_t L, int64_t D, int64_t W);
hipError_t launch_conv_bwd(const ConvBwdArgs& a, int io, void* workspace, hipStream_t stream);
hipError_t launch_conv_step(const ConvStepArgs& a, int io, hipStream_t stream);

// ---------------------------------------------------------------- one token of a layer (ssm_step.hip)

struct SsmStepArgs {
  float* state;              // (nslots, D, N)
  void* window;              // (nslots, W - 1, D)
  const void* x;             // (batch, D)
  const float* conv_weight;  // (D, W)
  const float* conv_bias;    // may be null
  const void* Wx;            // (R + 2N, D)
  const void* Wdt;           // (D, R)
  const float* dt_bias;      // may be null
  const float* A;            // (D, N)
  const float* dskip;        // may be null
  const void* z;             // (batch, D), may be null
  const int32_t* slots;      // (batch), may be null
  void* out;                 // (batch, D)
  int64_t batch, D, N, R, nslots;
  int32_t W;
};

size_t ssm_step_ws_bytes(int64_t batch, int64_t D, int64_t N, int64_t R);
hipError_t launch_ssm_step(const SsmStepArgs& a, int io, void* workspace, hipStream_t stream);

// ---------------------------------------------------------------- norms around a block (norm.hip)

constexpr int64_t kMaxNormDim = 16384;

struct NormArgs {
  const void* x;
  const void* gate;         // may be null
  const float* post;        // may be null
  const float* scale;       // may be null
  const void* residual;     // may be null
  const float* pre;         // may be null: no norm behind the sum
  void* residual_out;       // may be null
  void* out;                // null exactly where pre is
  int64_t rows, D;
  float alpha, eps;
  int32_t gate_first;
};

struct NormBwdArgs {
  NormArgs f;               // inputs of the forward; residual_out, out unused
  const void* dout;         // null exactly where pre is
  const void* dres_out;     // may be null
  void* dx;
  void* dgate;              // may be null
  void* dresidual;          // may be null
  float* dpost;             // may be null
  float* dscale;            // may be null
  float* dpre;              // may be null
};

bool norm_fits(int64_t rows, int64_t D);  // false: more threads than a launch can count
hipError_t launch_norm_fwd(const NormArgs& a, int io, int res, hipStream_t stream);
size_t norm_bwd_ws_bytes(int64_t rows, int64_t D);
hipError_t launch_norm_bwd(const NormBwdArgs& a, int io, int res, void* workspace, hipStream_t stream);

// ---------------------------------------------------------------- verification of drafts (verify.hip)

struct VerifyArgs {
  const void* target;     // (rows, K + 1, V)
  const void* draft;      // (rows, K, V)
  const int64_t* drafted; // (rows, K)
  const float* uniform;   // (rows, K)
  const float* noise;     // (rows, V)
  const int32_t* counts;  // (rows), may be null
  int64_t* tokens;        // (rows, K + 1)
  int32_t* accepted;      // (rows)
  int64_t rows, K, V;
};

size_t verify_ws_bytes(int64_t rows, int64_t V);
hipError_t launch_verify(const VerifyArgs& a, int io, void* workspace, hipStream_t stream);

}  // namespace s6
