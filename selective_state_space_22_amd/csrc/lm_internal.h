// lm_internal.h -- host-side plans and launchers of the token-model operators
// (include/mamba_mi355x_lm.h), shared by api_lm.cpp and the kernel files.  Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "s6_internal.h"

namespace s6 {

// ---------------------------------------------------------------- gated recurrence (gated_scan.hip)

constexpr int kGatedStateChunk = 8;  // tokens between two saved states (MAMBA_GATED_STATE_CHUNK)

struct GatedArgs {
  const void* u;
  const void* ra;        // gate_a
  const void* rx;        // gate_x
  const float* lam;
  const void* z;         // may be null
  const uint8_t* reset;  // may be null
  const float* h0;       // may be null
  void* out;             // null: states only
  float* last;           // may be null
  float* states;         // may be null
  int64_t batch, L, D;
  float c;
};

struct GatedBwdArgs {
  GatedArgs f;           // the forward's inputs; out, last unused; states: saved by the forward
  const void* dout;
  const float* dlast;    // may be null
  void* du;
  void* dra;
  void* drx;
  float* dlam;
  void* dz;              // may be null
  float* dh0;            // may be null
};

struct GatedStepArgs {
  float* state;
  const void* u;
  const void* ra;
  const void* rx;
  const float* lam;
  const void* z;         // may be null
  const uint8_t* reset;  // may be null
  void* out;
  int64_t batch, D;
  float c;
};

bool gated_fits(int64_t batch, int64_t L, int64_t D);  // false: more work items than a launch can count
size_t gated_fwd_ws_bytes(int64_t batch, int64_t L, int64_t D, int io);
hipError_t launch_gated_fwd(const GatedArgs& a, int io, void* workspace, hipStream_t stream);
size_t gated_bwd_ws_bytes(int64_t batch, int64_t L, int64_t D, int io);
hipError_t launch_gated_bwd(const GatedBwdArgs& a, int io, void* workspace, hipStream_t stream);
hipError_t launch_gated_step(const GatedStepArgs& a, int io, hipStream_t stream);

// ---------------------------------------------------------------- embedding (embed.hip)

hipError_t launch_embed_fwd(int64_t n, int64_t V, int64_t D, int io, const int64_t* ids, const void* W, float scale,
                            void* out, hipStream_t stream);
size_t embed_bwd_ws_bytes(int64_t n, int64_t V, int64_t D, int io);
hipError_t launch_embed_bwd(int64_t n, int64_t V, int64_t D, int io, const int64_t* ids, const void* dout, float scale,
                            void* dW, void* workspace, hipStream_t stream);

// ---------------------------------------------------------------- sampling (sample.hip)

struct SampleArgs {
  const void* logits;
  const float* noise;
  const float* temperature;  // may be null
  const int32_t* top_k;      // may be null
  const float* top_p;        // may be null
  const float* min_p;        // may be null
  int64_t* tokens;
  float* logprob;            // may be null
  int64_t rows, V;
};

hipError_t launch_sample(const SampleArgs& a, int io, hipStream_t stream);

}  // namespace s6
