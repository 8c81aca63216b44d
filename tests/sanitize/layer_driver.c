/* Host-side checks of the layer operators' C ABI (include/mamba_mi355x_layer.h) for a build of the library whose
 * host code carries AddressSanitizer and UndefinedBehaviorSanitizer (tests/test_layer_sanitizers.py).  Every call
 * here is rejected or answered on the host before the HIP runtime is touched; no GPU is needed.  The fake device
 * pointers are never dereferenced. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "mamba_mi355x_layer.h"

static int fails = 0;
#define CHECK(cond)                                                     \
  do {                                                                  \
    if (!(cond)) {                                                      \
      fprintf(stderr, "check failed line %d: %s\n", __LINE__, #cond); \
      ++fails;                                                          \
    }                                                                   \
  } while (0)

static void* F = (void*)(uintptr_t)0x10000; /* aligned, never dereferenced */
static void* M = (void*)(uintptr_t)0x10004; /* misaligned */

static int conv_bwd(int64_t b, int64_t l, int64_t d, int64_t w, int io, void* x, size_t bytes) {
  return mamba_conv_bwd(b, l, d, w, io, x, F, NULL, NULL, NULL, 1, F, NULL, F, F, NULL, NULL, bytes ? F : NULL, bytes, NULL);
}
static int step(int64_t b, int64_t d, int64_t n, int64_t r, int64_t w, int io, int64_t slots, void* x, size_t bytes) {
  return mamba_conv_ssm_update(b, d, n, r, w, io, slots, F, F, x, F, NULL, F, F, NULL, F, NULL, NULL, F, F,
                               bytes ? F : NULL, bytes, NULL);
}
static int norm_bwd(int64_t m, int64_t d, int io, int res, void* x, float alpha, float eps, size_t bytes) {
  return mamba_residual_norm_bwd(m, d, io, res, x, NULL, 1, NULL, NULL, NULL, F, alpha, eps, F, NULL, F, NULL, NULL, NULL,
                                 NULL, F, bytes ? F : NULL, bytes, NULL);
}
static int verify(int64_t m, int64_t k, int64_t v, int io, void* p, size_t bytes) {
  return mamba_draft_verify(m, k, v, io, p, F, F, F, F, NULL, F, F, bytes ? F : NULL, bytes, NULL);
}

int main(void) {
  const int64_t sizes[] = {INT64_MIN, -1, 0, 1, 7, 8, 63, 64, 65, 4096, 16384, 16385, 65535, 65536, 4194304, 4194305,
                           INT32_MAX, (int64_t)INT32_MAX + 1, (int64_t)1 << 40, ((int64_t)1 << 40) + 1, INT64_MAX};
  const int n = (int)(sizeof sizes / sizeof sizes[0]);
  /* every combination of sizes: a workspace or a refusal, no overflow on the way */
  for (int i = 0; i < n; ++i)
    for (int j = 0; j < n; ++j)
      for (int io = -1; io < 3; ++io) {
        const int64_t a = sizes[i], b = sizes[j];
        const int io_ok = io == 0 || io == 1;
        for (int k = 0; k < n; ++k) {
          const int64_t c = sizes[k];
          const size_t f = mamba_conv_bwd_workspace_size(a, b, c, 4, io);
          if (!(a > 0 && b >= 0 && c > 0 && io_ok)) CHECK(f == 0);
          CHECK(f < ((size_t)1 << 60));
          if (f) CHECK(conv_bwd(a, b, c, 4, io, F, f - 1) == MAMBA_ERR_WORKSPACE);
          else CHECK(!(a > 0 && b >= 0 && c > 0 && io_ok) || conv_bwd(a, b, c, 4, io, F, 1) == MAMBA_ERR_DIM);
          const size_t v = mamba_draft_verify_workspace_size(a, b, c, io);
          CHECK(v < ((size_t)1 << 60));
          if (v) CHECK(verify(a, b, c, io, F, v - 1) == MAMBA_ERR_WORKSPACE);
          const size_t s = mamba_conv_ssm_update_workspace_size(a, b, 16, c, io);
          CHECK(s < ((size_t)1 << 60));
          if (s && a > 0 && b > 0) CHECK(step(a, b, 16, c, 3, io, a, F, s - 1) == MAMBA_ERR_WORKSPACE);
        }
        const size_t w = mamba_residual_norm_bwd_workspace_size(a, b, io);
        CHECK(w < ((size_t)1 << 60));
        if (w) CHECK(norm_bwd(a, b, io, 0, F, 1.0f, 1e-5f, w - 1) == MAMBA_ERR_WORKSPACE);
        for (int k = 0; k < n; ++k) {
          if (sizes[k] < 2 || sizes[k] > 4) {
            CHECK(mamba_conv_bwd_workspace_size(2, 9, 8, sizes[k], 0) == 0);
            CHECK(conv_bwd(2, 9, 8, sizes[k], 0, F, 1) == MAMBA_ERR_UNSUPPORTED);
          }
        }
      }
  CHECK(conv_bwd(1, 1, 8, 4, 2, F, 0) == MAMBA_ERR_DTYPE && conv_bwd(1, 1, 8, 4, 0, M, 0) == MAMBA_ERR_ALIGN);
  CHECK(conv_bwd(1, 1, 8, 4, 0, NULL, 0) == MAMBA_ERR_NULL && conv_bwd(1, 1, 8, 4, 0, F, 0) == MAMBA_ERR_WORKSPACE);
  CHECK(conv_bwd(2, 9, 0, 4, 0, NULL, 0) == MAMBA_OK);
  CHECK(mamba_conv_fwd(1, 1, 8, 4, 0, F, M, NULL, NULL, NULL, NULL, 1, F, NULL, NULL) == MAMBA_ERR_ALIGN);
  CHECK(mamba_conv_fwd(0, 9, 8, 4, 0, NULL, NULL, NULL, NULL, NULL, NULL, 1, NULL, NULL, NULL) == MAMBA_OK);
  CHECK(mamba_conv_fwd(2, 0, 8, 4, 0, NULL, NULL, NULL, NULL, NULL, NULL, 1, NULL, NULL, NULL) == MAMBA_OK);
  CHECK(mamba_conv_update(2, 8, 4, 0, 1, F, F, F, NULL, NULL, 1, F, NULL) == MAMBA_ERR_DIM);
  CHECK(mamba_conv_update(2, 8, 4, 0, INT64_MAX, F, F, F, NULL, F, 1, F, NULL) == MAMBA_ERR_DIM);
  CHECK(mamba_conv_update(0, 8, 4, 0, 0, NULL, NULL, NULL, NULL, NULL, 1, NULL, NULL) == MAMBA_OK);
  CHECK(step(2, 8, 3, 4, 4, 0, 2, F, 0) == MAMBA_ERR_UNSUPPORTED && step(2, 8, 16, 0, 4, 0, 2, F, 0) == MAMBA_ERR_DIM);
  CHECK(step(2, 8, 16, 4, 5, 0, 2, F, 0) == MAMBA_ERR_UNSUPPORTED && step(2, 8, 16, 4, 4, 0, -1, F, 0) == MAMBA_ERR_DIM);
  CHECK(step(2, 8, 16, 4, 4, 0, 2, NULL, 0) == MAMBA_ERR_NULL && step(2, 8, 16, 4, 4, 0, 2, M, 0) == MAMBA_ERR_ALIGN);
  CHECK(norm_bwd(2, 8, 0, 1, F, 1.0f, 1e-5f, 0) == MAMBA_ERR_DTYPE && norm_bwd(2, 0, 0, 0, F, 1.0f, 1e-5f, 0) == MAMBA_ERR_DIM);
  CHECK(norm_bwd(2, 8, 0, 0, F, NAN, 1e-5f, 0) == MAMBA_ERR_OPTION && norm_bwd(2, 8, 0, 0, F, 1.0f, 0.0f, 0) == MAMBA_ERR_OPTION);
  CHECK(norm_bwd(2, 8, 0, 0, NULL, 1.0f, 1e-5f, 0) == MAMBA_ERR_NULL && norm_bwd(2, 8, 0, 0, M, 1.0f, 1e-5f, 0) == MAMBA_ERR_ALIGN);
  CHECK(mamba_residual_norm_fwd(2, 8, 0, 0, F, NULL, 1, NULL, NULL, NULL, F, 1.0f, 1e-5f, NULL, NULL, NULL) == MAMBA_ERR_NULL);
  CHECK(mamba_residual_norm_fwd(2, 8, 0, 0, F, NULL, 1, NULL, NULL, NULL, NULL, 1.0f, 1e-5f, NULL, NULL, NULL) == MAMBA_OK);
  CHECK(verify(1, 4097, 9, 0, F, 0) == MAMBA_ERR_DIM && verify(1, 1, 0, 0, F, 0) == MAMBA_ERR_DIM);
  CHECK(verify(1, 1, 9, 0, NULL, 0) == MAMBA_ERR_NULL && verify(1, 1, 9, 0, M, 0) == MAMBA_ERR_ALIGN);
  if (fails) {
    fprintf(stderr, "%d checks failed\n", fails);
    return 1;
  }
  printf("all checks passed\n");
  return 0;
}
