/* Host-side checks of the token-model operators' C ABI (include/mamba_mi355x_lm.h) for a build of the
 * library whose host code carries AddressSanitizer and UndefinedBehaviorSanitizer
 * (tests/test_lm_sanitizers.py).  Every call here is rejected or answered on the host before the HIP
 * runtime is touched; no GPU is needed.  The fake device pointers are never dereferenced. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>

#include "mamba_mi355x_lm.h"

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

static int scan(int64_t b, int64_t l, int64_t d, int io, void* u, float c, size_t bytes) {
  return mamba_gated_scan_fwd(b, l, d, io, u, F, F, F, c, NULL, NULL, NULL, F, NULL, NULL, bytes ? F : NULL, bytes, NULL);
}
static int back(int64_t b, int64_t l, int64_t d, int io, void* u, float c, size_t bytes) {
  return mamba_gated_scan_bwd(b, l, d, io, u, F, F, F, c, NULL, NULL, NULL, NULL, F, NULL, F, F, F, F, NULL, NULL,
                              bytes ? F : NULL, bytes, NULL);
}

int main(void) {
  const int64_t sizes[] = {INT64_MIN, -1, 0, 1, 7, 8, 63, 64, 65, 4096, 65535, 65536, 4194304, 4194305,
                           INT32_MAX, (int64_t)INT32_MAX + 1, (int64_t)1 << 40, ((int64_t)1 << 40) + 1, INT64_MAX};
  const int n = (int)(sizeof sizes / sizeof sizes[0]);
  /* every combination of sizes: a workspace or a refusal, no overflow on the way */
  for (int i = 0; i < n; ++i)
    for (int j = 0; j < n; ++j)
      for (int k = 0; k < n; ++k)
        for (int io = -1; io < 3; ++io) {
          const int64_t a = sizes[i], b = sizes[j], c = sizes[k];
          const size_t f = mamba_gated_scan_fwd_workspace_size(a, b, c, io);
          const size_t w = mamba_gated_scan_bwd_workspace_size(a, b, c, io);
          const size_t e = mamba_embed_bwd_workspace_size(a, b, c, io);
          const int positive = a > 0 && b > 0 && c > 0 && (io == 0 || io == 1);
          if (!positive) CHECK(f == 0 && w == 0 && e == 0);
          CHECK(f < ((size_t)1 << 60) && w < ((size_t)1 << 60) && e < ((size_t)1 << 60) && f <= w);
          if (w) CHECK(back(a, b, c, io, F, 8.0f, w - 1) == MAMBA_ERR_WORKSPACE);
          else CHECK(!positive || back(a, b, c, io, F, 8.0f, 1) == MAMBA_ERR_DIM);
          if (f) CHECK(scan(a, b, c, io, F, 8.0f, f - 1) == MAMBA_ERR_WORKSPACE);
          if (e) CHECK(mamba_embed_bwd(a, b, c, io, F, F, 1.0f, F, F, e - 1, NULL) == MAMBA_ERR_WORKSPACE);
          else CHECK(!positive || mamba_embed_bwd(a, b, c, io, F, F, 1.0f, F, F, 1, NULL) == MAMBA_ERR_DIM);
        }
  CHECK(scan(1, 1, 8, 2, F, 8.0f, 0) == MAMBA_ERR_DTYPE && scan(1, 1, 8, 0, M, 8.0f, 0) == MAMBA_ERR_ALIGN);
  CHECK(scan(1, 1, 8, 0, NULL, 8.0f, 0) == MAMBA_ERR_NULL && back(1, 1, 8, 0, NULL, 8.0f, 0) == MAMBA_ERR_NULL);
  CHECK(scan(1, 1, 8, 0, F, NAN, 0) == MAMBA_ERR_OPTION && back(1, 1, 8, 0, F, INFINITY, 0) == MAMBA_ERR_OPTION);
  CHECK(scan(0, 9, 8, 0, NULL, 8.0f, 0) == MAMBA_OK && back(2, 9, 0, 0, NULL, 8.0f, 0) == MAMBA_OK);
  CHECK(mamba_gated_state_update(65536, 8, 0, F, F, F, F, F, 8.0f, NULL, NULL, F, NULL) == MAMBA_ERR_DIM);
  CHECK(mamba_gated_state_update(2, 8, 0, M, F, F, F, F, 8.0f, NULL, NULL, F, NULL) == MAMBA_ERR_ALIGN);
  CHECK(mamba_gated_state_update(2, 8, 0, F, F, F, F, F, 0.0f, NULL, NULL, F, NULL) == MAMBA_ERR_OPTION);
  CHECK(mamba_gated_state_update(0, 8, 0, NULL, NULL, NULL, NULL, NULL, 8.0f, NULL, NULL, NULL, NULL) == MAMBA_OK);
  CHECK(mamba_embed_fwd(5, 7, 8, 0, NULL, F, 1.0f, F, NULL) == MAMBA_ERR_NULL);
  CHECK(mamba_embed_fwd(5, 7, 8, 0, F, F, NAN, F, NULL) == MAMBA_ERR_OPTION);
  CHECK(mamba_embed_fwd(5, INT64_MAX, 8, 0, F, F, 1.0f, F, NULL) == MAMBA_ERR_DIM);
  CHECK(mamba_embed_fwd(0, 7, 8, 0, NULL, NULL, 1.0f, NULL, NULL) == MAMBA_OK);
  for (int i = 0; i < n; ++i)
    for (int j = 0; j < n; ++j) {
      const int ok = sizes[i] >= 0 && sizes[i] <= (1 << 20) && sizes[j] >= 1 && sizes[j] <= (1 << 20);
      const int st = mamba_sample(sizes[i], sizes[j], 0, NULL, F, NULL, NULL, NULL, NULL, F, NULL, NULL);
      CHECK(st == (!ok ? MAMBA_ERR_DIM : sizes[i] == 0 ? MAMBA_OK : MAMBA_ERR_NULL));
    }
  CHECK(mamba_sample(1, 8, 0, F, F, M, NULL, NULL, NULL, F, NULL, NULL) == MAMBA_ERR_ALIGN);
  if (fails == 0) printf("all checks passed\n");
  return fails != 0;
}
