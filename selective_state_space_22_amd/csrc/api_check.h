// api_check.h -- host-side argument checks shared by the C-ABI files.  Not installed.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <cstdio>
#include <cstdlib>

#include "../../include/mamba_mi355x.h"

namespace s6 {

constexpr int64_t kMaxBatch = 65535;
constexpr int64_t kMaxDim = int64_t(1) << 22;

inline bool debug_enabled() {
  static const bool on = [] {
    const char* v = std::getenv("MAMBA_MI355X_DEBUG");
    return v && v[0] && v[0] != '0';
  }();
  return on;
}

inline int fail(int status, const char* where, const char* what) {
  if (debug_enabled()) std::fprintf(stderr, "[mamba_mi355x] %s: %s (%s)\n", where, mamba_status_string(status), what);
  return status;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct PtrCheck {
  const char* where;
  int status = MAMBA_OK;
  // A tensor that must be present when `needed`; any present pointer must be aligned.
  void req(const void* p, bool needed, const char* name) {
    if (status != MAMBA_OK) return;
    if (!p && needed) status = fail(MAMBA_ERR_NULL, where, name);
    else if (p && !aligned16(p)) status = fail(MAMBA_ERR_ALIGN, where, name);
  }
  void opt(const void* p, const char* name) { req(p, false, name); }
};

}  // namespace s6
