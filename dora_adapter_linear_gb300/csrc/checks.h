// Host-side argument checks and workspace carving shared by the C-ABI entry points.
#pragma once

#include <stddef.h>
#include <stdint.h>
#include <stdlib.h>

#include "../../include/lora_gb300.h"
#include "internal.h"

namespace lg {

constexpr size_t kErrBytes = 256;
inline size_t al256(size_t x) { return (x + 255) & ~size_t(255); }

// Dry-run-able bump allocator over the caller's workspace: with base == nullptr it only sums sizes.
struct Carve {
  char* base;
  size_t off = 0;
  template <typename T>
  T* take(size_t count) {
    char* p = base ? base + off : nullptr;
    off += al256(count * sizeof(T));
    return reinterpret_cast<T*>(p);
  }
};

inline uint64_t wait_timeout_ns() {
  static uint64_t v = 0;
  if (v == 0) {
    const char* e = getenv("LORA_GB300_WAIT_TIMEOUT_MS");
    double ms = e ? atof(e) : 2000.0;
    if (!(ms > 0)) ms = 2000.0;
    v = (uint64_t)(ms * 1e6);
  }
  return v;
}

inline bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
#define CK(x)                                  \
  do {                                         \
    if ((x) != cudaSuccess) return LORA_ERR_CUDA; \
  } while (0)
#define REQ(p)                                   \
  do {                                           \
    if ((p) == nullptr) return LORA_ERR_INVALID_ARG; \
  } while (0)
// tensors whose leading extent is the token count may be NULL when there are no tokens
#define REQM(M, p)                                                \
  do {                                                            \
    if ((M) > 0 && (p) == nullptr) return LORA_ERR_INVALID_ARG;   \
  } while (0)
#define ALN(p)                                   \
  do {                                           \
    if ((p) != nullptr && !al16(p)) return LORA_ERR_MISALIGNED; \
  } while (0)

inline lora_status check_ws(void* ws, size_t have, size_t need) {
  if (ws == nullptr || have < need) return LORA_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(ws) & 255) return LORA_ERR_MISALIGNED;
  return LORA_OK;
}

}  // namespace lg
