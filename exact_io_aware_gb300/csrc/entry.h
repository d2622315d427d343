// What the C entry points share: errors as codes with a message, and a range for timeline tools.
#pragma once
#include <nvtx3/nvToolsExt.h>

#include <cstddef>
#include <cstdint>
#include <string>

#include "exactattn.h"
#include "kernels.h"

namespace ea {

// Sets the calling thread's message; returns the code.
inline int fail(int code, const std::string& msg) {
  set_last_error(msg);
  return code;
}

// An NVTX range named after the entry point, open for the length of the host call (the range
// marks the call's argument checks and launches in a timeline; the kernels are asynchronous).
struct CallRange {
  explicit CallRange(const char* name) { nvtxRangePushA(name); }
  ~CallRange() { nvtxRangePop(); }
  CallRange(const CallRange&) = delete;
  CallRange& operator=(const CallRange&) = delete;
};

// Runs an entry point's body; a C++ exception (memory for a message, a mutex) becomes a code.
template <typename F>
int entry(const char* name, F&& body) noexcept {
  CallRange range(name);
  try {
    return body();
  } catch (...) {
    return ATTN_ERR_CUDA;
  }
}

// A launcher's outcome as the entry point's.  The runtime keeps a refused launch as its last error;
// it is taken here, so that no later call reads it as its own.
inline int outcome(int rc, const std::string& err) {
  if (rc == 0) return ATTN_OK;
  (void)cudaGetLastError();
  return fail(rc, err);
}

inline bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// Bytes [p, p + n) and [q, q + m) share a byte.
inline bool overlap(const void* p, size_t n, const void* q, size_t m) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + m && b < a + n;
}

}  // namespace ea
