// What the C entry points share: errors as codes with a message, and a range for timeline tools.
#pragma once
#include <nvtx3/nvToolsExt.h>

#include <string>

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

}  // namespace ea
