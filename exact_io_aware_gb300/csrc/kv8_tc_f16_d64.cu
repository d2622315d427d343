// Attention of many rows over the 8-bit cache: f16, head dimension 64.
#include "kv8_tc.cuh"

namespace ea {
template cudaError_t launch_kv8_tc<false, 64>(kv8::AttendParams<kv8::ByHead>& p, cudaStream_t s);
}  // namespace ea
