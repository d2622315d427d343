// Attention of a few rows over the 8-bit cache under a tree.
#include "kv8_attend_few.cuh"

namespace ea {
template cudaError_t launch_kv8_few<true, 128, true>(const kv8::AttendParams<kv8::ByQuery>& p, int sms, cudaStream_t s);
template cudaError_t launch_kv8_few<true, 64, true>(const kv8::AttendParams<kv8::ByQuery>& p, int sms, cudaStream_t s);
template cudaError_t launch_kv8_few<false, 128, true>(const kv8::AttendParams<kv8::ByQuery>& p, int sms, cudaStream_t s);
template cudaError_t launch_kv8_few<false, 64, true>(const kv8::AttendParams<kv8::ByQuery>& p, int sms, cudaStream_t s);
}  // namespace ea
