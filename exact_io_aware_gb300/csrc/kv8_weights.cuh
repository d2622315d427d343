// Arguments of the kernels that accumulate attention weights.
#pragma once
#include "kv8_plan.cuh"

namespace ea {
namespace kv8 {

template <class Geo>
struct WeightsParams {
  Geo geo;  // one tile of all rows
  int block;
  float c2;  // c log2(e)
  const uint16_t* q;
  const uint8_t* k8;
  const float* k_scales;
  const float* lse;
  const float* w_in;  // null: zeros
  float* w_out;
  uint32_t* status;
};

}  // namespace kv8

// The kernel for many rows (kv8_weights_tc.cu).
template <bool kBf16, int D>
cudaError_t launch_kv8_weights_tc(kv8::WeightsParams<kv8::ByHead> p, int sms, cudaStream_t s);

}  // namespace ea
