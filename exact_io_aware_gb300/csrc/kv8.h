// Internal interface of the 8-bit key/value cache operators (kv8_api.cu and the kernels).
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <string>

namespace ea {

// The cache and the call's tokens; pointers are device pointers.
struct Kv8Args {
  int B, Hk, G;      // sequences, key/value heads, query heads of each key/value head
  int n;             // new tokens (append) or query rows (attend, weights) of each sequence
  int d, cap, block;
  bool bf16;         // type of the 16-bit inputs and outputs (else fp16)
  bool causal;
  float c;
  const void* q;
  const void* k_new;
  const void* v_new;
  uint8_t* k8;
  uint8_t* v8;
  float* k_scales;
  float* v_scales;
  const int32_t* lengths;
  const int32_t* counts;  // null: n new tokens in every sequence
  void* o;
  float* lse;
  const float* weights;
  float* weights_out;
  void* workspace;
  uint32_t* status;
  int sms;
};

// Eviction: the heaviest tokens of one cache into another of capacity cap_out.
struct Kv8EvictArgs {
  int B, Hk, d, cap, block, keep, sink, recent, cap_out;
  const uint8_t* k8;
  const uint8_t* v8;
  const float* k_scales;
  const float* v_scales;
  const float* weights;
  const int32_t* lengths;
  uint8_t* k8_out;
  uint8_t* v8_out;
  float* k_scales_out;
  float* v_scales_out;
  float* weights_out;
  int32_t* lengths_out;
  int32_t* kept;
  uint32_t* status;
  int sms;
};

// Each launcher returns 0 or a negative ATTN_ERR_* code and fills `err` on failure.
int launch_kv8_append(const Kv8Args& a, cudaStream_t s, std::string& err);
int launch_kv8_attend(const Kv8Args& a, cudaStream_t s, std::string& err);
int launch_kv8_weights(const Kv8Args& a, cudaStream_t s, std::string& err);
int launch_kv8_evict(const Kv8EvictArgs& a, cudaStream_t s, std::string& err);

size_t kv8_attend_workspace_bytes(int B, int Hk, int G, int n, int d, int cap, int sms);

}  // namespace ea
