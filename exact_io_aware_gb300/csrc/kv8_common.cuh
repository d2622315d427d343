// Device building blocks of the 8-bit key/value cache kernels.
//
// The cache of one sequence and key/value head is cap rows of D E4M3 codes for K and for V, and
// one float32 scale for each `block` consecutive tokens (block 16, 32, 64 or 128, so a block
// never straddles a 128-token span).  Scales the library writes are powers of two: E4M3 is a
// floating-point format, so a power-of-two scale keeps the full relative precision of 2^-4, and
// moving codes to another block's scale (growth in place, eviction) is exact unless a value
// falls among E4M3's subnormals.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cstdint>

#include "kv8.h"
#include "ptx.cuh"

namespace ea {
namespace kv8 {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ------------------------------------------------------------------ launches in sequence

// A kernel launched with launch_after may start while the one before it still runs.  The first
// lets it (grid_launch_dependents) and the second waits, before it touches what the first
// writes, until the first has finished and its writes are visible (grid_dependency_wait).
__device__ __forceinline__ void grid_launch_dependents() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void grid_dependency_wait() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
inline cudaError_t launch_after(const void* kernel, dim3 grid, dim3 block, void** args, cudaStream_t s) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, kernel, args);
}

// Lets `kernel` have `bytes` of dynamic shared memory on the current device, asked of the runtime
// once a device (`done`: a bit for each, the caller's own for this kernel).
inline cudaError_t allow_smem(const void* kernel, size_t bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// ------------------------------------------------------------------ sequences

// Length and new-token count of sequence b, clamped to the buffers they index; a value outside
// its range raises the status flag (from one lane per call site that asks for it).
__device__ __forceinline__ int seq_len(const int32_t* lengths, int b, int cap) {
  return min(max(__ldg(lengths + b), 0), cap);
}
__device__ __forceinline__ int seq_count(const int32_t* counts, int b, int n) {
  return counts ? min(max(__ldg(counts + b), 0), n) : n;
}
__device__ __forceinline__ void check_seq(const int32_t* lengths, const int32_t* counts, int b,
                                          int cap, int n, uint32_t* status) {
  const int len = __ldg(lengths + b);
  const int cnt = counts ? __ldg(counts + b) : 0;
  if (len < 0 || len > cap || cnt < 0 || cnt > n) raise_clamped(status);
}

// ------------------------------------------------------------------ codes and scales

// Two E4M3 codes (low byte first) to two fp16 values, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}
__device__ __forceinline__ uint32_t lo_codes(uint32_t w) {
  return e4m3x2_to_f16x2(static_cast<uint16_t>(w & 0xFFFFu));
}
__device__ __forceinline__ uint32_t hi_codes(uint32_t w) {
  return e4m3x2_to_f16x2(static_cast<uint16_t>(w >> 16));
}
__device__ __forceinline__ void codes_to_float4(uint32_t w, float (&x)[4]) {
  const uint32_t a = lo_codes(w), b = hi_codes(w);
  const float2 u = __half22float2(*reinterpret_cast<const __half2*>(&a));
  const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&b));
  x[0] = u.x, x[1] = u.y, x[2] = v.x, x[3] = v.y;
}

// The same in E5M2: four floats to a word of codes, and back.
__device__ __forceinline__ uint32_t pack4_e5m2(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}
__device__ __forceinline__ void e5m2_to_float4(uint32_t w, float (&x)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t r;
    asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(w >> (16 * i))));
    const float2 u = __half22float2(*reinterpret_cast<const __half2*>(&r));
    x[2 * i] = u.x, x[2 * i + 1] = u.y;
  }
}

// Exponent of the least power of two s with amax <= 448 s, within [least, 120].  448 = 1.75 2^8,
// so for amax = m 2^e (1 <= m < 2) it is e - 8, one more when m > 1.75.
__device__ __forceinline__ int scale_exp(float amax, int least = -100) {
  const uint32_t u = __float_as_uint(amax);
  const int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(e, least), 120);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// |x| where x is finite, else 0 (what a block's scale is taken over).
__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < INFINITY ? a : 0.0f;
}
// x, or NaN where x is not finite: E4M3 has no infinity, and the conversion saturates.
__device__ __forceinline__ float nan_unless_finite(float x) {
  return fabsf(x) < INFINITY ? x : __uint_as_float(0x7FC00000u);
}
__device__ __forceinline__ uint32_t pack_codes(float a, float b, float c, float d) {
  return pack4_e4m3(nan_unless_finite(a), nan_unless_finite(b), nan_unless_finite(c),
                    nan_unless_finite(d));
}

// Two 16-bit inputs of one word as floats.
template <bool kBf16>
__device__ __forceinline__ float2 unpack16(uint32_t w) {
  if constexpr (kBf16) return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

}  // namespace kv8
}  // namespace ea
