// C entry points of the 8-bit key/value cache: argument checks and dispatch.
// See include/exactattn.h for the contract.
#include <cuda_runtime.h>

#include <cstdint>
#include <exception>
#include <initializer_list>
#include <string>

#include "entry.h"
#include "exactattn.h"
#include "kv8.h"

namespace {

using ea::CallRange;
using ea::fail;

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
int outcome(int rc, const std::string& err) {
  if (rc == 0) return ATTN_OK;
  (void)cudaGetLastError();
  return fail(rc, err);
}

bool misaligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) != 0; }

// Bytes [p, p + n) and [q, q + m) share a byte.
bool overlap(const void* p, size_t n, const void* q, size_t m) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + m && b < a + n;
}

// The largest sizes: heads of a grid's y axis, tokens of a sequence, rows of a key/value head.
constexpr int64_t kMostHeads = 65535, kMostCap = int64_t(1) << 30, kMostRows = int64_t(1) << 24;

int check_cache(int B, int Hk, int d, int cap, int block, std::initializer_list<const void*> codes,
                std::initializer_list<const void*> words) {
  if (B < 1 || Hk < 1 || cap < 1) return fail(ATTN_ERR_INVALID_ARG, "B, H_kv and cap must be positive");
  if (d != 64 && d != 128) return fail(ATTN_ERR_UNSUPPORTED, "head dimension must be 64 or 128");
  if (block != 16 && block != 32 && block != 64 && block != 128)
    return fail(ATTN_ERR_UNSUPPORTED, "block must be 16, 32, 64 or 128");
  if (cap % block != 0) return fail(ATTN_ERR_INVALID_ARG, "cap must be a multiple of block");
  if (cap > kMostCap) return fail(ATTN_ERR_UNSUPPORTED, "cap must be at most 2^30");
  if (static_cast<int64_t>(B) * Hk > kMostHeads)
    return fail(ATTN_ERR_UNSUPPORTED, "B * H_kv must be at most 65535");
  for (const void* p : codes) {
    if (!p) return fail(ATTN_ERR_INVALID_ARG, "null pointer");
    if (misaligned(p, 16)) return fail(ATTN_ERR_ALIGNMENT, "codes and 16-bit arrays must be 16-byte aligned");
  }
  for (const void* p : words) {
    if (!p) return fail(ATTN_ERR_INVALID_ARG, "null pointer");
    if (misaligned(p, 4)) return fail(ATTN_ERR_ALIGNMENT, "float32 and int32 arrays must be 4-byte aligned");
  }
  return ATTN_OK;
}

int check_dtype(int dtype) {
  if (dtype < ATTN_F32 || dtype > ATTN_BF16) return fail(ATTN_ERR_INVALID_ARG, "unknown dtype");
  if (dtype == ATTN_F32)
    return fail(ATTN_ERR_UNSUPPORTED, "the 8-bit cache takes float16 or bfloat16 inputs");
  return ATTN_OK;
}

// Query heads and rows of the attention and weights calls.
int check_query(int H, int Hk, int n_q, int mask_kind, const int32_t* counts) {
  if (n_q < 1 || H < 1) return fail(ATTN_ERR_INVALID_ARG, "H and n_q must be positive");
  if (H % Hk != 0) return fail(ATTN_ERR_INVALID_ARG, "H must be a multiple of H_kv");
  if (static_cast<int64_t>(H / Hk) * n_q > kMostRows)
    return fail(ATTN_ERR_UNSUPPORTED, "H / H_kv * n_q must be at most 2^24");
  if (mask_kind < ATTN_MASK_NONE || mask_kind > ATTN_MASK_BITMAP)
    return fail(ATTN_ERR_INVALID_ARG, "unknown mask kind");
  if (mask_kind == ATTN_MASK_BITMAP)
    return fail(ATTN_ERR_UNSUPPORTED, "the 8-bit cache takes no bitmap mask");
  if (misaligned(counts, 4)) return fail(ATTN_ERR_ALIGNMENT, "counts must be 4-byte aligned");
  return ATTN_OK;
}

ea::Kv8Args cache_args(int B, int Hk, int G, int n, int d, int cap, int block, const int32_t* lengths,
                       const int32_t* counts) {
  ea::Kv8Args a{};
  a.B = B;
  a.Hk = Hk;
  a.G = G;
  a.n = n;
  a.d = d;
  a.cap = cap;
  a.block = block;
  a.lengths = lengths;
  a.counts = counts;
  return a;
}

}  // namespace

extern "C" {

int attn_kv8_append(int dtype, int B, int H_kv, int n_new, int d, int cap, int block,
                    const void* k_new, const void* v_new, const int32_t* lengths,
                    const int32_t* counts, void* k8, void* v8, float* k_scales, float* v_scales,
                    float* weights, void* stream) {
  return entry("attn_kv8_append", [&]() -> int {
    if (int rc = check_dtype(dtype)) return rc;
    if (int rc = check_cache(B, H_kv, d, cap, block, {k_new, v_new, k8, v8},
                             {k_scales, v_scales, lengths}))
      return rc;
    if (n_new < 1) return fail(ATTN_ERR_INVALID_ARG, "n_new must be positive");
    if (n_new > (1 << 30)) return fail(ATTN_ERR_UNSUPPORTED, "n_new must be at most 2^30");
    if (misaligned(counts, 4) || misaligned(weights, 4))
      return fail(ATTN_ERR_ALIGNMENT, "counts and weights must be 4-byte aligned");
    ea::Kv8Args a = cache_args(B, H_kv, 1, n_new, d, cap, block, lengths, counts);
    a.bf16 = dtype == ATTN_BF16;
    a.k_new = k_new;
    a.v_new = v_new;
    a.k8 = static_cast<uint8_t*>(k8);
    a.v8 = static_cast<uint8_t*>(v8);
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.weights_out = weights;
    if (int rc = ea::device_status_word(&a.status)) return rc;
    std::string err;
    const int rc = ea::launch_kv8_append(a, static_cast<cudaStream_t>(stream), err);
    return outcome(rc, err);
  });
}

size_t attn_fwd_kv8_workspace_bytes(int dtype, int B, int H, int H_kv, int n_q, int d, int cap) {
  if (dtype < ATTN_F16 || dtype > ATTN_BF16 || B < 1 || H < 1 || H_kv < 1 || n_q < 1 || cap < 1 ||
      H % H_kv != 0 || (d != 64 && d != 128) || cap % 16 != 0 || cap > kMostCap ||
      static_cast<int64_t>(B) * H_kv > kMostHeads || static_cast<int64_t>(H / H_kv) * n_q > kMostRows)
    return 0;
  return ea::kv8_attend_workspace_bytes(B, H_kv, H / H_kv, n_q, d, cap, ea::device_sm_count());
}

int attn_fwd_kv8(int dtype, int B, int H, int H_kv, int n_q, int d, int cap, int block, float c,
                 const void* q, const void* k8, const void* v8, const float* k_scales,
                 const float* v_scales, const int32_t* lengths, const int32_t* counts,
                 int mask_kind, void* o, float* lse, void* workspace, size_t workspace_bytes,
                 void* stream) {
  return entry("attn_fwd_kv8", [&]() -> int {
    if (int rc = check_dtype(dtype)) return rc;
    if (int rc = check_cache(B, H_kv, d, cap, block, {q, k8, v8, o},
                             {k_scales, v_scales, lengths, lse}))
      return rc;
    if (int rc = check_query(H, H_kv, n_q, mask_kind, counts)) return rc;
    ea::Kv8Args a = cache_args(B, H_kv, H / H_kv, n_q, d, cap, block, lengths, counts);
    a.sms = ea::device_sm_count();
    const size_t need = ea::kv8_attend_workspace_bytes(B, H_kv, a.G, n_q, d, cap, a.sms);
    if (need > 0 && (!workspace || workspace_bytes < need))
      return fail(ATTN_ERR_WORKSPACE, "workspace missing or smaller than attn_fwd_kv8_workspace_bytes");
    if (misaligned(workspace, 16)) return fail(ATTN_ERR_ALIGNMENT, "workspace must be 16-byte aligned");
    if (int rc = ea::device_status_word(&a.status)) return rc;
    if (a.sms < 1) return fail(ATTN_ERR_CUDA, "the device's multiprocessor count is unknown");
    a.bf16 = dtype == ATTN_BF16;
    a.causal = mask_kind == ATTN_MASK_CAUSAL;
    a.c = c;
    a.q = q;
    a.k8 = static_cast<uint8_t*>(const_cast<void*>(k8));
    a.v8 = static_cast<uint8_t*>(const_cast<void*>(v8));
    a.k_scales = const_cast<float*>(k_scales);
    a.v_scales = const_cast<float*>(v_scales);
    a.o = o;
    a.lse = lse;
    a.workspace = workspace;
    std::string err;
    const int rc = ea::launch_kv8_attend(a, static_cast<cudaStream_t>(stream), err);
    return outcome(rc, err);
  });
}

int attn_kv8_weights(int dtype, int B, int H, int H_kv, int n_q, int d, int cap, int block, float c,
                     const void* q, const void* k8, const float* k_scales, const int32_t* lengths,
                     const int32_t* counts, int mask_kind, const float* lse, const float* weights,
                     float* weights_out, void* stream) {
  return entry("attn_kv8_weights", [&]() -> int {
    if (int rc = check_dtype(dtype)) return rc;
    if (int rc = check_cache(B, H_kv, d, cap, block, {q, k8}, {k_scales, lengths, lse, weights_out}))
      return rc;
    if (int rc = check_query(H, H_kv, n_q, mask_kind, counts)) return rc;
    if (misaligned(weights, 4)) return fail(ATTN_ERR_ALIGNMENT, "weights must be 4-byte aligned");
    const size_t bytes = static_cast<size_t>(B) * H_kv * cap * sizeof(float);
    if (weights && weights != weights_out && overlap(weights, bytes, weights_out, bytes))
      return fail(ATTN_ERR_INVALID_ARG, "weights and weights_out must be the same array or disjoint");
    ea::Kv8Args a = cache_args(B, H_kv, H / H_kv, n_q, d, cap, block, lengths, counts);
    if (int rc = ea::device_status_word(&a.status)) return rc;
    a.sms = ea::device_sm_count();
    if (a.sms < 1) return fail(ATTN_ERR_CUDA, "the device's multiprocessor count is unknown");
    a.bf16 = dtype == ATTN_BF16;
    a.causal = mask_kind == ATTN_MASK_CAUSAL;
    a.c = c;
    a.q = q;
    a.k8 = static_cast<uint8_t*>(const_cast<void*>(k8));
    a.k_scales = const_cast<float*>(k_scales);
    a.lse = const_cast<float*>(lse);
    a.weights = weights;
    a.weights_out = weights_out;
    std::string err;
    const int rc = ea::launch_kv8_weights(a, static_cast<cudaStream_t>(stream), err);
    return outcome(rc, err);
  });
}

int attn_kv8_evict(int B, int H_kv, int d, int cap, int block, const void* k8, const void* v8,
                   const float* k_scales, const float* v_scales, const float* weights,
                   const int32_t* lengths, int keep, int sink, int recent, int cap_out,
                   void* k8_out, void* v8_out, float* k_scales_out, float* v_scales_out,
                   float* weights_out, int32_t* lengths_out, int32_t* kept, void* stream) {
  return entry("attn_kv8_evict", [&]() -> int {
    if (int rc = check_cache(B, H_kv, d, cap, block, {k8, v8, k8_out, v8_out},
                             {k_scales, v_scales, weights, lengths, k_scales_out, v_scales_out,
                              weights_out, lengths_out, kept}))
      return rc;
    if (cap_out < 1 || cap_out % block != 0)
      return fail(ATTN_ERR_INVALID_ARG, "cap_out must be a positive multiple of block");
    if (keep < 1 || keep > cap_out) return fail(ATTN_ERR_INVALID_ARG, "keep must lie in 1 .. cap_out");
    if (sink < 0 || recent < 0 || static_cast<int64_t>(sink) + recent > keep)
      return fail(ATTN_ERR_INVALID_ARG, "sink and recent must be non-negative and sum to at most keep");
    const size_t heads = static_cast<size_t>(B) * H_kv;
    struct Range { const void* p; size_t n; };
    const Range in[] = {{k8, heads * cap * d}, {v8, heads * cap * d},
                        {k_scales, heads * (cap / block) * 4}, {v_scales, heads * (cap / block) * 4},
                        {weights, heads * cap * 4}, {lengths, static_cast<size_t>(B) * 4}};
    const Range out[] = {{k8_out, heads * cap_out * d}, {v8_out, heads * cap_out * d},
                         {k_scales_out, heads * (cap_out / block) * 4},
                         {v_scales_out, heads * (cap_out / block) * 4},
                         {weights_out, heads * cap_out * 4}, {lengths_out, static_cast<size_t>(B) * 4},
                         {kept, heads * keep * 4}};
    for (const Range& x : out) {
      for (const Range& y : in)
        if (overlap(x.p, x.n, y.p, y.n))
          return fail(ATTN_ERR_INVALID_ARG, "the output cache must not overlap the input cache");
      for (const Range& y : out)
        if (&x != &y && overlap(x.p, x.n, y.p, y.n))
          return fail(ATTN_ERR_INVALID_ARG, "the outputs must not overlap one another");
    }
    ea::Kv8EvictArgs a{B, H_kv, d, cap, block, keep, sink, recent, cap_out,
                       static_cast<const uint8_t*>(k8), static_cast<const uint8_t*>(v8), k_scales,
                       v_scales, weights, lengths, static_cast<uint8_t*>(k8_out),
                       static_cast<uint8_t*>(v8_out), k_scales_out, v_scales_out, weights_out,
                       lengths_out, kept, nullptr, ea::device_sm_count()};
    if (int rc = ea::device_status_word(&a.status)) return rc;
    std::string err;
    const int rc = ea::launch_kv8_evict(a, static_cast<cudaStream_t>(stream), err);
    return outcome(rc, err);
  });
}

}  // extern "C"
