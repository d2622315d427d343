// Writing new keys and values into the 8-bit cache.
//
// The cnt new tokens of a sequence take the positions len - cnt .. len - 1.  Each block of
// tokens and head has one scale, the least power of two s with |x| <= 448 s for every finite
// value it holds, and codes E4M3(x / s).  A block that already holds tokens keeps the larger of
// its scale and the one the new tokens need; where that grows, the held codes become
// E4M3(code * old / new) (a power-of-two factor: exact down to E4M3's subnormals).
//
// One CTA takes a span of 128 positions of one head's K or V, each warp 16 of them, so a block
// is one to eight whole warps of one CTA: the values stay in registers between the block's
// maximum and the conversion, and the input is read once.  Memory-bound for prompts (4 x 8 heads of
// up to 8192 tokens, d = 128: 26.7 us, 5.1 TB/s, 77 % of the measured copy rate); for one token a
// sequence it is the latency of its two dependent loads (length, then token and scale; 4 us for 256
// heads).
#include "kv8_common.cuh"

namespace ea {
namespace kv8 {

constexpr int kSpan = 128;
constexpr int kAppendThreads = 256;

struct AppendParams {
  int n, cap, block, Hk;
  const void* x[2];
  uint8_t* codes[2];
  float* scales[2];
  const int32_t* lengths;
  const int32_t* counts;
  float* weights;
  uint32_t* status;
};

// Largest magnitude of a 16-bit pair as bit patterns (ordered as the values are, not finite above
// all that is); `most` accumulates both halves.
__device__ __forceinline__ void pair_max(uint32_t& most, uint32_t w) { most = __vmaxu2(most, w & 0x7FFF7FFFu); }

template <bool kBf16, int D>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(AppendParams p) {
  constexpr int kLanes = D / 8;            // lanes of one row (16 bytes of input each)
  constexpr int kRowsIt = 32 / kLanes;     // rows a warp takes at once
  constexpr int kIters = 16 / kRowsIt;
  constexpr uint32_t kInf = kBf16 ? 0x7F80u : 0x7C00u;
  __shared__ float red[kAppendThreads / 32];
  const int lane = lane_id(), warp = warp_id();
  const int bh = blockIdx.y, b = bh / p.Hk, side = blockIdx.z;
  const int len = seq_len(p.lengths, b, p.cap);
  const int cnt = seq_count(p.counts, b, p.n);
  const int first = len - cnt;  // may lie below 0 (tokens there have no place and are dropped)
  const int from = max(first, 0);
  if (blockIdx.x == 0 && side == 0 && bh % p.Hk == 0 && threadIdx.x == 0) {
    check_seq(p.lengths, p.counts, b, p.cap, p.n, p.status);
    if (first < 0) raise_clamped(p.status);
  }
  const int s0 = (from / kSpan + blockIdx.x) * kSpan;
  if (s0 >= len || from >= len) return;
  const int p0 = s0 + 16 * warp;
  const int wpb = p.block / 16;
  const int start = s0 + warp / wpb * p.block;
  const bool takes = start < len && start + p.block > from;
  const bool holds = takes && from > start;

  const uint16_t* src = static_cast<const uint16_t*>(side ? p.x[1] : p.x[0]) + static_cast<int64_t>(bh) * p.n * D;
  uint8_t* dst = (side ? p.codes[1] : p.codes[0]) + static_cast<int64_t>(bh) * p.cap * D;
  float* scale = (side ? p.scales[1] : p.scales[0]) + static_cast<int64_t>(bh) * (p.cap / p.block) + start / p.block;
  const int sub = lane / kLanes, col = lane % kLanes * 8;

  const float old = holds ? *scale : 0.0f;
  uint4 raw[kIters];
  uint32_t most = 0;
#pragma unroll
  for (int it = 0; it < kIters; ++it) {
    const int pos = p0 + it * kRowsIt + sub;
    raw[it] = make_uint4(0, 0, 0, 0);
    if (pos >= from && pos < len)
      raw[it] = __ldg(reinterpret_cast<const uint4*>(src + static_cast<int64_t>(pos - first) * D + col));
  }
#pragma unroll
  for (int it = 0; it < kIters; ++it) {
    pair_max(most, raw[it].x);
    pair_max(most, raw[it].y);
    pair_max(most, raw[it].z);
    pair_max(most, raw[it].w);
  }
  most = __reduce_max_sync(0xFFFFFFFFu, max(most >> 16, most & 0xFFFFu));
  const bool strange = most >= kInf;  // of the whole warp: some value is not finite
  float amax;
  if (!strange) {
    amax = unpack16<kBf16>(most).x;
  } else {
    amax = 0.0f;
#pragma unroll
    for (int it = 0; it < kIters; ++it) {
      const uint32_t w[4] = {raw[it].x, raw[it].y, raw[it].z, raw[it].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpack16<kBf16>(w[i]);
        amax = fmaxf(amax, fmaxf(finite_abs(f.x), finite_abs(f.y)));
      }
    }
    amax = warp_max(amax);
  }
  if (lane == 0) red[warp] = amax;
  __syncthreads();
  if (!takes) return;
  const int w0 = warp / wpb * wpb;
  for (int w = w0; w < w0 + wpb; ++w) amax = fmaxf(amax, red[w]);
  float s = pow2(scale_exp(amax));
  if (holds && !(old < s)) s = old;
  const float inv = 1.0f / s;
  if (warp == w0 && lane == 0) *scale = s;

  const bool grow = holds && s != old;
  const float ratio = old * inv;
#pragma unroll
  for (int it = 0; it < kIters; ++it) {
    const int pos = p0 + it * kRowsIt + sub;
    uint2* out = reinterpret_cast<uint2*>(dst + static_cast<int64_t>(pos) * D + col);
    if (pos >= from && pos < len) {
      const uint32_t w[4] = {raw[it].x, raw[it].y, raw[it].z, raw[it].w};
      float2 f[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[i] = unpack16<kBf16>(w[i]);
        if (strange) {
          f[i].x = nan_unless_finite(f[i].x);
          f[i].y = nan_unless_finite(f[i].y);
        }
        f[i].x *= inv;
        f[i].y *= inv;
      }
      *out = make_uint2(pack4_e4m3(f[0].x, f[0].y, f[1].x, f[1].y),
                        pack4_e4m3(f[2].x, f[2].y, f[3].x, f[3].y));
    } else if (grow && pos >= start && pos < from) {
      const uint2 c = *out;
      float u[4], v[4];
      codes_to_float4(c.x, u);
      codes_to_float4(c.y, v);
      *out = make_uint2(pack_codes(u[0] * ratio, u[1] * ratio, u[2] * ratio, u[3] * ratio),
                        pack_codes(v[0] * ratio, v[1] * ratio, v[2] * ratio, v[3] * ratio));
    }
  }
  if (p.weights && side == 0) {
    const int pos = p0 + lane;
    if (lane < 16 && pos >= from && pos < len)
      p.weights[static_cast<int64_t>(bh) * p.cap + pos] = 0.0f;
  }
}

}  // namespace kv8

int launch_kv8_append(const Kv8Args& a, cudaStream_t s, std::string& err) {
  kv8::AppendParams p{a.n, a.cap, a.block, a.Hk, {a.k_new, a.v_new}, {a.k8, a.v8},
                      {a.k_scales, a.v_scales}, a.lengths, a.counts, a.weights_out, a.status};
  // n tokens at any place touch at most (n + 254) / 128 spans of 128.
  const dim3 grid(static_cast<unsigned>((static_cast<int64_t>(a.n) + 254) / kv8::kSpan),
                  static_cast<unsigned>(a.B * a.Hk), 2);
  auto* kernel = a.bf16 ? (a.d == 128 ? kv8::append_kernel<true, 128> : kv8::append_kernel<true, 64>)
                        : (a.d == 128 ? kv8::append_kernel<false, 128> : kv8::append_kernel<false, 64>);
  void* args[] = {&p};
  const cudaError_t e = cudaLaunchKernel(reinterpret_cast<const void*>(kernel), grid,
                                         dim3(kv8::kAppendThreads), args, 0, s);
  if (e != cudaSuccess) {
    err = std::string("kv8 append launch: ") + cudaGetErrorString(e);
    return -5;
  }
  return 0;
}

}  // namespace ea
