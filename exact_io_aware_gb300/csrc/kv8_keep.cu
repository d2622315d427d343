// Bringing the 8-bit cache from a tree of drafted tokens to the accepted ones.
//
// The tree's cnt tokens lie at the end of a sequence, from position first = len - cnt on.  Accepted
// token i moves from position first + path[i] to first + i, and its values are quantized again there
// by the append rule: a block's scale is the least power of two s with |x| <= 448 s for every value x
// that moves into it, and a block that also holds tokens before the tree keeps the larger of that and
// its own scale.  Between powers of two a code changes exactly, down to E4M3's subnormals.
//
// In place: no token moves up (path[i] >= i, which ascending nodes fulfil and others are made to), so
// a CTA that takes one head's K or V in spans of 128 positions from the front, each read before it is
// written, finds every later token and its scale as they were: they lie past all it has written.
//
// Bound by the latency of its dependent loads (lengths, path, then codes and scales): 128 heads of d = 128
// with up to 8 accepted tokens 5.2 us; 512 heads, where the accepted tokens may take two spans, 9.5 us.
#include "kv8_common.cuh"

namespace ea {
namespace kv8 {

constexpr int kKeepThreads = 256;

struct KeepParams {
  int n, cap, block, Hk;
  uint8_t* codes[2];
  float* scales[2];
  const int32_t* lengths;
  const int32_t* counts;
  const int32_t* path;
  const int32_t* accepted;
  float* weights;
  int32_t* lengths_out;
  uint32_t* status;
};

template <int D>
__global__ void __launch_bounds__(kKeepThreads) keep_kernel(KeepParams p) {
  constexpr int kSpan = 128;
  constexpr int kLanes = D / 8;         // lanes of one row (8 codes each)
  constexpr int kRowsIt = 32 / kLanes;  // rows a warp takes at once
  constexpr int kIters = 16 / kRowsIt;
  // Values are handled over 2^8: those under the largest scales would leave float32.
  constexpr float kDown = 1.0f / 256.0f, kUp = 256.0f;
  __shared__ float red[kKeepThreads / 32];
  const int lane = lane_id(), warp = warp_id();
  const int bh = blockIdx.x, b = bh / p.Hk, side = blockIdx.y;
  const int len = seq_len(p.lengths, b, p.cap), cnt = seq_count(p.counts, b, p.n);
  const int asked = __ldg(p.accepted + b), acc = min(max(asked, 0), cnt);
  const int first = len - cnt;  // may lie below 0 (tokens there have no place)
  const int from = max(first, 0), end = first + acc;
  if (side == 0 && bh % p.Hk == 0 && threadIdx.x == 0) {
    check_seq(p.lengths, p.counts, b, p.cap, p.n, p.status);
    if (asked != acc) raise_clamped(p.status);
    p.lengths_out[b] = max(end, 0);
  }
  uint8_t* codes = (side ? p.codes[1] : p.codes[0]) + static_cast<int64_t>(bh) * p.cap * D;
  float* scales = (side ? p.scales[1] : p.scales[0]) + static_cast<int64_t>(bh) * (p.cap / p.block);
  float* weights = p.weights ? p.weights + static_cast<int64_t>(bh) * p.cap : nullptr;
  const int32_t* path = p.path + static_cast<int64_t>(b) * p.n;
  const int shift = 31 - __clz(p.block), wpb = p.block / 16;
  const int sub = lane / kLanes, col = lane % kLanes * 8;

  for (int s0 = from / kSpan * kSpan; s0 < end; s0 += kSpan) {
    const int p0 = s0 + 16 * warp;
    const int start = s0 + warp / wpb * p.block;
    const bool takes = start < end && start + p.block > from;
    const bool holds = takes && from > start;
    const float old = holds ? scales[start >> shift] : 0.0f;
    // Where the warp's 16 positions come from: -1 for those that are not written.
    int src16 = -1;
    {
      const int pos = p0 + (lane & 15);
      if (pos >= from && pos < end) {
        const int i = pos - first, node = __ldg(path + i), to = min(max(node, i), cnt - 1);
        if (node != to) raise_clamped(p.status);
        src16 = first + to;
      }
    }
    const float weight = weights && side == 0 && lane < 16 && src16 >= 0 ? weights[src16] : 0.0f;
    uint2 raw[kIters];
    float sc[kIters], amax = 0.0f;
#pragma unroll
    for (int it = 0; it < kIters; ++it) {
      const int src = __shfl_sync(0xFFFFFFFFu, src16, it * kRowsIt + sub);
      raw[it] = make_uint2(0u, 0u);
      sc[it] = 0.0f;
      if (src >= 0) {
        raw[it] = *reinterpret_cast<const uint2*>(codes + static_cast<int64_t>(src) * D + col);
        sc[it] = scales[src >> shift] * kDown;
      }
    }
    // (a warp into whose positions nothing moves has nothing to look at)
    if (__any_sync(0xFFFFFFFFu, src16 >= 0)) {
#pragma unroll
      for (int it = 0; it < kIters; ++it) {
        float x[4], y[4];
        codes_to_float4(raw[it].x, x);
        codes_to_float4(raw[it].y, y);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          amax = fmaxf(amax, fmaxf(finite_abs(x[e] * sc[it]), finite_abs(y[e] * sc[it])));
      }
      amax = warp_max(amax);
    }
    if (lane == 0) red[warp] = amax;
    __syncthreads();  // the span is read
    if (takes) {
      const int w0 = warp / wpb * wpb;
      for (int w = w0; w < w0 + wpb; ++w) amax = fmaxf(amax, red[w]);
      float s = pow2(min(max(scale_exp(amax, -120) + 8, -100), 120));
      if (holds && !(old < s)) s = old;
      const float inv = 1.0f / s * kUp;
      if (warp == w0 && lane == 0) scales[start >> shift] = s;
      const bool grow = holds && s != old;
      const float ratio = old * (1.0f / s);
#pragma unroll
      for (int it = 0; it < kIters; ++it) {
        const int pos = p0 + it * kRowsIt + sub;
        uint2* out = reinterpret_cast<uint2*>(codes + static_cast<int64_t>(pos) * D + col);
        const bool moved = pos >= from && pos < end, held = grow && pos >= start && pos < from;
        if (!moved && !held) continue;
        const uint2 c = moved ? raw[it] : *out;
        const float f = moved ? sc[it] : ratio, g = moved ? inv : 1.0f;
        float u[4], v[4];
        codes_to_float4(c.x, u);
        codes_to_float4(c.y, v);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          u[e] = u[e] * f * g;
          v[e] = v[e] * f * g;
        }
        *out = make_uint2(pack_codes(u[0], u[1], u[2], u[3]), pack_codes(v[0], v[1], v[2], v[3]));
      }
      if (weights && side == 0 && lane < 16 && src16 >= 0) weights[p0 + lane] = weight;
    }
    __syncthreads();  // red is read
  }
}

}  // namespace kv8

int launch_kv8_keep(const Kv8KeepArgs& a, cudaStream_t s, std::string& err) {
  kv8::KeepParams p{a.n, a.cap, a.block, a.Hk, {a.k8, a.v8}, {a.k_scales, a.v_scales}, a.lengths, a.counts,
                    a.path, a.accepted, a.weights, a.lengths_out, a.status};
  auto* kernel = a.d == 128 ? kv8::keep_kernel<128> : kv8::keep_kernel<64>;
  void* args[] = {&p};
  const cudaError_t e = cudaLaunchKernel(reinterpret_cast<const void*>(kernel),
                                         dim3(static_cast<unsigned>(a.B) * a.Hk, 2), dim3(kv8::kKeepThreads),
                                         args, 0, s);
  if (e != cudaSuccess) {
    err = std::string("kv8 keep launch: ") + cudaGetErrorString(e);
    return -5;
  }
  return 0;
}

}  // namespace ea
