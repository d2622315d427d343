// Eviction: the tokens that drew the most attention, moved into another cache.
//
// A sequence of len > keep tokens keeps its first `sink`, its last `recent`, and of the middle
// the keep - sink - recent of the largest accumulated weight (ties: the lower position; NaN
// counts as -inf).  The kept tokens keep their order.  Their dequantised values form the
// destination's blocks, each with the least power-of-two scale that holds them.
//
// Two launches.  select: one CTA for each (sequence, head) finds the weight of the last token
// taken, by a radix descent of 8 bits a pass over order-preserving integer keys, then compacts
// the kept positions with a scan.  move: as the append kernel, 128 destination positions a CTA
// and 16 a warp, values in registers between the block's maximum and the conversion.  The move
// is memory-bound (each kept row is read and written once).
#include "kv8_common.cuh"

namespace ea {
namespace kv8 {

constexpr int kSelThreads = 1024;
constexpr int kMoveThreads = 256;

struct EvictParams {
  int Hk, d, cap, block, keep, sink, recent, cap_out;
  const uint8_t* codes[2];
  const float* scales[2];
  const float* weights;
  const int32_t* lengths;
  uint8_t* codes_out[2];
  float* scales_out[2];
  float* weights_out;
  int32_t* lengths_out;
  int32_t* kept;
  uint32_t* status;
};

// Integer whose unsigned order is the order of the weights (NaN lowest, -0 = +0).
__device__ __forceinline__ uint32_t order_key(float w) {
  if (!(w == w)) w = -INFINITY;
  const uint32_t u = __float_as_uint(w + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive sum over the CTA of two counts packed in one word's halves of 64 bits.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* red, uint64_t& total) {
  const int lane = lane_id(), warp = warp_id();
  uint64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) red[warp] = x;
  __syncthreads();
  if (warp == 0) {
    uint64_t t = red[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t y = __shfl_up_sync(0xFFFFFFFFu, t, o);
      if (lane >= o) t += y;
    }
    red[lane] = t;
  }
  __syncthreads();
  total = red[31];
  return x - v + (warp ? red[warp - 1] : 0);
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(EvictParams p) {
  __shared__ uint32_t hist[256];
  __shared__ uint64_t red[32];
  __shared__ uint32_t s_digit, s_left;
  const int bh = blockIdx.x, b = bh / p.Hk, tid = threadIdx.x;
  if (bh % p.Hk == 0 && tid == 0) check_seq(p.lengths, nullptr, b, p.cap, 0, p.status);
  const int len = seq_len(p.lengths, b, p.cap);
  int32_t* kept = p.kept + static_cast<int64_t>(bh) * p.keep;
  const float* w = p.weights + static_cast<int64_t>(bh) * p.cap;
  if (len <= p.keep) {
    for (int i = tid; i < p.keep; i += kSelThreads) kept[i] = i < len ? i : -1;
    return;
  }
  const int lo = p.sink, hi = len - p.recent;  // the middle; hi - lo > want
  const uint32_t want = p.keep - p.sink - p.recent;
  uint32_t prefix = 0, left = want;
  if (want > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int i = lo + tid; i < hi; i += kSelThreads) {
        const uint32_t k = order_key(w[i]);
        if (shift == 24 || (k >> (shift + 8)) == (prefix >> (shift + 8)))
          atomicAdd(&hist[(k >> shift) & 255u], 1u);
      }
      __syncthreads();
      if (tid == 0) {
        uint32_t l = left;
        int dgt = 255;
        while (dgt > 0 && hist[dgt] < l) l -= hist[dgt--];
        s_digit = dgt;
        s_left = l;
      }
      __syncthreads();
      prefix |= s_digit << shift;
      left = s_left;
    }
  }
  // Keys above `prefix` are kept, and the first `left` of those equal to it.
  uint32_t base_above = 0, base_equal = 0;
  for (int i0 = 0; i0 < len; i0 += kSelThreads) {
    const int i = i0 + tid;
    bool above = false, equal = false;
    if (i < len) {
      if (i < lo || i >= hi) {
        above = true;
      } else if (want > 0) {
        const uint32_t k = order_key(w[i]);
        above = k > prefix;
        equal = k == prefix;
      }
    }
    uint64_t total;
    const uint64_t ex = block_scan((static_cast<uint64_t>(equal) << 32) | above, red, total);
    const uint32_t eq = base_equal + static_cast<uint32_t>(ex >> 32);
    const uint32_t ab = base_above + static_cast<uint32_t>(ex);
    if (above || (equal && eq < left)) kept[ab + min(eq, left)] = i;
    base_above += static_cast<uint32_t>(total);
    base_equal += static_cast<uint32_t>(total >> 32);
  }
}

template <int D>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(EvictParams p) {
  constexpr int kLanes = D / 16;           // lanes of one row (16 codes each)
  constexpr int kRowsIt = 32 / kLanes;
  constexpr int kIters = 16 / kRowsIt;
  __shared__ float red[kMoveThreads / 32];
  const int lane = lane_id(), warp = warp_id();
  const int bh = blockIdx.y, b = bh / p.Hk, side = blockIdx.z;
  const int live = min(seq_len(p.lengths, b, p.cap), p.keep);
  if (blockIdx.x == 0 && side == 0 && bh % p.Hk == 0 && threadIdx.x == 0) p.lengths_out[b] = live;
  const int s0 = blockIdx.x * 128;
  if (s0 >= live) return;
  const int p0 = s0 + 16 * warp;
  const int wpb = p.block / 16;
  const int start = s0 + warp / wpb * p.block;
  const int sub = lane / kLanes, col = lane % kLanes * 16;
  const int32_t* kept = p.kept + static_cast<int64_t>(bh) * p.keep;
  const uint8_t* src = p.codes[side] + static_cast<int64_t>(bh) * p.cap * D;
  const float* src_scale = p.scales[side] + static_cast<int64_t>(bh) * (p.cap / p.block);

  uint4 raw[kIters];
  float sc[kIters];
  float amax = 0.0f;
#pragma unroll
  for (int it = 0; it < kIters; ++it) {
    const int pos = p0 + it * kRowsIt + sub;
    raw[it] = make_uint4(0, 0, 0, 0);
    sc[it] = 0.0f;
    if (pos < live) {
      const int from = kept[pos];
      raw[it] = __ldg(reinterpret_cast<const uint4*>(src + static_cast<int64_t>(from) * D + col));
      sc[it] = __ldg(src_scale + from / p.block);
    }
  }
#pragma unroll
  for (int it = 0; it < kIters; ++it) {
    const uint32_t w[4] = {raw[it].x, raw[it].y, raw[it].z, raw[it].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x[4];
      codes_to_float4(w[i], x);
#pragma unroll
      for (int e = 0; e < 4; ++e) amax = fmaxf(amax, finite_abs(x[e] * sc[it]));
    }
  }
  amax = warp_max(amax);
  if (lane == 0) red[warp] = amax;
  __syncthreads();
  if (start >= live) return;
  const int w0 = warp / wpb * wpb;
  for (int w = w0; w < w0 + wpb; ++w) amax = fmaxf(amax, red[w]);
  const float s = pow2(scale_exp(amax));
  const float inv = 1.0f / s;
  if (warp == w0 && lane == 0)
    p.scales_out[side][static_cast<int64_t>(bh) * (p.cap_out / p.block) + start / p.block] = s;
  uint8_t* dst = p.codes_out[side] + static_cast<int64_t>(bh) * p.cap_out * D;
#pragma unroll
  for (int it = 0; it < kIters; ++it) {
    const int pos = p0 + it * kRowsIt + sub;
    if (pos >= live) continue;
    const uint32_t w[4] = {raw[it].x, raw[it].y, raw[it].z, raw[it].w};
    uint32_t out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x[4];
      codes_to_float4(w[i], x);
      out[i] = pack_codes(x[0] * sc[it] * inv, x[1] * sc[it] * inv, x[2] * sc[it] * inv,
                          x[3] * sc[it] * inv);
    }
    *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(pos) * D + col) =
        make_uint4(out[0], out[1], out[2], out[3]);
  }
  if (side == 0) {
    const int pos = p0 + lane;
    if (lane < 16 && pos < live)
      p.weights_out[static_cast<int64_t>(bh) * p.cap_out + pos] =
          p.weights[static_cast<int64_t>(bh) * p.cap + kept[pos]];
  }
}

}  // namespace kv8

int launch_kv8_evict(const Kv8EvictArgs& a, cudaStream_t s, std::string& err) {
  kv8::EvictParams p{a.Hk, a.d, a.cap, a.block, a.keep, a.sink, a.recent, a.cap_out,
                     {a.k8, a.v8}, {a.k_scales, a.v_scales}, a.weights, a.lengths,
                     {a.k8_out, a.v8_out}, {a.k_scales_out, a.v_scales_out}, a.weights_out,
                     a.lengths_out, a.kept, a.status};
  void* args[] = {&p};
  cudaError_t e = cudaLaunchKernel(reinterpret_cast<const void*>(kv8::evict_select_kernel),
                                   dim3(static_cast<unsigned>(a.B * a.Hk)), dim3(kv8::kSelThreads),
                                   args, 0, s);
  if (e == cudaSuccess) {
    const int most = a.keep < a.cap ? a.keep : a.cap;
    const dim3 grid(static_cast<unsigned>((most + 127) / 128), static_cast<unsigned>(a.B * a.Hk), 2);
    auto* kernel = a.d == 128 ? kv8::evict_move_kernel<128> : kv8::evict_move_kernel<64>;
    e = cudaLaunchKernel(reinterpret_cast<const void*>(kernel), grid, dim3(kv8::kMoveThreads), args,
                         0, s);
  }
  if (e != cudaSuccess) {
    err = std::string("kv8 evict launch: ") + cudaGetErrorString(e);
    return -5;
  }
  return 0;
}

}  // namespace ea
