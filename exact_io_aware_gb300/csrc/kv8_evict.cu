// Eviction: the tokens that drew the most attention, moved into another cache.
//
// A sequence of len > keep tokens keeps its first `sink`, its last `recent`, and of the middle
// the keep - sink - recent of the largest accumulated weight (ties: the lower position; NaN
// counts as -inf).  The kept tokens keep their order.  Their dequantised values form the
// destination's blocks, each with the least power-of-two scale that holds them.
//
// Two launches.  select: a cluster of CTAs for each (sequence, head) finds the weight of the last
// token taken, by a radix descent of 8 bits a pass over order-preserving integer keys (each CTA
// counts its share of the tokens; the counts are added through distributed shared memory), then
// compacts the kept positions: ballots inside a warp, a scan over warps, and the lower CTAs'
// totals.  On 32 heads of 32768 tokens: 2048 bins in three passes 67 us, 256 in four 49, both in CTAs
// of 1024 threads, which fit a multiprocessor once and so started in turns; 21 in CTAs of 512, 19
// stopping at a bin that is taken whole.  move: as the append kernel, 128 destination positions a
// CTA and 16 a warp, values in registers between the block's maximum and the conversion, magnitudes
// compared as code bytes and codes rescaled as fp16 pairs (17 us for 256 heads of 1024 tokens, d =
// 64; by float32 values, a CTA for K and one for V, 32).  The move is memory-bound
// (each kept row is read and written once).  Measured: 32 heads of up to 32768 tokens to 4096, d =
// 128, 34 us (select 19, by the latency of its cluster barriers); 256 heads of up to 1280 to 1024,
// d = 64, 24 us (select 7).
#include <cooperative_groups.h>

#include "kv8_common.cuh"

namespace ea {
namespace kv8 {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 512;  // two CTAs and more fit a multiprocessor, so clusters start at once
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 256;
constexpr int kPasses = 4;
constexpr int kMostRanks = 8;  // CTAs of a cluster (the portable size)
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

// Exclusive sum of v over the CTA's threads.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* red) {
  const int lane = lane_id(), warp = warp_id();
  uint32_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) red[warp] = x;
  __syncthreads();
  const uint32_t w = lane < warp ? red[lane] : 0u;  // at most 32 warps
  return x - v + __reduce_add_sync(0xFFFFFFFFu, w);
}

struct SelectSmem {
  uint32_t hist[kPasses][kBins];
  uint32_t red[kPasses][kSelWarps];
  uint32_t digit[kPasses], left[kPasses];
  bool whole[kPasses];
  uint32_t above[kSelWarps], equal[kSelWarps];
  uint32_t total[2];
};

__global__ void __launch_bounds__(kSelThreads, 2) evict_select_kernel(EvictParams p) {
  __shared__ SelectSmem sm;
  const cg::cluster_group cluster = cg::this_cluster();
  const int ranks = cluster.num_blocks(), rank = cluster.block_rank();
  const int bh = blockIdx.x / ranks, b = bh / p.Hk, tid = threadIdx.x;
  const int lane = lane_id(), warp = warp_id();
  auto sync_cluster = [&] {
    if (ranks > 1)
      cluster.sync();
    else
      __syncthreads();
  };
  grid_launch_dependents();
  if (bh % p.Hk == 0 && rank == 0 && tid == 0) check_seq(p.lengths, nullptr, b, p.cap, 0, p.status);
  const int len = seq_len(p.lengths, b, p.cap);
  int32_t* kept = p.kept + static_cast<int64_t>(bh) * p.keep;
  const float* w = p.weights + static_cast<int64_t>(bh) * p.cap;
  if (len <= p.keep) {
    for (int i = rank * kSelThreads + tid; i < p.keep; i += ranks * kSelThreads) kept[i] = i < len ? i : -1;
    return;
  }
  // This CTA's share of the tokens, and of the middle ones that compete.
  const int share = (len + ranks - 1) / ranks;
  const int i0 = min(rank * share, len), i1 = min(i0 + share, len);
  const int lo = max(i0, p.sink), hi = min(i1, len - p.recent);
  const uint32_t want = p.keep - p.sink - p.recent;  // below the middle's size
  for (int i = tid; i < kPasses * kBins; i += kSelThreads) (&sm.hist[0][0])[i] = 0;
  __syncthreads();
  uint32_t prefix = 0, left = want;
  int low = 0;  // bits of a key that were not needed
#pragma unroll 1  // rolled: what a pass costs is the latency of its steps, instruction fetches among them
  for (int pass = 0; pass < kPasses; ++pass) {
    const int shift = 24 - 8 * pass;
    uint32_t* hist = sm.hist[pass];
#pragma unroll 4
    for (int i = lo + tid; i < hi; i += kSelThreads) {
      const uint32_t k = order_key(__ldg(w + i));
      if (pass == 0 || ((k ^ prefix) >> (shift + 8)) == 0) atomicAdd(&hist[(k >> shift) & 255u], 1u);
    }
    sync_cluster();
    // kPer threads to a bin, from the top bin down: its count over the whole cluster.
    constexpr int kPer = kSelThreads / kBins;
    const int bin = kBins - 1 - tid / kPer;
    uint32_t h = 0;
#pragma unroll
    for (int i = 0; i < kMostRanks / kPer; ++i) {  // loads from other CTAs take long: all at once
      const int r = i * kPer + tid % kPer;
      if (r < ranks) h += cluster.map_shared_rank(hist, r)[bin];
    }
#pragma unroll
    for (int o = 1; o < kPer; o <<= 1) h += __shfl_xor_sync(0xFFFFFFFFu, h, o);
    const uint32_t ex = block_scan(tid % kPer == 0 ? h : 0u, sm.red[pass]);
    if (tid % kPer == 0 && ex < left && left <= ex + h) {
      sm.digit[pass] = bin;
      sm.left[pass] = left - ex;
      sm.whole[pass] = left == ex + h;
    }
    __syncthreads();
    if (want > 0) {
      prefix |= sm.digit[pass] << shift;
      left = sm.left[pass];
    }
    // The whole of the last bin is taken: its keys need no telling apart.
    if (want > 0 && sm.whole[pass]) {
      low = shift;
      break;
    }
  }
  // Keys above `prefix` are kept, and the first `left` of those equal to it.  A warp takes
  // consecutive tokens of the CTA's share, 32 at a time.
  const int per_warp = ((i1 - i0 + kSelWarps - 1) / kSelWarps + 31) / 32 * 32;
  const int w0 = min(i0 + warp * per_warp, i1), w1 = min(w0 + per_warp, i1);
  auto judge = [&](int i, bool& above, bool& equal) {
    above = equal = false;
    if (i >= w1) return;
    if (i < p.sink || i >= len - p.recent) {
      above = true;
    } else if (want > 0) {
      const uint32_t k = order_key(__ldg(w + i)) >> low;
      above = k > prefix >> low;
      equal = k == prefix >> low;
    }
  };
  uint32_t na = 0, ne = 0;
#pragma unroll 4
  for (int i = w0; i < w1; i += 32) {
    bool above, equal;
    judge(i + lane, above, equal);
    na += __popc(__ballot_sync(0xFFFFFFFFu, above));
    ne += __popc(__ballot_sync(0xFFFFFFFFu, equal));
  }
  if (lane == 0) sm.above[warp] = na, sm.equal[warp] = ne;
  __syncthreads();
  uint32_t xa = lane < kSelWarps ? sm.above[lane] : 0u, xe = lane < kSelWarps ? sm.equal[lane] : 0u;
  uint32_t ab = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? xa : 0u);
  uint32_t eq = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? xe : 0u);
  if (warp == 0) {
    xa = __reduce_add_sync(0xFFFFFFFFu, xa);
    xe = __reduce_add_sync(0xFFFFFFFFu, xe);
    if (lane == 0) sm.total[0] = xa, sm.total[1] = xe;
  }
  sync_cluster();
  {
    uint32_t la = 0, le = 0;
    if (lane < rank) {
      const uint32_t* t = cluster.map_shared_rank(sm.total, lane);
      la = t[0];
      le = t[1];
    }
    ab += __reduce_add_sync(0xFFFFFFFFu, la);
    eq += __reduce_add_sync(0xFFFFFFFFu, le);
  }
#pragma unroll 2
  for (int i = w0; i < w1; i += 32) {
    bool above, equal;
    judge(i + lane, above, equal);
    const uint32_t ba = __ballot_sync(0xFFFFFFFFu, above), be = __ballot_sync(0xFFFFFFFFu, equal);
    const uint32_t below = (1u << lane) - 1u;
    const uint32_t ma = ab + __popc(ba & below), me = eq + __popc(be & below);
    if (above || (equal && me < left)) kept[ma + min(me, left)] = i + lane;
    ab += __popc(ba);
    eq += __popc(be);
  }
  if (ranks > 1) cluster.sync();  // no CTA leaves while its counts may be read
}

// Codes times scale / s as codes again: the general rule, for any scales.
__device__ __forceinline__ uint32_t requantize4(uint32_t w, float scale, float inv) {
  float x[4];
  codes_to_float4(w, x);
  return pack_codes(x[0] * scale * inv, x[1] * scale * inv, x[2] * scale * inv, x[3] * scale * inv);
}
// The same where scale / s is a power of two 2^-14 .. 2^15, given as two fp16 values: the product
// is exact in fp16 wherever its E4M3 value is not zero, and rounds once.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, uint32_t ratio2) {
  uint32_t out = 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t c = h ? hi_codes(w) : lo_codes(w);
    const __half2 y = __hmul2(*reinterpret_cast<const __half2*>(&c), *reinterpret_cast<const __half2*>(&ratio2));
    uint16_t e;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(e) : "r"(*reinterpret_cast<const uint32_t*>(&y)));
    out |= static_cast<uint32_t>(e) << (16 * h);
  }
  return out;
}

template <int D>
__global__ void __launch_bounds__(kMoveThreads, D == 64 ? 6 : 4) evict_move_kernel(EvictParams p) {
  constexpr int kLanes = D / 16;           // lanes of one row (16 codes each)
  constexpr int kRowsIt = 32 / kLanes;
  constexpr int kIters = 16 / kRowsIt;
  __shared__ float red[2][kMoveThreads / 32];
  const int lane = lane_id(), warp = warp_id();
  const int bh = blockIdx.y, b = bh / p.Hk;
  const int live = min(seq_len(p.lengths, b, p.cap), p.keep);
  grid_dependency_wait();
  if (blockIdx.x == 0 && bh % p.Hk == 0 && threadIdx.x == 0) p.lengths_out[b] = live;
  const int s0 = blockIdx.x * 128;
  if (s0 >= live) return;
  const int p0 = s0 + 16 * warp;
  const int wpb = p.block / 16;
  const int start = s0 + warp / wpb * p.block;
  const int sub = lane / kLanes, col = lane % kLanes * 16;
  const int32_t* kept = p.kept + static_cast<int64_t>(bh) * p.keep;
  const int shift = 31 - __clz(p.block);

  uint4 raw[2][kIters];
  float sc[2][kIters];
  {
    // Kept inside the cache even if the lengths changed since the first kernel read them.
    const int from16 = p0 + (lane & 15) < live ? min(kept[p0 + (lane & 15)], p.cap - 1) : -1;
    if (lane < 16 && from16 >= 0)
      p.weights_out[static_cast<int64_t>(bh) * p.cap_out + p0 + lane] =
          __ldg(p.weights + static_cast<int64_t>(bh) * p.cap + from16);
#pragma unroll
    for (int it = 0; it < kIters; ++it) {
      const int from = __shfl_sync(0xFFFFFFFFu, from16, it * kRowsIt + sub);
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        raw[side][it] = make_uint4(0, 0, 0, 0);
        sc[side][it] = 0.0f;
        if (from >= 0) {
          const uint8_t* src = p.codes[side] + (static_cast<int64_t>(bh) * p.cap + from) * D + col;
          raw[side][it] = __ldg(reinterpret_cast<const uint4*>(src));
          sc[side][it] = __ldg(p.scales[side] + static_cast<int64_t>(bh) * (p.cap >> shift) + (from >> shift));
        }
      }
    }
  }
  float amax[2] = {0.0f, 0.0f};
#pragma unroll
  for (int side = 0; side < 2; ++side)
#pragma unroll
    for (int it = 0; it < kIters; ++it) {
      // Magnitudes are ordered as their 7-bit codes, so the row piece's largest is found on bytes
      // (0x7F, NaN, is looked at by value).
      const uint4 u = raw[side][it];
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) m = __vmaxu2(m, __vmaxu2(w[i] & 0x7F007F00u, (w[i] & 0x007F007Fu) << 8));
      m = max(m >> 24, (m >> 8) & 0xFFu);
      if (m == 0x7Fu) {
#pragma unroll 1
        for (int i = 0; i < 4; ++i) {
          float x[4];
          codes_to_float4(i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w, x);
          for (int e = 0; e < 4; ++e) amax[side] = fmaxf(amax[side], finite_abs(x[e] * sc[side][it]));
        }
      } else {
        const uint32_t h = e4m3x2_to_f16x2(static_cast<uint16_t>(m));
        amax[side] = fmaxf(amax[side], finite_abs(__half2float(__ushort_as_half(h & 0xFFFFu)) * sc[side][it]));
      }
    }
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    amax[side] = warp_max(amax[side]);
    if (lane == 0) red[side][warp] = amax[side];
  }
  __syncthreads();
  if (start >= live) return;
  const int w0 = warp / wpb * wpb;
#pragma unroll
  for (int side = 0; side < 2; ++side) {
    float a = amax[side];
    for (int w = w0; w < w0 + wpb; ++w) a = fmaxf(a, red[side][w]);
    const int e = scale_exp(a);
    const float s = pow2(e), inv = pow2(-e);
    if (warp == w0 && lane == 0)
      p.scales_out[side][static_cast<int64_t>(bh) * (p.cap_out >> shift) + (start >> shift)] = s;
    uint8_t* dst = p.codes_out[side] + static_cast<int64_t>(bh) * p.cap_out * D;
#pragma unroll
    for (int it = 0; it < kIters; ++it) {
      const int pos = p0 + it * kRowsIt + sub;
      const float scale = sc[side][it];
      // Both scales powers of two (mantissa zero) and their ratio within fp16: rescale4.  Scales
      // past 2^118, whose values may pass float32's range, go by value.
      const uint32_t su = __float_as_uint(scale);
      const int k = static_cast<int>(su >> 23) - 127 - e;
      const bool quick = (su & 0x7FFFFFu) == 0 && su < (245u << 23) && k >= -14 && k <= 15;
      uint4 u = raw[side][it];
      if (pos >= live) continue;
      if (quick) {
        if (k != 0) {
          const uint32_t h = static_cast<uint32_t>(k + 15) << 10;  // 2^k
          const uint32_t ratio2 = h | (h << 16);
          u = make_uint4(rescale4(u.x, ratio2), rescale4(u.y, ratio2), rescale4(u.z, ratio2),
                         rescale4(u.w, ratio2));
        }
      } else {
        u = make_uint4(requantize4(u.x, scale, inv), requantize4(u.y, scale, inv),
                       requantize4(u.z, scale, inv), requantize4(u.w, scale, inv));
      }
      *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(pos) * D + col) = u;
    }
  }
}

}  // namespace kv8

int launch_kv8_evict(const Kv8EvictArgs& a, cudaStream_t s, std::string& err) {
  kv8::EvictParams p{a.Hk, a.d, a.cap, a.block, a.keep, a.sink, a.recent, a.cap_out,
                     {a.k8, a.v8}, {a.k_scales, a.v_scales}, a.weights, a.lengths,
                     {a.k8_out, a.v8_out}, {a.k_scales_out, a.v_scales_out}, a.weights_out,
                     a.lengths_out, a.kept, a.status};
  void* args[] = {&p};
  // CTAs of a head's cluster: doubled (to the portable 8) while a CTA has more than 4096 tokens
  // to look at and the clusters leave multiprocessors idle.
  const int heads = a.B * a.Hk;
  int ranks = 1;
  while (ranks < kv8::kMostRanks && a.cap > 4096 * ranks && heads * ranks * 2 <= 2 * a.sms) ranks *= 2;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {static_cast<unsigned>(ranks), 1, 1};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(heads * ranks));
  cfg.blockDim = dim3(kv8::kSelThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(kv8::evict_select_kernel), args);
  if (e == cudaSuccess) {
    const int most = a.keep < a.cap ? a.keep : a.cap;
    const dim3 grid(static_cast<unsigned>((most + 127) / 128), static_cast<unsigned>(heads));
    auto* kernel = a.d == 128 ? kv8::evict_move_kernel<128> : kv8::evict_move_kernel<64>;
    e = kv8::launch_after(reinterpret_cast<const void*>(kernel), grid, dim3(kv8::kMoveThreads), args, s);
  }
  if (e != cudaSuccess) {
    err = std::string("kv8 evict launch: ") + cudaGetErrorString(e);
    return -5;
  }
  return 0;
}

}  // namespace ea
