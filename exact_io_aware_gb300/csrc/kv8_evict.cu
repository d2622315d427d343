// Eviction: the tokens that drew the most attention, moved into another cache.
//
// A sequence of len > keep tokens keeps its first `sink`, its last `recent`, and of the middle
// the keep - sink - recent of the largest accumulated weight (ties: the lower position; NaN
// counts as -inf).  The kept tokens keep their order.  Their dequantised values form the
// destination's blocks, each with the least power-of-two scale that holds them.
//
// Two launches.  select: a cluster of CTAs for each (sequence, head) finds the weight of the last
// token taken, by a radix descent of 11, 11 and 10 bits over order-preserving integer keys (each
// CTA counts its share of the tokens; the counts are added through distributed shared memory),
// then compacts the kept positions: ballots inside a warp, a scan over warps, and the lower
// CTAs' totals.  move: as the append kernel, 128 destination positions a CTA and 16 a warp,
// values in registers between the block's maximum and the conversion.  The move is memory-bound
// (each kept row is read and written once).
#include <cooperative_groups.h>

#include "kv8_common.cuh"

namespace ea {
namespace kv8 {

namespace cg = cooperative_groups;

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
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
  const uint32_t w = lane < warp ? red[lane] : 0u;
  return x - v + __reduce_add_sync(0xFFFFFFFFu, w);
}

struct SelectSmem {
  uint32_t hist[3][kBins];
  uint32_t red[3][kSelWarps];
  uint32_t digit[3], left[3];
  uint32_t above[kSelWarps], equal[kSelWarps];
  uint32_t total[2];
};

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(EvictParams p) {
  __shared__ SelectSmem sm;
  const cg::cluster_group cluster = cg::this_cluster();
  const int ranks = cluster.num_blocks(), rank = cluster.block_rank();
  const int bh = blockIdx.x / ranks, b = bh / p.Hk, tid = threadIdx.x;
  const int lane = lane_id(), warp = warp_id();
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
  for (int i = tid; i < 3 * kBins; i += kSelThreads) (&sm.hist[0][0])[i] = 0;
  __syncthreads();
  uint32_t prefix = 0, left = want;
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const uint32_t bins = pass == 2 ? 1024 : 2048;
    uint32_t* hist = sm.hist[pass];
#pragma unroll 4
    for (int i = lo + tid; i < hi; i += kSelThreads) {
      const uint32_t k = order_key(__ldg(w + i));
      if (pass == 0 || (k >> (pass == 1 ? 21 : 10)) == (prefix >> (pass == 1 ? 21 : 10)))
        atomicAdd(&hist[(k >> shift) & (bins - 1)], 1u);
    }
    cluster.sync();
    // Thread t: the counts of the t-th pair of bins from the top, over the whole cluster.
    uint32_t h0 = 0, h1 = 0;
    const uint32_t top = bins - 1 - 2 * tid;
    if (2 * tid < static_cast<int>(bins)) {
      for (int r = 0; r < ranks; ++r) {
        const uint32_t* rh = cluster.map_shared_rank(hist, r);
        h0 += rh[top];
        h1 += rh[top - 1];
      }
    }
    const uint32_t ex = block_scan(h0 + h1, sm.red[pass]);
    if (ex < left && left <= ex + h0 + h1) {
      const bool second = left > ex + h0;
      sm.digit[pass] = top - (second ? 1 : 0);
      sm.left[pass] = left - ex - (second ? h0 : 0);
    }
    __syncthreads();
    if (want > 0) {
      prefix |= sm.digit[pass] << shift;
      left = sm.left[pass];
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
      const uint32_t k = order_key(__ldg(w + i));
      above = k > prefix;
      equal = k == prefix;
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
  uint32_t xa = sm.above[lane], xe = sm.equal[lane];
  uint32_t ab = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? xa : 0u);
  uint32_t eq = __reduce_add_sync(0xFFFFFFFFu, lane < warp ? xe : 0u);
  if (warp == 0) {
    xa = __reduce_add_sync(0xFFFFFFFFu, xa);
    xe = __reduce_add_sync(0xFFFFFFFFu, xe);
    if (lane == 0) sm.total[0] = xa, sm.total[1] = xe;
  }
  cluster.sync();
  for (int r = 0; r < rank; ++r) {
    const uint32_t* t = cluster.map_shared_rank(sm.total, r);
    ab += t[0];
    eq += t[1];
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
  cluster.sync();  // no CTA leaves while its counts may be read
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
  grid_dependency_wait();
  if (blockIdx.x == 0 && side == 0 && bh % p.Hk == 0 && threadIdx.x == 0) p.lengths_out[b] = live;
  const int s0 = blockIdx.x * 128;
  if (s0 >= live) return;
  const int p0 = s0 + 16 * warp;
  const int wpb = p.block / 16;
  const int start = s0 + warp / wpb * p.block;
  const int sub = lane / kLanes, col = lane % kLanes * 16;
  const int32_t* kept = p.kept + static_cast<int64_t>(bh) * p.keep;
  const uint8_t* src = (side ? p.codes[1] : p.codes[0]) + static_cast<int64_t>(bh) * p.cap * D;
  const float* src_scale = (side ? p.scales[1] : p.scales[0]) + static_cast<int64_t>(bh) * (p.cap / p.block);

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
    (side ? p.scales_out[1] : p.scales_out[0])[static_cast<int64_t>(bh) * (p.cap_out / p.block) + start / p.block] = s;
  uint8_t* dst = (side ? p.codes_out[1] : p.codes_out[0]) + static_cast<int64_t>(bh) * p.cap_out * D;
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
  // CTAs of a head's cluster: doubled (to the portable 8) while a CTA has more than 4096 tokens
  // to look at and the clusters leave multiprocessors idle.
  const int heads = a.B * a.Hk;
  int ranks = 1;
  while (ranks < 8 && a.cap > 4096 * ranks && heads * ranks * 2 <= 2 * a.sms) ranks *= 2;
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
    const dim3 grid(static_cast<unsigned>((most + 127) / 128), static_cast<unsigned>(heads), 2);
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
