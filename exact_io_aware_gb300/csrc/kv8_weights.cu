// Accumulated attention weight of each cached key:
//     w_j += sum over the query rows r of the key/value head of e^{s_rj - LSE_r},
// with the LSE of the attention call on the same queries.  The sum runs over a key's rows in a
// fixed order, so the result does not depend on the launch.
//
// This file: the kernel for few rows, which is bound by reading the codes, and the choice between
// it and the tcgen05 kernel for many (kv8_weights_tc.cu).  Scores are formed as in kv8_attend_few.cuh
// (S^T = K Q^T, a warp to 32 keys), the queries stay in registers, and a key's weight is summed
// over the rows of a lane and then over the four lanes that share the key.  Measured (d = 128, four
// rows): 256 heads of 2000 to 8192 keys, 36.2 us, 4.9 TB/s, 73 % of the measured copy rate.
#include "kv8_mma.cuh"
#include "kv8_weights.cuh"

namespace ea {
namespace kv8 {

constexpr int kWeightsWarps = 4;
constexpr int kWeightsThreads = kWeightsWarps * 32;

template <int D>
constexpr int weights_stage_bytes() { return Chunk<D>::kBytes + 16 + 4 * kChunk; }  // K, scales, sums
template <int NT>
constexpr int weights_ctas_per_sm() { return NT == 1 ? 4 : 3; }
template <int D, int NT>
constexpr int weights_stages() {
  const int fit = (225 * 1024 / weights_ctas_per_sm<NT>() - 1024) / (kWeightsWarps * weights_stage_bytes<D>());
  return fit < 4 ? fit : 4;
}

template <bool kBf16, int D, int NT>
__global__ void __launch_bounds__(kWeightsThreads, weights_ctas_per_sm<NT>())
    weights_kernel(const WeightsParams<ByQuery> p) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int kStages = weights_stages<D, NT>();
  const int lane = lane_id(), warp = warp_id(), g = lane >> 2, t = lane & 3;
  const ByQuery& geo = p.geo;
  int u0, u1;
  Place pl = plan_run(geo, blockIdx.x, gridDim.x, kWeightsWarps, u0, u1);
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < geo.B; b += kWeightsThreads)
      check_seq(geo.lengths, geo.counts, b, geo.cap, geo.n, p.status);
  if (u0 >= u1) return;
  uint8_t* ring = smem + warp * (kStages * weights_stage_bytes<D>());
  const int nblk = geo.cap / p.block;

  for (;;) {
    const int tile_chunks = chunks_of(geo, pl.keys);
    const int c0 = max(u0 - pl.start, 0);
    const int c1 = min(u1 - pl.start, tile_chunks);
    const int len = seq_len(geo.lengths, pl.b, geo.cap), cnt = seq_count(geo.counts, pl.b, geo.n);
    const int64_t bh = static_cast<int64_t>(pl.b) * geo.Hk + pl.hk;
    const uint8_t* kp = p.k8 + bh * geo.cap * D;
    const float* ksp = p.k_scales + bh * nblk;

    auto issue = [&](int ch, int stage) {
      if (ch < c1) {
        const uint32_t s = smem_u32(ring + stage * weights_stage_bytes<D>());
        const int key0 = ch * kChunk;
        load_chunk<D>(s, kp, key0, len);
        if (lane < 2) {
          const int key = key0 + lane * 16;
          cp_async4(s + Chunk<D>::kBytes + lane * 4, ksp + (key < len ? key : key0) / p.block);
        }
        if (p.w_in && key0 + lane < len)
          cp_async4(s + Chunk<D>::kBytes + 16 + lane * 4, p.w_in + bh * geo.cap + key0 + lane);
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(c0 + warp + i * kWeightsWarps, i);

    QFrag<D> q[NT];
    float neg_lse[NT][2];  // -log2(e) LSE
    int lim[NT][2];        // keys the row sees; 0 for a row that counts for nothing
    int least = len;
    float kmul[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      {
        const int r = j * 8 + g;
        float x[D / 4];
        load_q_row<kBf16, D>(r < geo.R && geo.query(r) < cnt ? p.q + geo.row_offset(pl.b, pl.hk, r) * D : nullptr, x);
        pack_q<D>(x, p.c2, q[j], kmul[j]);
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = j * 8 + 2 * t + c;
        const bool real = r < geo.R && geo.query(r) < cnt;
        const float lse = real ? __ldg(p.lse + geo.row_offset(pl.b, pl.hk, r)) : -INFINITY;
        neg_lse[j][c] = lse != -INFINITY ? -lse * kLog2e : -INFINITY;
        lim[j][c] = lse != -INFINITY ? query_keys(geo, len, cnt, geo.query(r)) : 0;
        least = min(least, lim[j][c]);
      }
    }
    least = __reduce_min_sync(0xFFFFFFFFu, least);

    int stage = 0;
    for (int ch = c0 + warp; ch < c1; ch += kWeightsWarps) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      issue(ch + (kStages - 1) * kWeightsWarps, stage == 0 ? kStages - 1 : stage - 1);
      const int key0 = ch * kChunk;
      const uint8_t* st = ring + stage * weights_stage_bytes<D>();
      const float* sc = reinterpret_cast<const float*>(st + Chunk<D>::kBytes);
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        float acc[NT][4];
        scores16<D, NT>(st, mt, q, acc);
        const float ks = sc[mt];
        float sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const float kf[2] = {kmul[j][0] * ks, kmul[j][1] * ks};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float pr = ex2(fmaf(acc[j][e], kf[e & 1], neg_lse[j][e & 1]));
            if (key0 + kChunk > least) {
              const int key = key0 + mt * 16 + (e >> 1) * 8 + Chunk<D>::key_of_slot(g);
              if (key >= lim[j][e & 1]) pr = 0.0f;
            }
            sum[e >> 1] += pr;
          }
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float s = sum[e];
          s += __shfl_xor_sync(0xFFFFFFFFu, s, 1);
          s += __shfl_xor_sync(0xFFFFFFFFu, s, 2);
          const int at = mt * 16 + e * 8 + Chunk<D>::key_of_slot(g), key = key0 + at;
          if (t == 0 && key < len) p.w_out[bh * geo.cap + key] = (p.w_in ? sc[4 + at] : 0.0f) + s;
        }
      }
      __syncwarp();
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    cp_async_wait<0>();
    if (pl.start + tile_chunks >= u1) break;
    next_place(geo, pl);
  }
}

template <bool kBf16, int D, int NT>
cudaError_t launch_weights(WeightsParams<ByQuery> p, int sms, cudaStream_t s) {
  auto* kernel = weights_kernel<kBf16, D, NT>;
  constexpr int smem = kWeightsWarps * weights_stages<D, NT>() * weights_stage_bytes<D>();
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), smem, allowed);
  if (e != cudaSuccess) return e;
  void* args[] = {&p};
  return cudaLaunchKernel(reinterpret_cast<const void*>(kernel), dim3(weights_ctas_per_sm<NT>() * sms),
                          dim3(kWeightsThreads), args, smem, s);
}

template <bool kBf16, int D>
cudaError_t launch_weights_nt(const WeightsParams<ByQuery>& p, int sms, cudaStream_t s) {
  if (p.geo.R <= 8) return launch_weights<kBf16, D, 1>(p, sms, s);
  return launch_weights<kBf16, D, 2>(p, sms, s);
}

}  // namespace kv8

namespace {

// Rows per key/value head up to which this file's kernel is used, the tcgen05 kernel above.  us here
// and there, 16 sequences x 8 heads of 8187 keys, d = 128: bf16 16 rows 33 and 39, 24 rows 47 and 41; fp16
// 16 rows 33 and 47.  One sequence of 65001 keys, 16 rows: bf16 21 and 24, fp16 21 and 29.  d = 64: bf16
// 25 and 31, fp16 25 and 34.
constexpr int kFewRows = 16;

template <class Geo>
kv8::WeightsParams<Geo> weights_params(const Kv8Args& a) {
  kv8::WeightsParams<Geo> p{};
  const int R = a.G * a.n;
  // Every held key is on the work list, so that the sums of keys no row sees are carried over.
  static_cast<kv8::Geometry&>(p.geo) = {a.B, a.Hk, a.G,      a.n,       a.cap,    R,
                                        R,   1,    a.causal, a.lengths, a.counts, true};
  p.block = a.block;
  p.c2 = a.c * kv8::kLog2e;
  p.q = static_cast<const uint16_t*>(a.q);
  p.k8 = a.k8;
  p.k_scales = a.k_scales;
  p.lse = a.lse;
  p.w_in = a.weights;
  p.w_out = a.weights_out;
  p.status = a.status;
  return p;
}

}  // namespace

int launch_kv8_weights(const Kv8Args& a, cudaStream_t s, std::string& err) {
  if (kv8::list_too_long(a.B, a.Hk, 1, a.cap, kv8::kChunk)) {
    err = "B * H_kv * cap is too large for one call";
    return -2;
  }
  cudaError_t e;
  if (static_cast<int64_t>(a.G) * a.n > kFewRows) {
    const auto p = weights_params<kv8::ByHead>(a);
    if (a.bf16)
      e = a.d == 128 ? launch_kv8_weights_tc<true, 128>(p, a.sms, s) : launch_kv8_weights_tc<true, 64>(p, a.sms, s);
    else
      e = a.d == 128 ? launch_kv8_weights_tc<false, 128>(p, a.sms, s) : launch_kv8_weights_tc<false, 64>(p, a.sms, s);
  } else {
    const auto p = weights_params<kv8::ByQuery>(a);
    if (a.bf16)
      e = a.d == 128 ? kv8::launch_weights_nt<true, 128>(p, a.sms, s) : kv8::launch_weights_nt<true, 64>(p, a.sms, s);
    else
      e = a.d == 128 ? kv8::launch_weights_nt<false, 128>(p, a.sms, s) : kv8::launch_weights_nt<false, 64>(p, a.sms, s);
  }
  if (e != cudaSuccess) {
    err = std::string("kv8 weights launch: ") + cudaGetErrorString(e);
    return -5;
  }
  return 0;
}

}  // namespace ea
