// Accumulated attention weight of each cached key:
//     w_j += sum over the query rows r of the key/value head of e^{s_rj - LSE_r},
// with the LSE of the attention call on the same queries.  The sum runs over a key's rows inside
// one warp, in a fixed order, so the result does not depend on the launch.
//
// The scores are formed as in the attention kernel (S^T = K Q^T, a warp to 32 keys), but here
// a chunk's keys stay in registers as the A operand while all rows pass, eight at a time, from
// shared memory: the codes are read and widened once for up to 128 rows.  For few rows the
// kernel is bound by reading the codes, for many by the exponentials and products.
#include "kv8_mma.cuh"

namespace ea {
namespace kv8 {

constexpr int kWeightsWarps = 4;
constexpr int kWeightsThreads = kWeightsWarps * 32;
constexpr int kWeightsStages = 4;
constexpr int kWeightsRows = 128;  // rows held in shared memory at once

struct WeightsParams {
  ByQuery geo;  // one tile of all rows
  int block;
  float c2;
  const uint16_t* q;
  const uint8_t* k8;
  const float* k_scales;
  const float* lse;
  const float* w_in;
  float* w_out;
  uint32_t* status;
};

template <int D>
constexpr int weights_stage_bytes() { return Chunk<D>::kBytes + 16 + 4 * kChunk; }  // K, scales, sums
template <int D>
constexpr int q_row_bytes() { return 2 * D + 16; }  // the pad keeps eight lanes' loads apart

template <int D>
struct WeightsSmem {
  uint8_t ring[kWeightsWarps * kWeightsStages * weights_stage_bytes<D>()];
  uint8_t q[kWeightsRows * q_row_bytes<D>()];
  float lse2[kWeightsRows];   // log2(e) LSE; +inf for a row that counts for nothing
  int lim[kWeightsRows];      // keys the row sees
  int least[kWeightsRows / 8];
  float red[kWeightsWarps];
};

template <bool kBf16, int D>
__global__ void __launch_bounds__(kWeightsThreads, 2) weights_kernel(const WeightsParams p) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  WeightsSmem<D>& sm = *reinterpret_cast<WeightsSmem<D>*>(smem_raw);
  const int lane = lane_id(), warp = warp_id(), g = lane >> 2, t = lane & 3;
  const ByQuery& geo = p.geo;
  int64_t u0, u1;
  Place pl = plan_run(geo, blockIdx.x, gridDim.x, 1, u0, u1);
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < geo.B; b += kWeightsThreads)
      check_seq(geo.lengths, geo.counts, b, geo.cap, geo.n, p.status);
  if (u0 >= u1) return;
  uint8_t* ring = sm.ring + warp * (kWeightsStages * weights_stage_bytes<D>());
  const int nblk = geo.cap / p.block;

  for (;;) {
    const int tile_chunks = chunks_of(geo, pl.keys);
    const int c0 = static_cast<int>(max(u0 - pl.start, static_cast<int64_t>(0)));
    const int c1 = static_cast<int>(min(u1 - pl.start, static_cast<int64_t>(tile_chunks)));
    const int len = seq_len(geo.lengths, pl.b, geo.cap), cnt = seq_count(geo.counts, pl.b, geo.n);
    const int64_t bh = static_cast<int64_t>(pl.b) * geo.Hk + pl.hk;
    const uint8_t* kp = p.k8 + bh * geo.cap * D;
    const float* ksp = p.k_scales + bh * nblk;

    for (int rbase = 0; rbase < geo.R; rbase += kWeightsRows) {
      const int rows = min(kWeightsRows, geo.R - rbase), blocks = (rows + 7) / 8;
      const float* w_in = rbase ? p.w_out : p.w_in;  // later passes add to the first's
      auto issue = [&](int ch, int stage) {
        if (ch < c1) {
          const uint32_t s = smem_u32(ring + stage * weights_stage_bytes<D>());
          const int key0 = ch * kChunk;
          load_chunk<D>(s, kp, key0, len);
          if (lane < 2) {
            const int key = key0 + lane * 16;
            cp_async4(s + Chunk<D>::kBytes + lane * 4, ksp + (key < len ? key : key0) / p.block);
          }
          if (w_in && key0 + lane < len)
            cp_async4(s + Chunk<D>::kBytes + 16 + lane * 4, w_in + bh * geo.cap + key0 + lane);
        }
        cp_async_commit();
      };
#pragma unroll
      for (int i = 0; i < kWeightsStages - 1; ++i) issue(c0 + warp + i * kWeightsWarps, i);

      __syncthreads();  // the rows of the pass before are read
      constexpr int kPer = D / 32;  // columns of a lane
      float amax = 0.0f, qmul = 1.0f;
      for (int pass = 0; pass < 2; ++pass) {
        for (int r = warp; r < blocks * 8; r += kWeightsWarps) {
          const bool real = r < rows && geo.query(rbase + r) < cnt;
          float x[kPer];
          int64_t off = 0;
#pragma unroll
          for (int e = 0; e < kPer; ++e) x[e] = 0.0f;
          if (real) {
            off = geo.row_offset(pl.b, pl.hk, rbase + r);
#pragma unroll
            for (int e = 0; e < kPer / 2; ++e) {
              const float2 f = unpack16<kBf16>(
                  __ldg(reinterpret_cast<const uint32_t*>(p.q + off * D + lane * kPer) + e));
              x[2 * e] = f.x;
              x[2 * e + 1] = f.y;
            }
          }
          if (pass == 0) {
#pragma unroll
            for (int e = 0; e < kPer; ++e) amax = fmaxf(amax, finite_abs(x[e]));
          } else {
            uint32_t* dst = reinterpret_cast<uint32_t*>(sm.q + r * q_row_bytes<D>()) + lane * (kPer / 2);
#pragma unroll
            for (int e = 0; e < kPer / 2; ++e) dst[e] = pack_f16(x[2 * e] * qmul, x[2 * e + 1] * qmul);
            if (lane == 0) {
              const float lse = real ? p.lse[off] : -INFINITY;
              const bool counts = lse != -INFINITY;
              sm.lse2[r] = counts ? lse * kLog2e : INFINITY;
              sm.lim[r] = real && counts ? query_keys(geo, len, cnt, geo.query(rbase + r)) : 0;
            }
          }
        }
        if (pass == 0) {
          amax = warp_max(amax);
          if (lane == 0) sm.red[warp] = amax;
          __syncthreads();
          for (int w = 0; w < kWeightsWarps; ++w) amax = fmaxf(amax, sm.red[w]);
          qmul = pow2(q_exp(amax));
        }
      }
      __syncthreads();
      if (threadIdx.x < blocks) {
        int least = sm.lim[threadIdx.x * 8];
        for (int i = 1; i < 8; ++i) least = min(least, sm.lim[threadIdx.x * 8 + i]);
        sm.least[threadIdx.x] = least;
      }
      __syncthreads();
      const float kmul = p.c2 / qmul;
      int stage = 0;
      for (int ch = c0 + warp; ch < c1; ch += kWeightsWarps) {
        cp_async_wait<kWeightsStages - 2>();
        __syncwarp();
        issue(ch + (kWeightsStages - 1) * kWeightsWarps, stage == 0 ? kWeightsStages - 1 : stage - 1);
        const int key0 = ch * kChunk;
        const uint8_t* st = ring + stage * weights_stage_bytes<D>();
        const float* sc = reinterpret_cast<const float*>(st + Chunk<D>::kBytes);
        uint32_t a[2][D / 16][4];
#pragma unroll
        for (int mt = 0; mt < 2; ++mt) {
          const int r0 = mt * 16 + Chunk<D>::key_of_slot(g);
#pragma unroll
          for (int h = 0; h < D / 64; ++h) {
            const uint4 u = *reinterpret_cast<const uint4*>(st + Chunk<D>::at(r0, h * 4 + t));
            const uint4 v = *reinterpret_cast<const uint4*>(st + Chunk<D>::at(r0 + 8, h * 4 + t));
            const uint32_t x[4] = {u.x, u.y, u.z, u.w}, y[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int s = 0; s < 4; ++s) {
              a[mt][h * 4 + s][0] = lo_codes(x[s]);
              a[mt][h * 4 + s][1] = lo_codes(y[s]);
              a[mt][h * 4 + s][2] = hi_codes(x[s]);
              a[mt][h * 4 + s][3] = hi_codes(y[s]);
            }
          }
        }
        const float kf[2] = {kmul * sc[0], kmul * sc[1]};
        float sum[2][2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
        for (int j = 0; j < blocks; ++j) {
          const uint8_t* qrow = sm.q + (j * 8 + g) * q_row_bytes<D>();
          float acc[2][4] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
          for (int h = 0; h < D / 64; ++h) {
            const uint4 u = *reinterpret_cast<const uint4*>(qrow + h * 128 + t * 32);
            const uint4 v = *reinterpret_cast<const uint4*>(qrow + h * 128 + t * 32 + 16);
            const uint32_t b[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
              for (int mt = 0; mt < 2; ++mt) {
                const uint32_t (&am)[4] = a[mt][h * 4 + s];
                mma_f16(acc[mt], am[0], am[1], am[2], am[3], b[2 * s], b[2 * s + 1]);
              }
          }
          const float2 ls = *reinterpret_cast<const float2*>(&sm.lse2[j * 8 + 2 * t]);
          float pr[2][4];
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              pr[mt][e] = ex2(fmaf(acc[mt][e], kf[mt], e & 1 ? -ls.y : -ls.x));
          if (key0 + kChunk > sm.least[j]) {
            const int2 lm = *reinterpret_cast<const int2*>(&sm.lim[j * 8 + 2 * t]);
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int key = key0 + mt * 16 + (e >> 1) * 8 + Chunk<D>::key_of_slot(g);
                if (key >= (e & 1 ? lm.y : lm.x)) pr[mt][e] = 0.0f;
              }
          }
#pragma unroll
          for (int mt = 0; mt < 2; ++mt) {
            sum[mt][0] += pr[mt][0] + pr[mt][1];
            sum[mt][1] += pr[mt][2] + pr[mt][3];
          }
        }
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float s = sum[mt][e];
            s += __shfl_xor_sync(0xFFFFFFFFu, s, 1);
            s += __shfl_xor_sync(0xFFFFFFFFu, s, 2);
            const int key = key0 + mt * 16 + e * 8 + Chunk<D>::key_of_slot(g);
            if (t == 0 && key < len)
              p.w_out[bh * geo.cap + key] = (w_in ? sc[4 + key - key0] : 0.0f) + s;
          }
        __syncwarp();
        stage = stage + 1 == kWeightsStages ? 0 : stage + 1;
      }
      cp_async_wait<0>();
    }
    if (pl.start + tile_chunks >= u1) break;
    next_place(geo, pl);
  }
}

template <bool kBf16, int D>
cudaError_t launch_weights(WeightsParams p, int sms, cudaStream_t s) {
  auto* kernel = weights_kernel<kBf16, D>;
  const cudaError_t attr = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(sizeof(WeightsSmem<D>)));
  if (attr != cudaSuccess) return attr;
  void* args[] = {&p};
  return cudaLaunchKernel(reinterpret_cast<const void*>(kernel), dim3(2 * sms), dim3(kWeightsThreads),
                          args, sizeof(WeightsSmem<D>), s);
}

}  // namespace kv8

int launch_kv8_weights(const Kv8Args& a, cudaStream_t s, std::string& err) {
  kv8::WeightsParams p{};
  const int R = a.G * a.n;
  // Every held key is on the work list, so that the sums of keys no row sees are carried over.
  p.geo = {{a.B, a.Hk, a.G, a.n, a.cap, R, R, 1, a.causal, a.lengths, a.counts, true}};
  p.block = a.block;
  p.c2 = a.c * kv8::kLog2e;
  p.q = static_cast<const uint16_t*>(a.q);
  p.k8 = a.k8;
  p.k_scales = a.k_scales;
  p.lse = a.lse;
  p.w_in = a.weights;
  p.w_out = a.weights_out;
  p.status = a.status;
  cudaError_t e;
  if (a.bf16)
    e = a.d == 128 ? kv8::launch_weights<true, 128>(p, a.sms, s) : kv8::launch_weights<true, 64>(p, a.sms, s);
  else
    e = a.d == 128 ? kv8::launch_weights<false, 128>(p, a.sms, s) : kv8::launch_weights<false, 64>(p, a.sms, s);
  if (e != cudaSuccess) {
    err = std::string("kv8 weights launch: ") + cudaGetErrorString(e);
    return -5;
  }
  return 0;
}

}  // namespace ea
