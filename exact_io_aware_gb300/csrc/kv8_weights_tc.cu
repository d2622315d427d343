// Accumulated attention weight of each cached key from many query rows, on the tcgen05 tensor
// cores (the mathematics: kv8_weights.cu).
//
// S^T = K Q^T with keys as the 128 rows of the accumulator: the A operand is a tile of codes as TMA
// brings it, the B operands are the queries' 8-bit terms (kv8_tc.cuh), so one thread holds all of a
// key's scores and sums its weight without a word to another.  The codes are read once for up to
// 256 rows; more rows pass in groups of 256.
//
// Warps: 0 issues the products, 1 loads K tiles, the others take the blocks of 128 keys in turn,
// four warps a block with an accumulator of their own: with two such groups instead of four the
// latencies of a block (tensor memory, exponentials) lay bare, 40 us against 32 on 128 rows,
// 8 heads of 65001 keys.
#include "kv8_tc.cuh"
#include "kv8_weights.cuh"

namespace ea {
namespace kv8 {
namespace wtc {

using tc::kRows;
constexpr int kTeams = 4;       // groups of four warps that take blocks of keys in turn
constexpr int kThreads = 128 * (1 + kTeams);
constexpr int kStages = 4;      // of K tiles
constexpr int kMostRows = 256;  // held at once
constexpr int kCols = 16;       // rows that are looked at for masks together

struct Shared {
  uint64_t q_full, q_free;
  uint64_t k_full[kStages], k_empty[kStages];
  uint64_t s_full[kTeams], s_empty[kTeams];
  uint32_t tmem_base;
  // read four rows at a time
  alignas(16) float row_mul[kMostRows];  // factor of the row's scores
  alignas(16) float neg_lse[kMostRows];  // -log2(e) LSE; -inf: counts for nothing
  int lim[kMostRows];          // keys the row sees
  int least[kMostRows / kCols];
};

template <bool kBf16, int D>
struct Config {
  using T8 = typename tc::Config<kBf16, D>::T8;
  static constexpr int kTerms = tc::Config<kBf16, D>::kTerms;
  static constexpr int kOffK = 2 * kTerms * T8::kBytes;
  static constexpr int kOffShared = kOffK + kStages * T8::kBytes;
  static_assert(kOffShared % alignof(Shared) == 0, "the shared block is misaligned");
};

template <bool kBf16, int D>
__global__ void __launch_bounds__(kThreads, 1)
    weights_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const WeightsParams<ByHead> p) {
  using C = Config<kBf16, D>;
  using T8 = typename C::T8;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem;
  uint8_t* sK = smem + C::kOffK;
  Shared& sh = *reinterpret_cast<Shared*>(smem + C::kOffShared);
  const int warp = warp_id(), lane = lane_id(), group = warp >> 2;
  const ByHead& geo = p.geo;
  if ((smem_u32(smem) & 1023u) != 0) {  // the swizzled tiles need it
    if (threadIdx.x == 0) raise_timeout(p.status, 0x20);
    return;
  }
  int u0, u1;
  Place pl = plan_run(geo, blockIdx.x, gridDim.x, 2, u0, u1);
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < geo.B; b += kThreads)
      check_seq(geo.lengths, geo.counts, b, geo.cap, geo.n, p.status);
  if (u0 >= u1) return;
  if (threadIdx.x == 0) {
    mbar_init(&sh.q_full, 4 * kTeams);
    mbar_init(&sh.q_free, 1 + 4 * kTeams);  // the products, and the warps that read the rows
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sh.k_full[s], 1);
      mbar_init(&sh.k_empty[s], 1);
    }
    for (int w = 0; w < kTeams; ++w) {
      mbar_init(&sh.s_full[w], 1);
      mbar_init(&sh.s_empty[w], 4);
    }
    fence_barrier_init();
  }
  constexpr uint32_t kTmem = 128 * kTeams;
  if (warp == 0) tmem_alloc(&sh.tmem_base, kTmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;  // team w's accumulator at 128 w

  // Every role walks the same tiles, and in each the same groups of rows and blocks of keys.
  const int block_shift = 31 - __clz(p.block);
  bool ok = true;
  uint32_t c = 0, part = 0;        // blocks and groups of rows so far
  uint32_t use[kTeams] = {};       // uses of each accumulator so far
  for (;;) {
    const int blocks = chunks_of(geo, pl.keys);
    const int j0 = max(u0 - pl.start, 0);
    const int j1 = min(u1 - pl.start, blocks);
    const int len = seq_len(geo.lengths, pl.b, geo.cap), cnt = seq_count(geo.counts, pl.b, geo.n);
    const int64_t bh = static_cast<int64_t>(pl.b) * geo.Hk + pl.hk;
    for (int r0 = 0; r0 < geo.R && ok; r0 += kMostRows, ++part) {
      const int rows = min(kMostRows, geo.R - r0), tiles = rows > kRows ? 2 : 1;
      if (warp == 0) {
        // ------------------------------------------------------------ products
        constexpr uint32_t id_s = idesc_e4m3(128, kRows), id_rest = id_s | tc::kE5m2InB;
        const uint64_t dq = T8::desc_k(smem_u32(sQ), 0), dk0 = T8::desc_k(smem_u32(sK), 0);
        ok = mbar_wait_warp(&sh.q_full, part & 1, p.status, 0x32);
        for (int j = j0; j < j1 && ok; ++j) {
          const uint32_t b = c + (j - j0), s = b % kStages, w = j % kTeams;
          ok = mbar_wait_warp(&sh.k_full[s], (b / kStages) & 1, p.status, 0x33);
          for (int rt = 0; rt < tiles && ok; ++rt) {
            ok = mbar_wait_warp(&sh.s_empty[w], (use[w] & 1) ^ 1, p.status, 0x34);
            if (!ok) break;
            ++use[w];
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int term = 0; term < C::kTerms; ++term)
#pragma unroll
                for (int kk = 0; kk < D / 32; ++kk)
                  mma_ss_f8(tmem + 128 * w,
                            dk0 + s * static_cast<uint64_t>(T8::kBytes >> 4) + T8::k_step(kk),
                            dq + (rt * C::kTerms + term) * static_cast<uint64_t>(T8::kBytes >> 4) + T8::k_step(kk),
                            term > 0 ? id_rest : id_s, (term > 0 || kk > 0) ? 1u : 0u);
              mma_commit(&sh.s_full[w]);
              if (rt + 1 == tiles) {
                mma_commit(&sh.k_empty[s]);
                if (j + 1 == j1) mma_commit(&sh.q_free);
              }
            }
            __syncwarp();
          }
        }
      } else if (warp == 1) {
        // ------------------------------------------------------------ K tiles
        for (int j = j0; j < j1 && ok; ++j) {
          const uint32_t b = c + (j - j0), s = b % kStages;
          ok = mbar_wait_warp(&sh.k_empty[s], ((b / kStages) & 1) ^ 1, p.status, 0x35);
          if (ok && lane == 0) {
            mbar_arrive_expect_tx(&sh.k_full[s], T8::kBytes);
            tma_load_3d(sK + s * T8::kBytes, &tm_k, &sh.k_full[s], 0, j * kBlockKeys, static_cast<int>(bh));
          }
          __syncwarp();
        }
      } else if (group >= 1) {
        // ------------------------------------------------------------ exponentials and sums
        const int w = group - 1, key_lane = (warp & 3) * 32 + lane, tid = w * 128 + key_lane;
        const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
        if (part > 0) ok = mbar_wait_warp(&sh.q_free, (part - 1) & 1, p.status, 0x36);
        if (!ok) break;
        tc::put_queries<kBf16, D, 128 * kTeams, 0>(sQ, sh.row_mul, tc::Rows<D>{p.q + geo.row_offset(pl.b, pl.hk, r0) * D}, rows, tiles * kRows,
                                  p.c2, tid);
        if (tid < kMostRows) {
          const int r = r0 + tid;
          const bool real = r < geo.R && geo.query(r) < cnt;
          const float lse = real ? __ldg(p.lse + geo.row_offset(pl.b, pl.hk, r)) : -INFINITY;
          sh.neg_lse[tid] = lse != -INFINITY ? -lse * kLog2e : -INFINITY;
          const int lim = lse != -INFINITY ? query_keys(geo, len, cnt, geo.query(r)) : 0;
          sh.lim[tid] = lim;
          int least = lim;
#pragma unroll
          for (int o = 1; o < kCols; o <<= 1) least = min(least, __shfl_xor_sync(0xFFFFFFFFu, least, o));
          if (lane % kCols == 0) sh.least[tid / kCols] = least;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.q_full);
        ok = mbar_wait_warp(&sh.q_full, part & 1, p.status, 0x38);
        const float* w_in = r0 ? p.w_out : p.w_in;  // later passes add to the first's
        // A key's scale and sum so far are fetched a block ahead.
        float next_kf = 0.0f, next_before = 0.0f;
        auto fetch = [&](int j) {
          const int key = j * kBlockKeys + key_lane;
          const bool in = j < j1 && key < len;
          next_kf = in ? __ldg(p.k_scales + bh * (geo.cap >> block_shift) + (key >> block_shift)) : 0.0f;
          next_before = in && w_in ? w_in[bh * geo.cap + key] : 0.0f;
        };
        int j = j0 + (w + kTeams - j0 % kTeams) % kTeams;
        fetch(j);
        for (; j < j1 && ok; j += kTeams) {
          const int key0 = j * kBlockKeys, key = key0 + key_lane;
          const bool held = key < len;
          const float kf = next_kf, before = next_before;
          fetch(j + kTeams);
          float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
          for (int rt = 0; rt < tiles; ++rt) {
            ok = mbar_wait_warp(&sh.s_full[w], use[w] & 1, p.status, 0x37);
            if (!ok) break;
            ++use[w];
            tc_fence_after();
            const uint32_t tS = tmem + 128 * w + lane_off;
            const int groups = (min(kRows, rows - rt * kRows) + kCols - 1) / kCols;
            for (int g0 = 0; g0 < groups; g0 += 2) {
              uint32_t s[32];
              tmem_ld32(tS + g0 * kCols, s);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int col = rt * kRows + (g0 + i) * kCols;
                const uint32_t* x = s + i * kCols;
                if (i == 1 && g0 + 1 == groups) break;
                if (key0 + kBlockKeys <= sh.least[col / kCols]) {
                  const float2 kf2 = make_float2(kf, kf), zero = make_float2(0.0f, 0.0f);
#pragma unroll
                  for (int k = 0; k < kCols; k += 4) {
                    const float4 f = *reinterpret_cast<const float4*>(&sh.row_mul[col + k]);
                    const float4 b = *reinterpret_cast<const float4*>(&sh.neg_lse[col + k]);
                    float2 u = make_float2(__uint_as_float(x[k]), __uint_as_float(x[k + 1]));
                    float2 v = make_float2(__uint_as_float(x[k + 2]), __uint_as_float(x[k + 3]));
                    u = tc::fma2(tc::fma2(u, kf2, zero), make_float2(f.x, f.y), make_float2(b.x, b.y));
                    v = tc::fma2(tc::fma2(v, kf2, zero), make_float2(f.z, f.w), make_float2(b.z, b.w));
                    sum[0] = tc::add2(sum[0], make_float2(ex2(u.x), ex2(u.y)));
                    sum[1] = tc::add2(sum[1], make_float2(ex2(v.x), ex2(v.y)));
                  }
                } else {  // some row does not see all of the block, or counts for nothing
#pragma unroll
                  for (int k = 0; k < kCols; ++k) {
                    const float e = ex2(fmaf(__uint_as_float(x[k]) * kf, sh.row_mul[col + k], sh.neg_lse[col + k]));
                    sum[k & 1].x += key < sh.lim[col + k] ? e : 0.0f;
                  }
                }
              }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.s_empty[w]);
          }
          if (ok && held) p.w_out[bh * geo.cap + key] = before + ((sum[0].x + sum[0].y) + (sum[1].x + sum[1].y));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.q_free);
      }
      c += j1 - j0;
    }
    if (!ok || pl.start + blocks >= u1) break;
    next_place(geo, pl);
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmem);
  }
}

}  // namespace wtc
}  // namespace kv8

template <bool kBf16, int D>
cudaError_t launch_kv8_weights_tc(kv8::WeightsParams<kv8::ByHead> p, int sms, cudaStream_t s) {
  using C = kv8::wtc::Config<kBf16, D>;
  auto* kernel = kv8::wtc::weights_tc_kernel<kBf16, D>;
  constexpr size_t smem = C::kOffShared + sizeof(kv8::wtc::Shared);
  static_assert(smem <= 227 * 1024, "shared memory overflow");
  CUtensorMap tm_k;
  if (!encode_byte_map(&tm_k, p.k8, static_cast<uint64_t>(p.geo.B) * p.geo.Hk, p.geo.cap, D, kv8::kBlockKeys, D))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> allowed{0};
  const cudaError_t e = kv8::allow_smem(reinterpret_cast<const void*>(kernel), smem, allowed);
  if (e != cudaSuccess) return e;
  void* args[] = {&tm_k, &p};
  return cudaLaunchKernel(reinterpret_cast<const void*>(kernel), dim3(sms), dim3(kv8::wtc::kThreads), args, smem, s);
}

template cudaError_t launch_kv8_weights_tc<true, 64>(kv8::WeightsParams<kv8::ByHead>, int, cudaStream_t);
template cudaError_t launch_kv8_weights_tc<true, 128>(kv8::WeightsParams<kv8::ByHead>, int, cudaStream_t);
template cudaError_t launch_kv8_weights_tc<false, 64>(kv8::WeightsParams<kv8::ByHead>, int, cudaStream_t);
template cudaError_t launch_kv8_weights_tc<false, 128>(kv8::WeightsParams<kv8::ByHead>, int, cudaStream_t);

}  // namespace ea
