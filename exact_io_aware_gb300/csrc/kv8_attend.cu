// Attention of a few query rows over the 8-bit cache.
//
// Row r of a key/value head (query i of head g, r = i G + g) has the scores
//     s_rj = c ks_j (q_r . k_j)          (ks, vs: the scales of key j's block)
// and O_r = sum_j e^{s_rj - LSE_r} vs_j v_j.  In base 2, with x_rj = log2(e) s_rj + log2(vs_j),
// a shift m_r near the running maximum of x_r, and P_rj = 2^{x_rj - m_r}:
//     z_r = sum_j P_rj v_j,   l_r = sum_j P_rj / vs_j,   O_r = z_r / l_r,
//     LSE_r = ln 2 (m_r + log2 l_r),
// so a value block's scale costs one constant a block: P is what the product takes and z needs
// no second scaling (scales at the ends of their range: kv8_attend.cuh).  P enters that product as fp16 (half a step 2^-11, an eighth of the bf16
// output's; for fp16 outputs, whose own rounding that would equal, as a pair of fp16 values and
// two products, which for bf16 too would take 34.3 us instead of 33.4 on 256 heads of four rows and
// 48.7 instead of 44.8 on twelve); m_r is set so that the largest P is 2^6 and is raised only when a P would
// pass 2^14, which keeps P inside fp16 and weights down to 2^-20 of the largest at full precision
// (the sums z and l are float32).
//
// The work is every chunk of 32 keys of every (sequence, head, row tile); each CTA takes an equal
// run of that list, whatever the sequences' lengths, and its warps take the run's chunks in turn,
// each with its own z, l and m.  At the end of a tile the warps' states are merged; a tile that
// one CTA holds whole is written at once, and a CTA's part of a tile shared with others (at most
// one at each end of its run) goes to the workspace as (z, l, m), joined by a second kernel.
//
// Bound by reading the cache.  Measured (d = 128): 128 heads of 16384 keys, one row each, 88 us, 6.1
// TB/s, 91 % of the measured copy rate; 256 heads of 500 to 4096 keys, four rows each, 33 us, 61 %,
// where planning the run (1.7 us), the join (4 us) and the launches are not hidden.  CTAs of four
// warps, three to a multiprocessor, against one of eight: 33 and 61 us.
#include "kv8_attend.cuh"
#include "kv8_mma.cuh"

namespace ea {
namespace kv8 {

constexpr int kAttendWarps = 4;
constexpr int kAttendThreads = kAttendWarps * 32;
// A cache of at most this many tokens a sequence is not cut: each tile is one CTA's, and there is
// nothing to join.  us uncut and cut, at d = 64, G = 1 and d = 128, G = 8: 8 heads of 512 tokens 5.8, 7.4
// and 8.1, 8.8, of 1024 8.2, 7.9 and 11.6, 8.9; 256 heads of 512 tokens 6.9, 11.6 and 10.4, 15.9 (of 1024
// still 10.6, 14.9 and 16.4, 20.8: with many heads longer tiles fill the device, with few they do not).
constexpr int kAlignedCap = 512;
constexpr int kMostCtas = 3;  // of any variant, on a multiprocessor

// CTAs resident on a multiprocessor (registers and shared memory are sized for them): while one
// starts on a tile or merges its warps, the others stream.
template <int NT>
constexpr int attend_ctas_per_sm() { return NT == 1 ? 3 : 2; }
template <int D>
constexpr int stage_bytes() { return 2 * Chunk<D>::kBytes + 32; }  // K, V, four scales
template <int D, int NT>
constexpr int attend_stages() {
  const int fit = (225 * 1024 / attend_ctas_per_sm<NT>() - 1024) / (kAttendWarps * stage_bytes<D>());
  return fit < 5 ? fit : 5;
}
template <int D, int NT>
constexpr size_t ring_bytes() { return static_cast<size_t>(kAttendWarps) * attend_stages<D, NT>() * stage_bytes<D>(); }
// The warps' states at a tile's end, over the drained ring: z (rows padded apart), then l and m.
template <int D>
constexpr int merge_stride() { return D + 4; }
template <int D, int NT>
constexpr size_t merge_bytes() {
  return static_cast<size_t>(kAttendWarps) * NT * 8 * (merge_stride<D>() + 2) * sizeof(float);
}

// One chunk of 32 keys against the tile's rows.  kPair: P as a pair of fp16 values.
template <int D, int NT, bool kPair>
__device__ __forceinline__ void attend_chunk(const uint8_t* st, int key0, bool masked,
                                             const float (&kmul)[NT][2], const QFrag<D> (&q)[NT],
                                             const int (&lim)[NT][2], float (&z)[NT][D / 16][4],
                                             float (&l)[NT][2], float (&m)[NT][2], float& hi) {
  const int lane = lane_id(), g = lane >> 2, t = lane & 3;
  const float* sc = reinterpret_cast<const float*>(st + 2 * Chunk<D>::kBytes);
  float x[2][NT][4];
  float lvs[2] = {log2f(sc[2]), log2f(sc[3])}, inv_vs[2] = {kLiftFactor / sc[2], kLiftFactor / sc[3]};
  float rest[2] = {1.0f, 1.0f};  // factor of what the V product takes
  hi = fmaxf(hi, fmaxf(lvs[0], lvs[1]));
  const float floor = fmaxf(kLeastScale, hi - kScaleSpan);
  const bool small = fminf(lvs[0], lvs[1]) < floor;  // the same in every lane
  if (__builtin_expect(small, 0)) {
#pragma unroll
    for (int mt = 0; mt < 2; ++mt) {
      if (lvs[mt] >= floor) continue;
      rest[mt] = ex2(lvs[mt] - floor);
      inv_vs[mt] = ex2(kLift - floor);
      lvs[mt] = floor;
    }
  }
  float top = -INFINITY;  // largest excess of x over the allowed shift
#pragma unroll
  for (int mt = 0; mt < 2; ++mt) {
    scores16<D, NT>(st, mt, q, x[mt]);
    const float ks = sc[mt];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const float kf[2] = {kmul[j][0] * ks, kmul[j][1] * ks};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float y = fmaf(x[mt][j][e], kf[e & 1], lvs[mt]);
        if (masked) {
          const int key = key0 + mt * 16 + (e >> 1) * 8 + Chunk<D>::key_of_slot(g);
          if (key >= lim[j][e & 1]) y = -INFINITY;
        }
        x[mt][j][e] = y;
        top = fmaxf(top, y - m[j][e & 1]);
      }
    }
  }
  if (__any_sync(0xFFFFFFFFu, top > kRaise)) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float mx = fmaxf(fmaxf(x[0][j][c], x[0][j][c + 2]), fmaxf(x[1][j][c], x[1][j][c + 2]));
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
        const float mn = fmaxf(m[j][c], mx - kTop);
        const float half = ex2(0.5f * (m[j][c] - mn)), r = half * half;
        m[j][c] = mn;
        l[j][c] = l[j][c] * half * half;
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          z[j][i][c] *= r;
          z[j][i][c + 2] *= r;
        }
      }
  }
  const uint8_t* vbase = st + Chunk<D>::kBytes;
#pragma unroll
  for (int mt = 0; mt < 2; ++mt) {
    uint32_t b0[NT], b1[NT];
    uint32_t lo0[kPair ? NT : 1], lo1[kPair ? NT : 1];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      float pr[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        pr[e] = ex2(x[mt][j][e] - m[j][e & 1]);
        l[j][e & 1] = fmaf(pr[e], inv_vs[mt], l[j][e & 1]);
        if (small) pr[e] *= rest[mt];
      }
      const uint32_t h0 = pack_f16(pr[0], pr[1]), h1 = pack_f16(pr[2], pr[3]);
      b0[j] = transpose8x8(h0);
      b1[j] = transpose8x8(h1);
      if constexpr (kPair) {
        const float2 u = unpack16<false>(h0), v = unpack16<false>(h1);
        lo0[j] = transpose8x8(pack_f16(pr[0] - u.x, pr[1] - u.y));
        lo1[j] = transpose8x8(pack_f16(pr[2] - v.x, pr[3] - v.y));
      }
    }
    // V rows of the slots 2t, 2t + 1 (of the lower, then the upper eight keys).
    uint32_t v[4][D / 32];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = mt * 16 + (i >> 1) * 8 + Chunk<D>::key_of_slot(2 * t + (i & 1));
      if constexpr (D == 128) {
        const uint4 u = *reinterpret_cast<const uint4*>(vbase + Chunk<D>::at(row, g));
        v[i][0] = u.x, v[i][1] = u.y, v[i][2] = u.z, v[i][3] = u.w;
      } else {
        const uint2 u = *reinterpret_cast<const uint2*>(vbase + Chunk<D>::at(row, g >> 1) + (g & 1) * 8);
        v[i][0] = u.x, v[i][1] = u.y;
      }
    }
    if (masked) {
      // A NaN value must not reach a row that does not see its key (0 NaN = NaN): such codes
      // are taken out of the product and their columns set to NaN for the rows that see them.
      bool bad = false;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int w = 0; w < D / 32; ++w) bad |= __vcmpeq4(v[i][w] & 0x7F7F7F7Fu, 0x7F7F7F7Fu) != 0;
      if (__any_sync(0xFFFFFFFFu, bad)) {
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          uint32_t s[2];
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const int key = key0 + mt * 16 + hh * 8 + Chunk<D>::key_of_slot(g);
            s[hh] = transpose8x8((key < lim[j][0] ? 0x3C00u : 0u) | (key < lim[j][1] ? 0x3C000000u : 0u));
          }
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            uint32_t a[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {  // a0, a1: first key pair; a2, a3: second; odd: column + 1
              const int pair = (e >> 1) * 2, byte = (2 * i + (e & 1)) & 3, w = i >> 1;
              const uint32_t c0 = (v[pair][w] >> (8 * byte)) & 0x7Fu, c1 = (v[pair + 1][w] >> (8 * byte)) & 0x7Fu;
              a[e] = (c0 == 0x7Fu ? 0x3C00u : 0u) | (c1 == 0x7Fu ? 0x3C000000u : 0u);
            }
            float n[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            mma_f16(n, a[0], a[1], a[2], a[3], s[0], s[1]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (n[e] > 0.0f) z[j][i][e] = __uint_as_float(0x7FC00000u);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int w = 0; w < D / 32; ++w)
            v[i][w] &= ~__vcmpeq4(v[i][w] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
      }
    }
    // Lane (g, t) holds columns D/8 g + 2i (A rows g) and + 1 (A rows g + 8) in block i.
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
      const uint32_t p0 = __byte_perm(v[0][w], v[1][w], 0x5140), p1 = __byte_perm(v[0][w], v[1][w], 0x7362);
      const uint32_t r0 = __byte_perm(v[2][w], v[3][w], 0x5140), r1 = __byte_perm(v[2][w], v[3][w], 0x7362);
      const uint32_t a0 = lo_codes(p0), a1 = hi_codes(p0), a2 = lo_codes(r0), a3 = hi_codes(r0);
      const uint32_t c0 = lo_codes(p1), c1 = hi_codes(p1), c2 = lo_codes(r1), c3 = hi_codes(r1);
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        mma_f16(z[j][2 * w], a0, a1, a2, a3, b0[j], b1[j]);
        mma_f16(z[j][2 * w + 1], c0, c1, c2, c3, b0[j], b1[j]);
        if constexpr (kPair) {
          mma_f16(z[j][2 * w], a0, a1, a2, a3, lo0[j], lo1[j]);
          mma_f16(z[j][2 * w + 1], c0, c1, c2, c3, lo0[j], lo1[j]);
        }
      }
    }
  }
}

template <bool kBf16, int D, int NT>
__global__ void __launch_bounds__(kAttendThreads, attend_ctas_per_sm<NT>())
    attend_kernel(const AttendParams<ByQuery> p) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int kStages = attend_stages<D, NT>();
  constexpr int kTile = NT * 8;
  const int lane = lane_id(), warp = warp_id(), g = lane >> 2, t = lane & 3;
  const ByQuery& geo = p.geo;
  grid_launch_dependents();
  uint8_t* ring = smem + warp * (kStages * stage_bytes<D>());
  const int nblk = geo.cap / p.block;

  int u0, u1;
  Place pl;
  if (p.ctas > 0) {
    pl = plan_run(geo, blockIdx.x, p.ctas, p.min_chunks, u0, u1);
    if (u0 >= u1) return;
  } else {
    pl.rt = 0;
    pl.hk = blockIdx.x % geo.Hk;
    pl.b = blockIdx.x / geo.Hk;
    pl.start = u0 = 0;
    const int len = seq_len(geo.lengths, pl.b, geo.cap), cnt = seq_count(geo.counts, pl.b, geo.n);
    pl.keys = tile_keys(geo, len, cnt, 0);
    u1 = chunks_of(geo, pl.keys);
    if (pl.hk == 0 && threadIdx.x == 0)
      check_seq(geo.lengths, geo.counts, pl.b, geo.cap, geo.n, p.status);
  }
  for (;;) {
    const int tile_chunks = chunks_of(geo, pl.keys);
    const int c0 = max(u0 - pl.start, 0);
    const int c1 = min(u1 - pl.start, tile_chunks);
    if (p.ctas > 0 && c0 == 0 && pl.start >= u0 && threadIdx.x == 0) note_run(p, pl, u0, u1);
    const int len = seq_len(geo.lengths, pl.b, geo.cap), cnt = seq_count(geo.counts, pl.b, geo.n);
    const int64_t bh = static_cast<int64_t>(pl.b) * geo.Hk + pl.hk;
    const uint8_t* kp = p.k8 + bh * geo.cap * D;
    const uint8_t* vp = p.v8 + bh * geo.cap * D;
    const float* ksp = p.k_scales + bh * nblk;
    const float* vsp = p.v_scales + bh * nblk;

    auto issue = [&](int ch, int stage) {
      if (ch < c1) {
        const uint32_t s = smem_u32(ring + stage * stage_bytes<D>());
        const int key0 = ch * kChunk;
        load_chunk<D>(s, kp, key0, len);
        load_chunk<D>(s + Chunk<D>::kBytes, vp, key0, len);
        if (lane < 4) {  // ks, vs of the chunk's two halves; a half past the end repeats the first
          const int key = key0 + (lane & 1) * 16;
          cp_async4(s + 2 * Chunk<D>::kBytes + lane * 4,
                    (lane < 2 ? ksp : vsp) + (key < len ? key : key0) / p.block);
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue(c0 + warp + i * kAttendWarps, i);

    // Queries of the tile as fp16 times a power of two a row.
    QFrag<D> q[NT];
    float kmul[NT][2];
    int lim[NT][2];
    int least = len;  // keys every real row sees
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      {
        const int r = j * 8 + g;
        const bool real = r < geo.R && geo.query(r) < cnt;  // what padding rows hold does not matter
        float x[D / 4];
        load_q_row<kBf16, D>(real ? p.q + geo.row_offset(pl.b, pl.hk, r) * D : nullptr, x);
        pack_q<D>(x, p.c2, q[j], kmul[j]);
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int r = j * 8 + 2 * t + c;
        const bool real = r < geo.R && geo.query(r) < cnt;
        lim[j][c] = real ? query_keys(geo, len, cnt, geo.query(r)) : len;
        least = min(least, lim[j][c]);
      }
    }
    least = __reduce_min_sync(0xFFFFFFFFu, least);

    float z[NT][D / 16][4], l[NT][2], m[NT][2];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) z[j][i][e] = 0.0f;
      l[j][0] = l[j][1] = 0.0f;
      m[j][0] = m[j][1] = kNoMax;
    }
    float hi = -INFINITY;  // log2 of the largest V scale so far

    int stage = 0;
    for (int ch = c0 + warp; ch < c1; ch += kAttendWarps) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      const int ahead = stage == 0 ? kStages - 1 : stage - 1;
      issue(ch + (kStages - 1) * kAttendWarps, ahead);
      const int key0 = ch * kChunk;
      const bool masked = key0 + kChunk > least;
      attend_chunk<D, NT, !kBf16>(ring + stage * stage_bytes<D>(), key0, masked, kmul, q, lim, z, l, m, hi);
      __syncwarp();
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    cp_async_wait<0>();

    // Merge the warps' states: each warp puts its z, l, m into shared memory.  Rows 2t and 2t + 1
    // of a block of eight lie at t and 4 + t, which keeps eight lanes' 16-byte stores apart.
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[j][c] += __shfl_xor_sync(0xFFFFFFFFu, l[j][c], o);
    __syncthreads();
    constexpr int kStride = merge_stride<D>();
    float* mz = reinterpret_cast<float*>(smem);
    float* mlm = mz + kAttendWarps * kTile * kStride;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int at = warp * kTile + j * 8 + c * 4 + t;
        float4* dst = reinterpret_cast<float4*>(mz + at * kStride + g * (D / 8));
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
          dst[i] = make_float4(z[j][2 * i][c], z[j][2 * i][c + 2], z[j][2 * i + 1][c], z[j][2 * i + 1][c + 2]);
        if (g == 0) {
          mlm[at * 2] = l[j][c];
          mlm[at * 2 + 1] = m[j][c];
        }
      }
    __syncthreads();
    const bool whole = c0 == 0 && c1 == tile_chunks;
    const int64_t slot = (2 * static_cast<int64_t>(blockIdx.x) + (c0 == 0 ? 1 : 0)) * kTile;
    for (int idx = threadIdx.x; idx < kTile * (D / 4); idx += kAttendThreads) {
      const int row = idx / (D / 4), col = idx % (D / 4) * 4;
      const int at = (row & ~7) + (row & 1) * 4 + ((row & 7) >> 1);
      float mx = kNoMax;
#pragma unroll
      for (int w = 0; w < kAttendWarps; ++w) mx = fmaxf(mx, mlm[(w * kTile + at) * 2 + 1]);
      float4 zs = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      float ls = 0.0f;
#pragma unroll
      for (int w = 0; w < kAttendWarps; ++w) {
        const float half = ex2(0.5f * (mlm[(w * kTile + at) * 2 + 1] - mx)), f = half * half;
        const float4 x = *reinterpret_cast<const float4*>(mz + (w * kTile + at) * kStride + col);
        zs.x = fmaf(f, x.x, zs.x);
        zs.y = fmaf(f, x.y, zs.y);
        zs.z = fmaf(f, x.z, zs.z);
        zs.w = fmaf(f, x.w, zs.w);
        ls = fmaf(mlm[(w * kTile + at) * 2] * half, half, ls);
      }
      if (whole) {
        if (row < geo.R)
          write_out<kBf16, D, ByQuery>(p, geo.row_offset(pl.b, pl.hk, row), col, zs, ls, mx,
                              geo.query(row) < cnt);
      } else {
        *reinterpret_cast<float4*>(p.part_z + (slot + row) * D + col) = zs;
        if (col == 0) *reinterpret_cast<float2*>(p.part_lm + (slot + row) * 2) = make_float2(ls, mx);
      }
    }
    if (pl.start + tile_chunks >= u1) break;
    next_place(geo, pl);
    __syncthreads();  // the merge area is read before the ring is filled again
  }
}

inline int rows_per_tile(int R) { return R <= 8 ? 8 : R <= 16 ? 16 : 32; }

template <bool kBf16, int D, int NT>
cudaError_t launch_attend(AttendParams<ByQuery> p, int sms, cudaStream_t s) {
  constexpr size_t smem = ring_bytes<D, NT>() > merge_bytes<D, NT>() ? ring_bytes<D, NT>() : merge_bytes<D, NT>();
  auto* kernel = attend_kernel<kBf16, D, NT>;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kernel), smem, allowed);
  if (e != cudaSuccess) return e;
  const unsigned tiles = static_cast<unsigned>(p.geo.B) * p.geo.Hk;
  const bool aligned = p.geo.cap <= kAlignedCap;
  p.ctas = aligned ? 0 : sms * attend_ctas_per_sm<NT>();
  void* args[] = {&p};
  e = cudaLaunchKernel(reinterpret_cast<const void*>(kernel), dim3(aligned ? tiles : p.ctas),
                       dim3(kAttendThreads), args, smem, s);
  if (e != cudaSuccess || aligned) return e;
  return launch_join<kBf16, D>(p, s);
}

template <bool kBf16, int D>
cudaError_t launch_attend_nt(const AttendParams<ByQuery>& p, int sms, cudaStream_t s) {
  if (p.geo.tile == 8) return launch_attend<kBf16, D, 1>(p, sms, s);
  if (p.geo.tile == 16) return launch_attend<kBf16, D, 2>(p, sms, s);
  if constexpr (D == 64) return launch_attend<kBf16, D, 4>(p, sms, s);
  return cudaErrorInvalidValue;  // more rows are the tcgen05 kernel's
}

}  // namespace kv8

namespace {

// Rows per key/value head up to which this file's kernel is used, the tcgen05 kernel above.  us here
// and there, for 16 sequences and for one, each 8 heads of 8187 keys:
//   d = 128  bf16  16 rows 57, 92 and 18, 24    fp16  16 rows 64, 140 and 19, 29
//            bf16  24 rows 123, 88 (32-row tiles of this kernel spill registers)
//   d = 64   bf16  32 rows 61, 80 and 21, 22    fp16  32 rows 71, 111 and 22, 24
//            bf16  48 rows 83, 74
constexpr int few_rows(int d) { return d == 64 ? 32 : 16; }

int rows_per_tile(int64_t R, int d) {
  if (R > few_rows(d)) return R > kTcTileRows / 2 ? kTcTileRows : kTcTileRows / 2;
  return kv8::rows_per_tile(static_cast<int>(R));
}

// Rows of the parts: two places a CTA (for tiles of 128 rows, two and one for what its second row
// tile hands over).
size_t part_rows(int64_t R, int d, int sms) {
  if (R > few_rows(d)) return static_cast<size_t>(2) * sms * kTcTileRows;
  return static_cast<size_t>(2) * sms * kv8::kMostCtas * rows_per_tile(R, d);
}

bool too_long(int B, int Hk, int tiles, int64_t R, int d, int cap) {
  return kv8::list_too_long(B, Hk, tiles, cap, R > few_rows(d) ? kv8::kBlockKeys : kv8::kChunk);
}

}  // namespace

size_t kv8_attend_workspace_bytes(int B, int Hk, int G, int n, int d, int cap, int sms) {
  const int64_t R = static_cast<int64_t>(G) * n;
  if (R <= few_rows(d) && cap <= kv8::kAlignedCap) return 0;  // nothing to join
  const int tiles = static_cast<int>((R + rows_per_tile(R, d) - 1) / rows_per_tile(R, d));
  if (too_long(B, Hk, tiles, R, d, cap)) return 0;  // refused
  return part_rows(R, d, sms) * (d + 2) * sizeof(float) + static_cast<size_t>(B) * Hk * tiles * sizeof(int2);
}

namespace {

template <class Geo>
kv8::AttendParams<Geo> attend_params(const Kv8Args& a, int ctas, int min_chunks) {
  kv8::AttendParams<Geo> p{};
  const int R = a.G * a.n, tile = rows_per_tile(R, a.d);
  const size_t rows = part_rows(R, a.d, a.sms);
  p.geo = {{a.B, a.Hk, a.G, a.n, a.cap, R, tile, (R + tile - 1) / tile, a.causal, a.lengths, a.counts, false}};
  p.block = a.block;
  p.c2 = a.c * kv8::kLog2e;
  p.q = static_cast<const uint16_t*>(a.q);
  p.k8 = a.k8;
  p.v8 = a.v8;
  p.k_scales = a.k_scales;
  p.v_scales = a.v_scales;
  p.o = static_cast<uint16_t*>(a.o);
  p.lse = a.lse;
  p.part_z = static_cast<float*>(a.workspace);
  p.part_lm = p.part_z + rows * a.d;
  p.runs = reinterpret_cast<int2*>(p.part_lm + rows * 2);
  p.ctas = ctas;
  p.min_chunks = min_chunks;
  p.status = a.status;
  return p;
}

}  // namespace

int launch_kv8_attend(const Kv8Args& a, cudaStream_t s, std::string& err) {
  const int64_t R = static_cast<int64_t>(a.G) * a.n;
  const int tiles = static_cast<int>((R + rows_per_tile(R, a.d) - 1) / rows_per_tile(R, a.d));
  if (too_long(a.B, a.Hk, tiles, R, a.d, a.cap)) {
    err = "B * H * n_q * cap is too large for one call";
    return -2;
  }
  cudaError_t e;
  if (R > few_rows(a.d)) {
    auto p = attend_params<kv8::ByHead>(a, a.sms, 2);
    if (a.bf16)
      e = a.d == 128 ? launch_kv8_tc<true, 128>(p, s) : launch_kv8_tc<true, 64>(p, s);
    else
      e = a.d == 128 ? launch_kv8_tc<false, 128>(p, s) : launch_kv8_tc<false, 64>(p, s);
  } else {
    auto p = attend_params<kv8::ByQuery>(a, kv8::kMostCtas * a.sms, 2 * kv8::kAttendWarps);
    if (a.bf16)
      e = a.d == 128 ? kv8::launch_attend_nt<true, 128>(p, a.sms, s) : kv8::launch_attend_nt<true, 64>(p, a.sms, s);
    else
      e = a.d == 128 ? kv8::launch_attend_nt<false, 128>(p, a.sms, s) : kv8::launch_attend_nt<false, 64>(p, a.sms, s);
  }
  if (e != cudaSuccess) {
    err = std::string("kv8 attention launch: ") + cudaGetErrorString(e);
    return -5;
  }
  return 0;
}

}  // namespace ea
