// Attention of a few query rows over the 8-bit cache.
//
// Row r of a key/value head (query i of head g, r = i G + g) has the scores
//     s_rj = c ks_j (q_r . k_j)          (ks, vs: the scales of key j's block)
// and O_r = sum_j e^{s_rj - LSE_r} vs_j v_j.  In base 2, with x_rj = log2(e) s_rj + log2(vs_j),
// a shift m_r near the running maximum of x_r, and P_rj = 2^{x_rj - m_r}:
//     z_r = sum_j P_rj v_j,   l_r = sum_j P_rj / vs_j,   O_r = z_r / l_r,
//     LSE_r = ln 2 (m_r + log2 l_r),
// so a value block's scale costs one constant a block: P is what the product takes and z needs
// no second scaling.  P is rounded to fp16 for that product (half a step is 2^-12, an eighth of
// the bf16 output's); m_r is set so that the largest P is 2^6 and is raised only when a P would
// pass 2^14, which keeps P inside fp16 and weights down to 2^-20 of the largest at full precision
// (the sums z and l are float32).
//
// The work is every chunk of 32 keys of every (sequence, head, row tile); each CTA takes an equal
// run of that list, whatever the sequences' lengths, and its warps take the run's chunks in turn,
// each with its own z, l and m.  At the end of a tile the warps' states are merged; a tile that
// one CTA holds whole is written at once, and a CTA's part of a tile shared with others (at most
// one at each end of its run) goes to the workspace as (z, l, m), joined by a second kernel.
#include "kv8_mma.cuh"

namespace ea {
namespace kv8 {

constexpr int kAttendWarps = 8;
constexpr int kAttendThreads = kAttendWarps * 32;
constexpr float kTop = 6.0f;     // log2 of the largest P when m is set
constexpr float kRaise = 14.0f;  // a larger log2 P raises m
constexpr float kNoMax = -3.0e38f;

struct AttendParams {
  Geometry geo;
  int block;
  float c2;  // c log2(e)
  const uint16_t* q;
  const uint8_t* k8;
  const uint8_t* v8;
  const float* k_scales;
  const float* v_scales;
  uint16_t* o;
  float* lse;
  float* part;     // [2 gridDim.x][tile][D + 2]: z, l, m
  int min_chunks;  // a CTA's run has at least this many
  uint32_t* status;
};

template <int D>
constexpr int attend_stages() { return D == 128 ? 3 : 6; }
template <int D>
constexpr int stage_bytes() { return 2 * Chunk<D>::kBytes + 32; }  // K, V, four scales
template <int D>
constexpr size_t ring_bytes() { return static_cast<size_t>(kAttendWarps) * attend_stages<D>() * stage_bytes<D>(); }
// The warps' states at a tile's end, over the drained ring: z, then l and m of each row.
template <int D, int NT>
constexpr size_t merge_bytes() { return static_cast<size_t>(kAttendWarps) * NT * 8 * (D + 2) * sizeof(float); }

__device__ __forceinline__ int64_t run_length(int64_t total, int ctas, int min_chunks) {
  const int64_t per = (total + ctas - 1) / ctas;
  return per < min_chunks ? min_chunks : per;
}

template <bool kBf16>
__device__ __forceinline__ uint16_t to16(float x) {
  if constexpr (kBf16) return __bfloat16_as_ushort(__float2bfloat16_rn(x));
  return __half_as_ushort(__float2half_rn(x));
}

// Writes one element of a finished row and, for column 0, its LSE.  z / l with l = 0 is a row
// that sees no key: O = 0, LSE = -inf.
template <bool kBf16>
__device__ __forceinline__ void write_out(const AttendParams& p, int D, int64_t row, int col,
                                          float z, float l, float m, bool real) {
  const bool empty = l == 0.0f;
  p.o[row * D + col] = to16<kBf16>(empty || !real ? 0.0f : z / l);
  if (col == 0) {
    p.lse[row] = empty || !real ? -INFINITY : kLn2 * (m + log2f(l));
    if (empty && real) raise_empty_row(p.status);
  }
}

// One chunk of 32 keys against the tile's rows.
template <int D, int NT>
__device__ __forceinline__ void attend_chunk(const uint8_t* st, int key0, bool masked, int block,
                                             float kmul, const QFrag<D> (&q)[NT],
                                             const int (&lim)[NT][2], float (&z)[NT][D / 16][4],
                                             float (&l)[NT][2], float (&m)[NT][2]) {
  const int lane = lane_id(), g = lane >> 2, t = lane & 3;
  const float* sc = reinterpret_cast<const float*>(st + 2 * Chunk<D>::kBytes);
  float x[2][NT][4];
  float inv_vs[2];
  float top = -INFINITY;  // largest excess of x over the allowed shift
#pragma unroll
  for (int mt = 0; mt < 2; ++mt) {
    scores16<D, NT>(st, mt, q, x[mt]);
    const float kf = kmul * sc[mt], vs = sc[2 + mt];
    const float lvs = log2f(vs);
    inv_vs[mt] = 1.0f / vs;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float y = fmaf(x[mt][j][e], kf, lvs);
        if (masked) {
          const int key = key0 + mt * 16 + (e >> 1) * 8 + Chunk<D>::key_of_slot(g);
          if (key >= lim[j][e & 1]) y = -INFINITY;
        }
        x[mt][j][e] = y;
        top = fmaxf(top, y - m[j][e & 1]);
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
        const float r = ex2(m[j][c] - mn);
        m[j][c] = mn;
        l[j][c] *= r;
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
    [[maybe_unused]] uint32_t seen0[NT], seen1[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      float pr[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        pr[e] = ex2(x[mt][j][e] - m[j][e & 1]);
        l[j][e & 1] = fmaf(pr[e], inv_vs[mt], l[j][e & 1]);
      }
      b0[j] = transpose8x8(pack_f16(pr[0], pr[1]));
      b1[j] = transpose8x8(pack_f16(pr[2], pr[3]));
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
      }
    }
  }
}

template <bool kBf16, int D, int NT>
__global__ void __launch_bounds__(kAttendThreads, 1) attend_kernel(const AttendParams p) {
  extern __shared__ __align__(128) uint8_t smem[];
  constexpr int kStages = attend_stages<D>();
  constexpr int kTile = NT * 8;
  const int lane = lane_id(), warp = warp_id(), g = lane >> 2, t = lane & 3;
  const Geometry& geo = p.geo;
  const int64_t total = total_chunks(geo);
  const int64_t per = run_length(total, gridDim.x, p.min_chunks);
  const int64_t u0 = blockIdx.x * per, u1 = min(u0 + per, total);
  if (u0 >= u1) return;
  uint8_t* ring = smem + warp * (kStages * stage_bytes<D>());
  const int nblk = geo.cap / p.block;

  Place pl = place_of(geo, u0);
  for (;;) {
    const int tile_chunks = chunks_of(pl.keys);
    const int c0 = static_cast<int>(max(u0 - pl.start, static_cast<int64_t>(0)));
    const int c1 = static_cast<int>(min(u1 - pl.start, static_cast<int64_t>(tile_chunks)));
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

    // Queries of the tile as fp16 times 2^e.
    QFrag<D> q[NT];
    int lim[NT][2];
    int least = len;  // keys every real row sees
    float qmul;
    {
      float amax = 0.0f;
#pragma unroll
      for (int pass = 0; pass < 2; ++pass) {
        if (pass) qmul = pow2(q_exp(warp_max(amax)));
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int r = pl.rt * kTile + j * 8 + g;
          float x[D / 4];
          load_q_row<kBf16, D>(
              r < geo.R ? p.q + row_offset(pl.b, pl.hk, geo.Hk, geo.G, geo.n, r) * D : nullptr, x);
          if (pass) {
            pack_q<D>(x, qmul, q[j]);
          } else {
#pragma unroll
            for (int e = 0; e < D / 4; ++e) amax = fmaxf(amax, finite_abs(x[e]));
          }
        }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int r = pl.rt * kTile + j * 8 + 2 * t + c;
          const bool real = r < geo.R && r / geo.G < cnt;
          lim[j][c] = real ? row_keys(geo, len, cnt, r) : len;
          least = min(least, lim[j][c]);
        }
      least = __reduce_min_sync(0xFFFFFFFFu, least);
    }
    const float kmul = p.c2 / qmul;

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

    int stage = 0;
    for (int ch = c0 + warp; ch < c1; ch += kAttendWarps) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      const int ahead = stage == 0 ? kStages - 1 : stage - 1;
      issue(ch + (kStages - 1) * kAttendWarps, ahead);
      const int key0 = ch * kChunk;
      const bool masked = key0 + kChunk > least;
      attend_chunk<D, NT>(ring + stage * stage_bytes<D>(), key0, masked, p.block, kmul, q, lim, z, l, m);
      __syncwarp();
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    cp_async_wait<0>();

    // Merge the warps' states: each warp puts its z, l, m into shared memory.
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[j][c] += __shfl_xor_sync(0xFFFFFFFFu, l[j][c], o);
    __syncthreads();
    float* mz = reinterpret_cast<float*>(smem);
    float* mlm = mz + kAttendWarps * kTile * D;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int row = j * 8 + 2 * t + c;
        float* dst = mz + (warp * kTile + row) * D + g * (D / 8);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          dst[2 * i] = z[j][i][c];
          dst[2 * i + 1] = z[j][i][c + 2];
        }
        if (g == 0) {
          mlm[(warp * kTile + row) * 2] = l[j][c];
          mlm[(warp * kTile + row) * 2 + 1] = m[j][c];
        }
      }
    __syncthreads();
    const bool whole = c0 == 0 && c1 == tile_chunks;
    float* part = p.part + (2 * static_cast<int64_t>(blockIdx.x) + (c0 == 0 ? 1 : 0)) * kTile * (D + 2);
    for (int idx = threadIdx.x; idx < kTile * D; idx += kAttendThreads) {
      const int row = idx / D, col = idx % D;
      float mx = kNoMax;
#pragma unroll
      for (int w = 0; w < kAttendWarps; ++w) mx = fmaxf(mx, mlm[(w * kTile + row) * 2 + 1]);
      float zs = 0.0f, ls = 0.0f;
#pragma unroll
      for (int w = 0; w < kAttendWarps; ++w) {
        const float f = ex2(mlm[(w * kTile + row) * 2 + 1] - mx);
        zs = fmaf(f, mz[(w * kTile + row) * D + col], zs);
        ls = fmaf(f, mlm[(w * kTile + row) * 2], ls);
      }
      const int r = pl.rt * kTile + row;
      if (whole) {
        if (r < geo.R)
          write_out<kBf16>(p, D, row_offset(pl.b, pl.hk, geo.Hk, geo.G, geo.n, r), col, zs, ls, mx,
                           r / geo.G < cnt);
      } else {
        part[row * (D + 2) + col] = zs;
        if (col == 0) {
          part[row * (D + 2) + D] = ls;
          part[row * (D + 2) + D + 1] = mx;
        }
      }
    }
    if (pl.start + tile_chunks >= u1) break;
    next_place(geo, pl);
    __syncthreads();  // the merge area is read before the ring is filled again
  }
}

// Joins the parts of tiles that several CTAs shared, and writes tiles that see no key at all.
// One CTA a tile.
template <bool kBf16, int D>
__global__ void __launch_bounds__(128) attend_join_kernel(const AttendParams p, int ctas) {
  const Geometry& geo = p.geo;
  int64_t id = blockIdx.x;
  Place pl;
  pl.rt = static_cast<int>(id % geo.tiles);
  id /= geo.tiles;
  pl.hk = static_cast<int>(id % geo.Hk);
  pl.b = static_cast<int>(id / geo.Hk);
  const int len = seq_len(geo.lengths, pl.b, geo.cap), cnt = seq_count(geo.counts, pl.b, geo.n);
  if (pl.rt == 0 && pl.hk == 0 && threadIdx.x == 0)
    check_seq(geo.lengths, geo.counts, pl.b, geo.cap, geo.n, p.status);
  pl.keys = tile_keys(geo, len, cnt, pl.rt);
  const int r0 = pl.rt * geo.tile, rows = min(geo.tile, geo.R - r0);
  if (pl.keys == 0) {
    for (int idx = threadIdx.x; idx < rows * D; idx += blockDim.x) {
      const int r = r0 + idx / D;
      write_out<kBf16>(p, D, row_offset(pl.b, pl.hk, geo.Hk, geo.G, geo.n, r), idx % D, 0.0f, 0.0f,
                       0.0f, r / geo.G < cnt);
    }
    return;
  }
  const int64_t per = run_length(total_chunks(geo), ctas, p.min_chunks);
  int64_t start = sequence_start(geo, pl.b) + pl.hk * head_chunks(geo, pl.b);
  for (int rt = 0; rt < pl.rt; ++rt) start += chunks_of(tile_keys(geo, len, cnt, rt));
  const int64_t end = start + chunks_of(pl.keys);
  const int64_t first = start / per, last = (end - 1) / per;
  if (first == last) return;
  for (int idx = threadIdx.x; idx < rows * D; idx += blockDim.x) {
    const int row = idx / D, col = idx % D, r = r0 + row;
    float mx = kNoMax, zs = 0.0f, ls = 0.0f;
    for (int64_t c = first; c <= last; ++c) {
      const float* part = p.part + ((2 * c + (c == first ? 1 : 0)) * geo.tile + row) * (D + 2);
      mx = fmaxf(mx, part[D + 1]);
    }
    for (int64_t c = first; c <= last; ++c) {
      const float* part = p.part + ((2 * c + (c == first ? 1 : 0)) * geo.tile + row) * (D + 2);
      const float f = ex2(part[D + 1] - mx);
      zs = fmaf(f, part[col], zs);
      ls = fmaf(f, part[D], ls);
    }
    write_out<kBf16>(p, D, row_offset(pl.b, pl.hk, geo.Hk, geo.G, geo.n, r), col, zs, ls, mx,
                     r / geo.G < cnt);
  }
}

inline int rows_per_tile(int R) { return R <= 8 ? 8 : R <= 16 ? 16 : 32; }

template <bool kBf16, int D, int NT>
cudaError_t launch_attend(const AttendParams& p, int ctas, cudaStream_t s) {
  constexpr size_t smem = ring_bytes<D>() > merge_bytes<D, NT>() ? ring_bytes<D>() : merge_bytes<D, NT>();
  auto* kernel = attend_kernel<kBf16, D, NT>;
  const cudaError_t attr = cudaFuncSetAttribute(
      kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (attr != cudaSuccess) return attr;
  AttendParams pp = p;
  void* args[] = {&pp};
  cudaError_t e = cudaLaunchKernel(reinterpret_cast<const void*>(kernel), dim3(ctas),
                                   dim3(kAttendThreads), args, smem, s);
  if (e != cudaSuccess) return e;
  void* jargs[] = {&pp, &ctas};
  return cudaLaunchKernel(reinterpret_cast<const void*>(attend_join_kernel<kBf16, D>),
                          dim3(static_cast<unsigned>(p.geo.B) * p.geo.Hk * p.geo.tiles), dim3(128),
                          jargs, 0, s);
}

template <bool kBf16, int D>
cudaError_t launch_attend_nt(const AttendParams& p, int ctas, cudaStream_t s) {
  if (p.geo.tile == 8) return launch_attend<kBf16, D, 1>(p, ctas, s);
  if (p.geo.tile == 16) return launch_attend<kBf16, D, 2>(p, ctas, s);
  return launch_attend<kBf16, D, 4>(p, ctas, s);
}

}  // namespace kv8

size_t kv8_attend_workspace_bytes(int, int, int G, int n, int d, int sms) {
  const int64_t R = static_cast<int64_t>(G) * n;
  const int tile = kv8::rows_per_tile(R > 32 ? 32 : static_cast<int>(R));
  return static_cast<size_t>(2) * sms * tile * (d + 2) * sizeof(float);
}

int launch_kv8_attend(const Kv8Args& a, cudaStream_t s, std::string& err) {
  kv8::AttendParams p{};
  const int R = a.G * a.n, tile = kv8::rows_per_tile(R);
  p.geo = {a.B, a.Hk, a.G, a.n, a.cap, R, tile, (R + tile - 1) / tile, a.causal, a.lengths, a.counts, false};
  p.block = a.block;
  p.c2 = a.c * kv8::kLog2e;
  p.q = static_cast<const uint16_t*>(a.q);
  p.k8 = a.k8;
  p.v8 = a.v8;
  p.k_scales = a.k_scales;
  p.v_scales = a.v_scales;
  p.o = static_cast<uint16_t*>(a.o);
  p.lse = a.lse;
  p.part = static_cast<float*>(a.workspace);
  p.min_chunks = 2 * kv8::kAttendWarps;
  p.status = a.status;
  const int ctas = a.sms;
  cudaError_t e;
  if (a.bf16)
    e = a.d == 128 ? kv8::launch_attend_nt<true, 128>(p, ctas, s) : kv8::launch_attend_nt<true, 64>(p, ctas, s);
  else
    e = a.d == 128 ? kv8::launch_attend_nt<false, 128>(p, ctas, s) : kv8::launch_attend_nt<false, 64>(p, ctas, s);
  if (e != cudaSuccess) {
    err = std::string("kv8 attention launch: ") + cudaGetErrorString(e);
    return -5;
  }
  return 0;
}

}  // namespace ea
