// What the attention kernels for few and for many rows share: their arguments, the way a row is
// written, and the kernel that joins the parts of tiles cut between CTAs.
#pragma once
#include "kv8_plan.cuh"

namespace ea {
namespace kv8 {

constexpr float kTop = 6.0f;     // log2 of the largest P when m is set
constexpr float kRaise = 14.0f;  // a larger log2 P raises m
constexpr float kNoMax = -3.0e38f;

// The sum l.  P follows x, the score and log2 of its V block's scale, while l adds 2^(s - m) of the
// bare score s as P / vs, and scales lie anywhere in 2^-100 .. 2^120 (a block of zeros has 2^-100).
// So that l neither overflows nor loses keys:
//   * scales below 2^kLeastScale, or more than 2^kScaleSpan below the tile's largest so far, enter x
//     and l as that bound, and what the V product takes of the block is multiplied by the rest (in
//     fp16: 2^-95 of a row's O, or 2^-101 of a code a key, can be lost).  P of a key that counts
//     (2^-24 of the largest 2^s) is then above 2^-126, where ex2 flushes, and s below m + 84;
//   * l is kept 2^kLift times as large: up to 2^30 keys sum to less than 2^127, and under scales of
//     2^120 keys of 2^-24 of the largest still count;
//   * factors of l that a new m brings are applied as two halves: one could be flushed where its
//     product with l is not.
constexpr float kLift = 12.0f;
constexpr float kLiftFactor = 4096.0f;
constexpr float kLeastScale = -70.0f;
constexpr float kScaleSpan = 96.0f;
// A row's LSE from its l and m.
__device__ __forceinline__ float row_lse(float l, float m) { return kLn2 * (m + log2f(l * (1.0f / kLiftFactor))); }

template <class Geo>
struct AttendParams {
  Geo geo;
  int block;
  float c2;  // c log2(e)
  const uint16_t* q;
  const uint8_t* k8;
  const uint8_t* v8;
  const float* k_scales;
  const float* v_scales;
  uint16_t* o;
  float* lse;
  float* part_z;   // [2 ctas][tile][D]: parts of shared tiles, two places a CTA
  float* part_lm;  // [2 ctas][tile][2]: their l and m
  int2* runs;      // [tiles of all heads] first and last CTA of a tile that some row of sees a key
  int ctas;        // runs the work is cut into; 0: one CTA a tile, and no parts
  int min_chunks;  // a run has at least this many
  uint32_t* status;
};

// Writes four columns of a finished row and, with the first of them, its LSE.  l = 0 is a row
// that sees no key: O = 0, LSE = -inf.
template <bool kBf16, int D, class Geo>
__device__ __forceinline__ void write_out(const AttendParams<Geo>& p, int64_t row, int col, float4 z,
                                          float l, float m, bool real) {
  const bool none = l == 0.0f || !real;
  const float inv = none ? 0.0f : kLiftFactor / l;
  uint2 w;
  if constexpr (kBf16) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(z.x * inv, z.y * inv), b = __floats2bfloat162_rn(z.z * inv, z.w * inv);
    w = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  } else {
    w = make_uint2(pack2<false>(z.x * inv, z.y * inv), pack2<false>(z.z * inv, z.w * inv));
  }
  if (none) w = make_uint2(0u, 0u);
  *reinterpret_cast<uint2*>(p.o + row * D + col) = w;
  if (col == 0) {
    p.lse[row] = none ? -INFINITY : row_lse(l, m);
    if (none && real) raise_empty_row(p.status);
  }
}

// The CTA that holds a tile's first chunk notes which CTAs share it (u0, u1: its run).
template <class Geo>
__device__ __forceinline__ void note_run(const AttendParams<Geo>& p, const Place& pl, int u0, int u1) {
  const int per = u1 - u0;  // a run that ends before its length is the last
  const int end = pl.start + chunks_of(p.geo, pl.keys);
  const int more = end > u1 ? (end - u1 + per - 1) / per : 0;
  const int64_t id = (static_cast<int64_t>(pl.b) * p.geo.Hk + pl.hk) * p.geo.tiles + pl.rt;
  p.runs[id] = make_int2(blockIdx.x, blockIdx.x + more);
}

// Joins the parts of tiles that several CTAs shared, and writes tiles that see no key at all.
// One warp a row, eight rows a CTA.
constexpr int kJoinWarps = 8;
template <bool kBf16, int D, class Geo>
__global__ void __launch_bounds__(kJoinWarps * 32) attend_join_kernel(const AttendParams<Geo> p) {
  constexpr int kCols = D / 32;  // columns of a lane
  const Geo& geo = p.geo;
  int id = blockIdx.x;
  Place pl;
  pl.rt = id % geo.tiles;
  id /= geo.tiles;
  pl.hk = id % geo.Hk;
  pl.b = id / geo.Hk;
  const int lane = lane_id();
  const int row = blockIdx.y * kJoinWarps + warp_id(), r = pl.rt * geo.tile + row;
  const int len = seq_len(geo.lengths, pl.b, geo.cap), cnt = seq_count(geo.counts, pl.b, geo.n);
  if (pl.rt == 0 && pl.hk == 0 && blockIdx.y == 0 && threadIdx.x == 0)
    check_seq(geo.lengths, geo.counts, pl.b, geo.cap, geo.n, p.status);
  pl.keys = tile_keys(geo, len, cnt, pl.rt);
  grid_dependency_wait();  // by every warp: what follows on the stream may rely on this kernel
  int first = 0, last = 0;
  if (pl.keys > 0) {
    // Kept inside the parts even if the lengths changed since the first kernel read them (which
    // leaves the result undefined, but not the addresses).
    const int2 run = p.runs[blockIdx.x];
    first = min(max(run.x, 0), p.ctas - 1);
    last = min(max(run.y, first), p.ctas - 1);
  }
  if (r >= geo.R || (pl.keys > 0 && first == last)) return;  // or one CTA held the tile whole
  float mx = kNoMax, l = 0.0f;
  float z[kCols];
#pragma unroll
  for (int i = 0; i < kCols; ++i) z[i] = 0.0f;
  if (pl.keys > 0) {
    // Place 1 of the first CTA (the tile starts there), place 0 of the others.
    const int all = last - first + 1;
    auto place = [&](int q) {
      return static_cast<int64_t>(2 * (first + q) + (q == 0 ? 1 : 0)) * geo.tile + row;
    };
    for (int q0 = 0; q0 < all; q0 += 32) {
      const int parts = min(all - q0, 32);
      float2 lm = make_float2(0.0f, kNoMax);
      if (lane < parts) lm = *reinterpret_cast<const float2*>(p.part_lm + place(q0 + lane) * 2);
      const float mn = fmaxf(mx, warp_max(lm.y)), old_half = ex2(0.5f * (mx - mn)), old = old_half * old_half;
      mx = mn;
      const float half = ex2(0.5f * (lm.y - mx)), f = half * half;
      float ls = lm.x * half * half;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ls += __shfl_xor_sync(0xFFFFFFFFu, ls, o);
      l = fmaf(l * old_half, old_half, ls);
#pragma unroll
      for (int i = 0; i < kCols; ++i) z[i] *= old;
#pragma unroll 4
      for (int c = 0; c < parts; ++c) {
        const float* src = p.part_z + place(q0 + c) * D + lane * kCols;
        const float w = __shfl_sync(0xFFFFFFFFu, f, c);
        if constexpr (kCols == 4) {
          const float4 x = *reinterpret_cast<const float4*>(src);
          z[0] = fmaf(w, x.x, z[0]), z[1] = fmaf(w, x.y, z[1]);
          z[2] = fmaf(w, x.z, z[2]), z[3] = fmaf(w, x.w, z[3]);
        } else {
          const float2 x = *reinterpret_cast<const float2*>(src);
          z[0] = fmaf(w, x.x, z[0]), z[1] = fmaf(w, x.y, z[1]);
        }
      }
    }
  }
  float4 out = make_float4(z[0], z[1], 0.0f, 0.0f);
  if constexpr (kCols == 4) {
    out.z = z[2], out.w = z[3];
  } else {  // two lanes' columns make one store
    out.z = __shfl_down_sync(0xFFFFFFFFu, z[0], 1);
    out.w = __shfl_down_sync(0xFFFFFFFFu, z[1], 1);
    if (lane & 1) return;
  }
  write_out<kBf16, D, Geo>(p, geo.row_offset(pl.b, pl.hk, r), lane * kCols, out, l, mx,
                      geo.query(r) < cnt);
}

template <bool kBf16, int D, class Geo>
cudaError_t launch_join(AttendParams<Geo>& p, cudaStream_t s) {
  void* args[] = {&p};
  const unsigned tiles = static_cast<unsigned>(p.geo.B) * p.geo.Hk * p.geo.tiles;
  const int rows = p.geo.R < p.geo.tile ? p.geo.R : p.geo.tile;
  return launch_after(reinterpret_cast<const void*>(attend_join_kernel<kBf16, D, Geo>),
                      dim3(tiles, (rows + kJoinWarps - 1) / kJoinWarps), dim3(kJoinWarps * 32), args, s);
}

}  // namespace kv8

// Attention of many rows on the tcgen05 tensor cores (kv8_tc_*.cu), in tiles of 256 rows, or of 128
// where a head has no more.
constexpr int kTcTileRows = 256;
template <bool kBf16, int D>
cudaError_t launch_kv8_tc(kv8::AttendParams<kv8::ByHead>& p, cudaStream_t s);

}  // namespace ea
