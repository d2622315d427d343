// Attention of many query rows over the 8-bit cache, on the tcgen05 tensor cores.
//
// The mathematics is that of kv8_attend.cu: in base 2, x_rj = log2(e) s_rj + log2(vs_j),
// P_rj = 2^{x_rj - m_r} rounded to fp16, z = P V on the codes, l = sum P / vs.
//   * S = Q K^T is kind::f8f6f4 on the codes as they lie in memory.  A query row over a power of
//     two (its largest value 224 .. 448) is a sum of 8-bit terms, q = q1 + q2 (+ q3), whose products
//     add up in one float32 accumulator; two of them cost what one product on 16-bit operands would.
//     q1 is E4M3 and leaves at most half of its step, 8 units of a bf16 value's last place or 64 of an
//     fp16 one's; the others are E5M2, whose three bits hold every whole number up to 8, and all but 4
//     of 64.  So two terms hold a bf16 value and three an fp16 one exactly, down to 2^-6, which is at
//     most 2^-13 of the largest.  Below, where q1 steps by 2^-9, E5M2's range is what counts: two
//     terms lose at most 2^-14, three 2^-17 (2^-21 and 2^-24 of the largest; E4M3 terms would lose up
//     to 2^-10 however many there were).
//   * P V is kind::f16: V's codes are widened to fp16 on the way into shared memory (exact); for fp16
//     outputs P is a pair of values (Config::kPair).
//
// One CTA walks its run's blocks of 128 keys with two row tiles of 128 (rows ordered by head, so
// they lie in a row in memory): rows r0 .. and r0 + 128 .. of the same head, or, for heads of at
// most 128 rows, the same rows twice, one tile taking the even blocks and the other the odd ones;
// tile 1 then hands its state to tile 0 (through L2) at the end.  Either way the tensor core works on one
// tile while the other's softmax runs.  Warpgroups:
//   0  warps 0, 1: MMA issuers of the two tiles (per block j: P V of the block before, then
//      S_j); warp 2: TMA producer of the code tiles of K and of V, and their scales; warp 3: the run's tiles one
//      after another, as the other warps need to know them (Seg)
//   1, 2  softmax of tile 0 and 1: one thread a row (TMEM lane of the warp's quadrant); at a
//      tile's start all of them cut the queries into terms
//   3  converters: one thread a key, its V codes into an fp16 tile
// S and P share TMEM columns; O stays in TMEM for the length of a tile.
//
// Measured (d = 128): 2048 rows against 32768 keys of 8 heads, causal, bf16, 225 us, 1.21 PFLOP/s, 64 %
// of the measured bf16 rate; bound by a block's chain of products and exponentials, the tensor pipe
// active about half of the cycles.  48 rows against up to 8191 keys of 128 heads: 81 us.  fp16: 345
// and 116 us.
//
// The registers of 512 threads are dealt again: softmax holds a row's 128 scores, the others
// need few (kRegs*: their sum over the warpgroups is what the block was launched with).
#pragma once
#include "kv8_attend.cuh"
#include "tile.cuh"
#include "tmap.h"

namespace ea {
namespace kv8 {
namespace tc {

constexpr int kRows = 128;   // of a row tile
constexpr int kThreads = 512;
constexpr int kGroups = kBlockKeys / 16;  // scale groups of a block
constexpr int kRegsIssue = 64, kRegsSoftmax = 184, kRegsConvert = 80;
// Format fields of a kind::f8f6f4 instruction descriptor (0 is E4M3) for E5M2 in A or in B, whatever the
// other operand is.
constexpr uint32_t kE5m2InA = 1u << 7, kE5m2InB = 1u << 10;
constexpr int kSegReaders = 15;  // warps that are told of each tile
static_assert(kRegsIssue + 2 * kRegsSoftmax + kRegsConvert <= 4 * 128, "more registers than launched");

template <bool kBf16, int D>
struct Config {
  using T8 = Tile<kRows, D / 2>;        // 128 rows of D bytes, as D / 2 16-bit columns
  using TV = Tile<kBlockKeys, D>;       // fp16
  static constexpr int kTerms = kBf16 ? 2 : 3;
  // P as a pair of fp16 values (two products): for fp16 outputs the rounding of one would equal
  // their own (relative error of 48 rows against 16 x 8191 keys 2.9e-4 beside the 2.1e-4 of float32
  // P, which the pair has too).  It costs 246 to 345 us on 2048 rows of 32768 keys, 8 heads, and 88 to
  // 117 on those 48; for bf16 outputs, whose error it would change from 1.67e-3 to 1.66e-3, 229 to 328
  // and 83 to 113.
  static constexpr bool kPair = !kBf16;
  static constexpr int kSK = 2, kSV = 2;  // stages of K tiles and of V tiles
  static constexpr int kSR = kBf16 ? 3 : 2;  // of raw V blocks
  static constexpr int kRaw = kBlockKeys * D;
  static constexpr int kOffK = 2 * kTerms * T8::kBytes;  // Q: [tile][term]
  static constexpr int kOffV = kOffK + kSK * T8::kBytes;
  static constexpr int kOffR = kOffV + kSV * TV::kBytes;
  static constexpr int kOffShared = kOffR + kSR * kRaw;
  static_assert(kOffShared % 16 == 0, "the shared block is misaligned");
};

// One tile of the run, as every role sees it.
struct Seg {
  int b, hk, len, cnt;
  int r0;            // first row
  int j0, steps;     // first block and number of blocks
  bool last;         // of the run
  bool whole;        // the tile is this CTA's alone
  int slot;          // else where its part goes
  int reach[2];      // blocks row tile t takes, counted from block 0
  int least[2];      // keys every real row of row tile t sees (blocks past them are masked)
};

struct Scales {  // of one block, per 16 keys
  float k[kGroups], log2_v[kGroups], inv_v[kGroups];  // inv_v: 2^kLift / vs
  int8_t rest[kGroups];  // log2 of what a raised scale (kv8_attend.cuh) leaves to the V values, else 0
  bool raised;           // some group's scale was
};

struct Shared {
  uint64_t q_full, q_free, h_full, h_free, turn[2];
  uint64_t s_full[2], p_full[2], o_done[2], o_read[2];
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], r_full[3], r_empty[3], sc_full[4];
  uint64_t seg_full[4], seg_empty[4];
  Seg seg[4];                       // by tile number mod 4
  uint32_t tmem_base;
  bool idle;                        // nothing to do for this CTA
  uint32_t nan_seen[4];             // by tile number mod 4: a masked block's V held NaN codes
                                    // (cleared two tiles ahead, where its last reader is done)
  float row_mul[2][2 * kRows];      // by tile number mod 2: what put_queries leaves
  Scales scales[4];                 // by block number mod 4
};

// Least factor of a score: 0 (c = 0) would turn masked scores, -inf, to NaN.
constexpr float kLeastFactor = 1.17549435e-38f;

// block_probs takes x - m in one rounding, so the largest P is off 2^kTop by the rounding of m.
// Up to this |m| that is at most 2^(1/4); far above, P would leave fp16 or all of a row's be 0.
constexpr float kExactShift = 4194304.0f;  // 2^22, where float32 steps by 1/2

template <int N>
__device__ __forceinline__ void regs_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void regs_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

__device__ __forceinline__ Seg segment(const ByHead& g, const Place& pl, int u0, int u1, int cta) {
  Seg s;
  s.b = pl.b, s.hk = pl.hk;
  s.len = seq_len(g.lengths, pl.b, g.cap);
  s.cnt = seq_count(g.counts, pl.b, g.n);
  s.r0 = pl.rt * g.tile;
  const int blocks = chunks_of(g, pl.keys);
  s.j0 = max(u0 - pl.start, 0);
  const int j1 = min(u1 - pl.start, blocks);
  s.steps = j1 - s.j0;
  s.whole = s.j0 == 0 && j1 == blocks;
  s.last = pl.start + blocks >= u1;
  s.slot = 2 * cta + (s.j0 == 0 ? 1 : 0);
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int a = s.r0 + (g.tile > kRows ? t * kRows : 0), z = min(a + kRows, g.R);
    int lo, hi;
    const bool any = a < g.R && g.span(a, z, s.cnt, lo, hi);
    s.reach[t] = any ? chunks_of(g, query_keys(g, s.len, s.cnt, hi)) : 0;
    s.least[t] = any ? query_keys(g, s.len, s.cnt, lo) : s.len;
  }
  return s;
}

// A key's V row in a converter thread.  Thread = key, and a swizzled row's 16-byte pieces lie at
// piece XOR key (within a 128-byte line), so eight lanes never meet in a bank, reading codes or
// writing fp16.
template <int D>
struct ValueRow {
  static constexpr int kN = D / 16;
  uint4 u[kN];
  __device__ __forceinline__ void load(const uint8_t* tile, int key) {
#pragma unroll
    for (int i = 0; i < kN; ++i)
      u[i] = *reinterpret_cast<const uint4*>(tile + Tile<kBlockKeys, D / 2>::offset(key, 8 * i));
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < kN; ++i) u[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void store(uint8_t* tile, int key) const {
    using T = Tile<kBlockKeys, D>;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      *reinterpret_cast<uint4*>(tile + T::offset(key, 16 * i)) =
          make_uint4(lo_codes(u[i].x), hi_codes(u[i].x), lo_codes(u[i].y), hi_codes(u[i].y));
      *reinterpret_cast<uint4*>(tile + T::offset(key, 16 * i + 8)) =
          make_uint4(lo_codes(u[i].z), hi_codes(u[i].z), lo_codes(u[i].w), hi_codes(u[i].w));
    }
  }
  // Multiplies a stored row by f (a block whose scale was raised).
  __device__ __forceinline__ static void scale(uint8_t* tile, int key, float f) {
#pragma unroll 1
    for (int col = 0; col < D; col += 2) {
      uint32_t& w = *reinterpret_cast<uint32_t*>(tile + Tile<kBlockKeys, D>::offset(key, col));
      const float2 x = unpack16<false>(w);
      w = pack2<false>(x.x * f, x.y * f);
    }
  }
  // Takes NaN codes out (to 0); true if there were any.
  __device__ __forceinline__ bool drop_nan() {
    bool any = false;
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      uint32_t* w[4] = {&u[i].x, &u[i].y, &u[i].z, &u[i].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t bad = __vcmpeq4(*w[e] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
        any |= bad != 0;
        *w[e] &= ~bad;
      }
    }
    return any;
  }
};

// Two float32 operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;"
      : "=l"(d)
      : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)),
        "l"(*reinterpret_cast<const uint64_t*>(&c)));
  return *reinterpret_cast<const float2*>(&d);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)));
  return *reinterpret_cast<const float2*>(&d);
}

// A row's largest x of a block, from its raw scores: their factor is uniform and not negative in a
// scale group.  kG: groups of a block that differ (1 where the cache's blocks are of 128 tokens).
template <int kG>
__device__ __forceinline__ float block_max(const float (&sv)[kBlockKeys], const Scales& sc, float mul) {
  constexpr int kW = kBlockKeys / kG;
  float mx = -INFINITY;
#pragma unroll
  for (int g = 0; g < kG; ++g) {
    float a[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int k = 0; k < kW; k += 8)
#pragma unroll
      for (int e = 0; e < 4; ++e) a[e] = fmax3(a[e], sv[kW * g + k + 2 * e], sv[kW * g + k + 2 * e + 1]);
    const float t = fmaxf(fmax3(a[0], a[1], a[2]), a[3]);
    mx = fmaxf(mx, fmaf(t, fmaxf(sc.k[g] * mul, kLeastFactor), sc.log2_v[g]));
  }
  return mx;
}

// P of the row under m into TMEM at tS (over the scores), two 16-bit values a word; returns the
// row's sum of 2^kLift P / vs.
// kPair: what the fp16 values leave, as fp16 too, goes behind them (kLowP columns on).
constexpr int kLowP = kBlockKeys / 2;
template <int kG, bool kPair>
__device__ __forceinline__ float block_probs(const float (&sv)[kBlockKeys], const Scales& sc, float mul, float m,
                                             uint32_t tS) {
  constexpr int kW = kBlockKeys / kG;
  float l = 0.0f;
  float2 sum[2];
#pragma unroll
  for (int c0 = 0; c0 < kBlockKeys; c0 += 32) {
    uint32_t pk[16], low[kPair ? 16 : 1];
#pragma unroll
    for (int k = 0; k < 32; k += 2) {
      const int key = c0 + k, g = key / kW;
      const float f = fmaxf(sc.k[g] * mul, kLeastFactor), shift = sc.log2_v[g] - m;
      if (key % kW == 0) sum[0] = sum[1] = make_float2(0.0f, 0.0f);
      const float2 x = fma2(make_float2(sv[key], sv[key + 1]), make_float2(f, f), make_float2(shift, shift));
      const float2 pr = make_float2(ex2(x.x), ex2(x.y));
      sum[(k >> 1) & 1] = add2(sum[(k >> 1) & 1], pr);
      pk[k / 2] = pack2<false>(pr.x, pr.y);
      if constexpr (kPair) {
        const float2 hi = unpack16<false>(pk[k / 2]);
        low[k / 2] = pack2<false>(pr.x - hi.x, pr.y - hi.y);
      }
      if ((key + 2) % kW == 0) {
        const float2 s = add2(sum[0], sum[1]);
        l = fmaf(s.x + s.y, sc.inv_v[g], l);
      }
    }
    tmem_st16(tS + c0 / 2, pk);
    if constexpr (kPair) tmem_st16(tS + kLowP + c0 / 2, low);
  }
  return l;
}

// For a row past kExactShift: scores that give block_probs, under m = 0, what x - m is with x rounded
// first, as the maximum was.
__device__ __forceinline__ void shift_far(float (&sv)[kBlockKeys], const Scales& sc, float mul, float m) {
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const float f = fmaxf(sc.k[g] * mul, kLeastFactor), lvs = sc.log2_v[g], back = 1.0f / f;
#pragma unroll
    for (int k = 16 * g; k < 16 * g + 16; ++k) sv[k] = (fmaf(sv[k], f, lvs) - m - lvs) * back;
  }
}

// The queries of a tile (rows of q from `q` on, `rows` of them; the tile's others are zeros) as
// 8-bit terms (the first E4M3, the others E5M2), by kN threads (tid): D / 16 lanes a row.  Row r's
// terms go to the tiles of row tile r / 128 and its factor, c2 times the power of two taken out, to
// row_mul[r].  The loop stays rolled: unrolled, fetching its instructions once a tile took longer than
// running them.
template <bool kBf16, int D, int kN>
__device__ __forceinline__ void put_queries(uint8_t* terms, float* row_mul, const uint16_t* q, int rows,
                                            int tile, float c2, int tid) {
  using C = Config<kBf16, D>;
  using T8 = typename C::T8;
  constexpr int kLanes = D / 16;
#pragma unroll 1
  for (int idx = tid; idx < tile * kLanes; idx += kN) {
    const int row = idx / kLanes, piece = idx % kLanes;
    uint4 u[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (row < rows) {
      const uint4* src = reinterpret_cast<const uint4*>(q + static_cast<int64_t>(row) * D + piece * 16);
      u[0] = __ldg(src);
      u[1] = __ldg(src + 1);
    }
    const uint32_t w[8] = {u[0].x, u[0].y, u[0].z, u[0].w, u[1].x, u[1].y, u[1].z, u[1].w};
    float x[16], amax = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 f = unpack16<kBf16>(w[e]);
      x[2 * e] = f.x, x[2 * e + 1] = f.y;
      amax = fmaxf(amax, fmaxf(finite_abs(f.x), finite_abs(f.y)));
    }
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
    const int e = scale_exp(amax, -126);
    const float mul = c2 < 0.0f ? -pow2(-e) : pow2(-e);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = nan_unless_finite(x[i]) * mul;
    uint8_t* dst = terms + row / kRows * C::kTerms * T8::kBytes + T8::offset(row % kRows, 8 * piece);
    uint32_t c[4];
    float y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = pack4_e4m3(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
      codes_to_float4(c[i], y);
#pragma unroll
      for (int k = 0; k < 4; ++k) x[4 * i + k] -= y[k];  // exact
    }
    *reinterpret_cast<uint4*>(dst) = make_uint4(c[0], c[1], c[2], c[3]);
#pragma unroll 1
    for (int term = 1; term < C::kTerms; ++term) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[i] = pack4_e5m2(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
        if (C::kTerms > 2) {  // (the last term's is not looked at)
          e5m2_to_float4(c[i], y);
#pragma unroll
          for (int k = 0; k < 4; ++k) x[4 * i + k] -= y[k];
        }
      }
      *reinterpret_cast<uint4*>(dst + term * T8::kBytes) = make_uint4(c[0], c[1], c[2], c[3]);
    }
    if (piece == 0) row_mul[row] = fabsf(c2) * pow2(e);
  }
}

template <bool kBf16, int D>
__global__ void __launch_bounds__(kThreads, 1)
    attend_tc_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const AttendParams<ByHead> p) {
  using C = Config<kBf16, D>;
  using T8 = typename C::T8;
  using TV = typename C::TV;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* sQ = smem;
  uint8_t* sK = smem + C::kOffK;
  uint8_t* sV = smem + C::kOffV;
  uint8_t* sR = smem + C::kOffR;
  Shared& sh = *reinterpret_cast<Shared*>(smem + C::kOffShared);
  const int warp = warp_id(), lane = lane_id(), group = warp >> 2;
  const ByHead& geo = p.geo;
  const bool split = geo.tile == kRows;  // the two tiles are the same rows, of alternate blocks
  grid_launch_dependents();
  if ((smem_u32(smem) & 1023u) != 0) {  // the swizzled tiles need it
    if (threadIdx.x == 0) raise_timeout(p.status, 0x20);
    return;
  }
  int u0 = 0, u1 = 0;
  Place pl{};
  if (warp == 3) {
    pl = plan_run(geo, blockIdx.x, p.ctas, p.min_chunks, u0, u1);
    if (lane == 0) sh.idle = u0 >= u1;
  }

  if (threadIdx.x == 0) {
    mbar_init(&sh.q_full, 8);
    mbar_init(&sh.q_free, 2);
    mbar_init(&sh.h_full, 4);
    mbar_init(&sh.h_free, 4);
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sh.s_full[t], 1);
      mbar_init(&sh.p_full[t], 4);
      mbar_init(&sh.o_done[t], 1);
      mbar_init(&sh.o_read[t], 4);
      mbar_init(&sh.turn[t], 4);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sh.k_full[s], 1);
      mbar_init(&sh.k_empty[s], 2);
      mbar_init(&sh.v_full[s], 4);
      mbar_init(&sh.v_empty[s], 2);
    }
    for (int s = 0; s < C::kSR; ++s) {
      mbar_init(&sh.r_full[s], 1);
      mbar_init(&sh.r_empty[s], 4);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sh.seg_full[i], 1);
      mbar_init(&sh.seg_empty[i], kSegReaders);
      mbar_init(&sh.sc_full[i], 1);
      sh.nan_seen[i] = 0;
    }
    fence_barrier_init();
  }
  constexpr uint32_t kTmem = 512;
  if (warp == 0) tmem_alloc(&sh.tmem_base, kTmem);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem_base;  // S_t (and P_t) at 128 t, O_t at 256 + D t

  // Tile number n of the run: waits until it is told, and gives its place back when done with.
  auto next_seg = [&](int n) { return mbar_wait_warp(&sh.seg_full[n & 3], (n >> 2) & 1, p.status, 0x30); };
  auto done_seg = [&](int n) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.seg_empty[n & 3]);
  };

  if (sh.idle) {
  } else if (group == 0) {
    regs_dec<kRegsIssue>();
    if (warp < 2) {
      // ------------------------------------------------------------ MMA issuer of row tile t
      const int t = warp;
      constexpr uint32_t id_s = idesc_e4m3(128, kBlockKeys), id_rest = id_s | kE5m2InA;
      constexpr uint32_t id_o = idesc_f16(128, D, 0, 0, 1);
      const uint64_t dq = T8::desc_k(smem_u32(sQ + (split ? 0 : t) * C::kTerms * T8::kBytes), 0);
      const uint64_t dk0 = T8::desc_k(smem_u32(sK), 0);
      const uint64_t dv0 = TV::desc_mn(smem_u32(sV), 0);
      const uint32_t tS = tmem + t * kBlockKeys, tO = tmem + 2 * kBlockKeys + t * D;
      uint32_t gi = 0, pph = 0;  // blocks before this tile; parity of the next p_full phase
      // Tiles in which this row tile takes no block have no o_done and o_read phases.
      uint32_t rph = 0;
      bool owed = false, ok = true;  // the tile before's O is still to be read
      for (int seg = 0;; ++seg) {
        ok = next_seg(seg);
        if (!ok) break;
        const Seg& sg = sh.seg[seg & 3];
        const int reach = sg.reach[t], steps = sg.steps, j0 = sg.j0;
        ok = mbar_wait_warp(&sh.q_full, seg & 1, p.status, 0x21);
        bool pend = false, started = false;
        for (int i = 0; i <= steps && ok; ++i) {
          const uint32_t cur_i = gi + i, prev_i = cur_i - 1;
          if (i > 0) {
            ok = mbar_wait_warp(&sh.v_full[prev_i & 1], (prev_i >> 1) & 1, p.status, 0x22);
            if (!ok) break;
          }
          const bool cur = i < steps && (split ? ((j0 + i) & 1) == t : j0 + i < reach);
          if (i < steps) {
            ok = mbar_wait_warp(&sh.k_full[cur_i & 1], (cur_i >> 1) & 1, p.status, 0x23);
            if (!ok) break;
          }
          tc_fence_after();
          if (pend) {
            ok = mbar_wait_warp(&sh.p_full[t], pph, p.status, 0x24);
            if (!ok) break;
            pph ^= 1u;
            tc_fence_after();
            const uint64_t dv = dv0 + (prev_i & 1) * static_cast<uint64_t>(TV::kBytes >> 4);
            if (elect_one()) {
#pragma unroll
              for (int kk = 0; kk < kBlockKeys / 16; ++kk)
                mma_ts(tO, tS + kk * 8, dv + TV::mn_step(kk), id_o, (started || kk > 0) ? 1u : 0u);
              if constexpr (C::kPair) {
#pragma unroll
                for (int kk = 0; kk < kBlockKeys / 16; ++kk)
                  mma_ts(tO, tS + kLowP + kk * 8, dv + TV::mn_step(kk), id_o, 1u);
              }
            }
            __syncwarp();
            started = true;
          }
          if (cur) {
            const uint64_t dk = dk0 + (cur_i & 1) * static_cast<uint64_t>(T8::kBytes >> 4);
            if (elect_one()) {
              // a step is 32 codes: 32 bytes, as 16 of the tile's 16-bit columns
#pragma unroll
              for (int term = 0; term < C::kTerms; ++term)
#pragma unroll
                for (int kk = 0; kk < D / 32; ++kk)
                  mma_ss_f8(tS, dq + term * static_cast<uint64_t>(T8::kBytes >> 4) + T8::k_step(kk),
                            dk + T8::k_step(kk), term > 0 ? id_rest : id_s, (term > 0 || kk > 0) ? 1u : 0u);
              mma_commit(&sh.s_full[t]);
            }
            __syncwarp();
          }
          if (i + 1 == steps && owed) {
            // Q is released for the next tile only when this row tile's last O has been read, so
            // what softmax holds by tile number stays at most two tiles behind the converters.
            ok = mbar_wait_warp(&sh.o_read[t], rph, p.status, 0x25);
            if (!ok) break;
            rph ^= 1u;
            owed = false;
          }
          if (elect_one()) {
            if (i < steps) mma_commit(&sh.k_empty[cur_i & 1]);
            if (i + 1 == steps) mma_commit(&sh.q_free);
            if (i > 0) mma_commit(&sh.v_empty[prev_i & 1]);
          }
          __syncwarp();
          pend = cur;
        }
        if (!ok) break;
        if (started) {
          if (elect_one()) mma_commit(&sh.o_done[t]);
          __syncwarp();
          owed = true;
        }
        gi += steps;
        const bool last = sg.last;
        done_seg(seg);
        if (last) break;
      }
    } else if (warp == 2) {
      // ------------------------------------------------------------ TMA producer
      const int nblk = geo.cap / p.block;
      uint32_t gi = 0;
      bool ok = true;
      for (int seg = 0;; ++seg) {
        ok = next_seg(seg);
        if (!ok) break;
        const Seg& sg = sh.seg[seg & 3];
        const int bh = sg.b * geo.Hk + sg.hk, steps = sg.steps, j0 = sg.j0, len = sg.len;
        const float* ksp = p.k_scales + static_cast<int64_t>(bh) * nblk;
        const float* vsp = p.v_scales + static_cast<int64_t>(bh) * nblk;
        // A block's scales, one lane to 16 keys, fetched a block ahead.  Their place's last readers
        // were softmax and the converters four blocks ago; the scores of two blocks ago (k_empty) came
        // after P V of those.
        float ks, vs;
        auto fetch = [&](int i) {
          const int key = (j0 + i) * kBlockKeys + lane * 16;
          const bool in = lane < kGroups && key < len;
          ks = in ? __ldg(ksp + key / p.block) : 1.0f;
          vs = in ? __ldg(vsp + key / p.block) : 1.0f;
        };
        fetch(0);
        int hi = -200;  // exponent of the tile's largest V scale so far
        for (int i = 0; i < steps && ok; ++i) {
          const uint32_t c = gi + i, rs = c % C::kSR;
          const int key0 = (j0 + i) * kBlockKeys;
          ok = mbar_wait_warp(&sh.k_empty[c & 1], ((c >> 1) & 1) ^ 1, p.status, 0x27);
          if (!ok) break;
          if (lane == 0) {  // rows past the cache read as zeros
            mbar_arrive_expect_tx(&sh.k_full[c & 1], T8::kBytes);
            tma_load_3d(sK + (c & 1) * T8::kBytes, &tm_k, &sh.k_full[c & 1], 0, key0, bh);
          }
          const int e = static_cast<int>(__float_as_uint(vs) >> 23) - 127;
          const bool in = lane < kGroups && key0 + lane * 16 < len;
          hi = max(hi, __reduce_max_sync(0xFFFFFFFFu, in ? e : -200));
          const int floor = max(static_cast<int>(kLeastScale), hi - static_cast<int>(kScaleSpan));
          const bool raised = __any_sync(0xFFFFFFFFu, in && e < floor);
          int rest = 0;  // whole powers of two, so the values stay exact down to fp16's subnormals
          if (in && e < floor) {
            rest = max(e - floor, -126);
            vs *= pow2(-rest);
          }
          if (lane < kGroups) {
            Scales& sc = sh.scales[c & 3];
            sc.k[lane] = ks;
            sc.log2_v[lane] = log2f(vs);
            sc.inv_v[lane] = kLiftFactor / vs;
            sc.rest[lane] = static_cast<int8_t>(rest);
            if (lane == 0) sc.raised = raised;
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.sc_full[c & 3]);  // (the converters are told by r_full)
          ok = mbar_wait_warp(&sh.r_empty[rs], ((c / C::kSR) & 1) ^ 1, p.status, 0x28);
          if (!ok) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(&sh.r_full[rs], C::kRaw);
            tma_load_3d(sR + rs * C::kRaw, &tm_v, &sh.r_full[rs], 0, key0, bh);
          }
          __syncwarp();
          if (i + 1 < steps) fetch(i + 1);
        }
        if (!ok) break;
        gi += steps;
        const bool last = sg.last;
        done_seg(seg);
        if (last) break;
      }
    } else if (warp == 3) {
      // ------------------------------------------------------------ the run's tiles
      for (int seg = 0;; ++seg) {
        if (!mbar_wait_warp(&sh.seg_empty[seg & 3], ((seg >> 2) & 1) ^ 1, p.status, 0x31)) break;
        const Seg sg = segment(geo, pl, u0, u1, blockIdx.x);
        if (lane == 0) {
          sh.seg[seg & 3] = sg;
          if (sg.j0 == 0) note_run(p, pl, u0, u1);
          mbar_arrive(&sh.seg_full[seg & 3]);
        }
        __syncwarp();
        if (sg.last) break;
        next_place(geo, pl);
      }
    }
  } else if (group == 3) {
    // ---------------------------------------------------------------- converters
    regs_dec<kRegsConvert>();
    const int tid = threadIdx.x - 3 * 128;
    uint32_t gi = 0;
    for (int seg = 0;; ++seg) {
      bool ok = next_seg(seg);
      if (!ok) break;
      const Seg& sg = sh.seg[seg & 3];
      const int steps = sg.steps, j0 = sg.j0, len = sg.len, least = min(sg.least[0], sg.least[1]);
      // Block i + 1's codes are read from their stage while block i's tile is being written.
      ValueRow<D> x;
      auto take = [&](int i) -> bool {
        const uint32_t c = gi + i, rs = c % C::kSR;
        if (!mbar_wait_warp(&sh.r_full[rs], (c / C::kSR) & 1, p.status, 0x2B)) return false;
        x.load(sR + rs * C::kRaw, tid);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.r_empty[rs]);
        return true;
      };
      ok = take(0);
      for (int i = 0; i < steps && ok; ++i) {
        const uint32_t c = gi + i;
        const int key0 = (j0 + i) * kBlockKeys;
        const bool raised = sh.scales[c & 3].raised;  // there since r_full
        ok = mbar_wait_warp(&sh.v_empty[c & 1], ((c >> 1) & 1) ^ 1, p.status, 0x2C);
        if (!ok) break;
        if (key0 + kBlockKeys > least) {
          if (key0 + tid >= len) x.clear();
          if (x.drop_nan()) atomicOr(&sh.nan_seen[seg & 3], 1u);
        }
        x.store(sV + (c & 1) * TV::kBytes, tid);
        if (__builtin_expect(raised, 0)) x.scale(sV + (c & 1) * TV::kBytes, tid, pow2(sh.scales[c & 3].rest[tid / 16]));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.v_full[c & 1]);
        if (i + 1 < steps) ok = take(i + 1);
      }
      if (!ok) break;
      gi += steps;
      const bool last = sg.last;
      done_seg(seg);
      if (last) break;
    }
  } else {
    // ---------------------------------------------------------------- softmax of row tile t
    regs_inc<kRegsSoftmax>();
    const int t = group - 1, quad = warp & 3, r = quad * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t tS = tmem + t * kBlockKeys + lane_off, tO = tmem + 2 * kBlockKeys + t * D + lane_off;
    const bool uniform = p.block >= kBlockKeys;  // one scale a block of keys
    uint32_t gi = 0, s_phase = 0, o_phase = 0, h_phase = 0, turn_phase = 0;
    bool ok = true;
    for (int seg = 0;; ++seg) {
      ok = next_seg(seg);
      if (!ok) break;
      const Seg& sg = sh.seg[seg & 3];
      const int row = sg.r0 + (split ? 0 : t * kRows) + r;
      const int query = geo.query(row < geo.R ? row : 0);
      const bool real = row < geo.R && query < sg.cnt;
      const int lim = real ? query_keys(geo, sg.len, sg.cnt, query) : sg.len;
      const int reach = sg.reach[t], least = sg.least[t], j0 = sg.j0;
      // The tile's blocks: all up to its reach, or every other one.
      const int steps = min(sg.steps, reach - j0);
      const int i0 = split ? (j0 + t) & 1 : 0, stride = split ? 2 : 1;
      const bool have = i0 < steps;
      // Two row tiles' exponentials take turns in the blocks that both take: in step they would share
      // the exponential units and then wait for the tensor core together (2048 rows of 32768 keys, 8
      // heads: 254 us without turns, 223 with).  Tiles of alternate blocks are out of step already
      // (77 us without, 79 with, on 48 rows).
      const int both = split ? 0 : min(sg.steps, min(sg.reach[0], sg.reach[1]) - j0);
      float m = kNoMax, l = 0.0f, mul = 0.0f;  // mul: |c| log2(e) times the row's power of two
      ok = seg == 0 || mbar_wait_warp(&sh.q_free, (seg - 1) & 1, p.status, 0x26);
      if (!ok) break;
      if (t == 0 && r == 0) sh.nan_seen[(seg + 2) & 3] = 0;  // read last two tiles ago
      put_queries<kBf16, D, 2 * kRows>(sQ, sh.row_mul[seg & 1], p.q + geo.row_offset(sg.b, sg.hk, sg.r0) * D,
                            geo.R - sg.r0, geo.tile, p.c2, t * kRows + r);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_full);

      for (int i = i0; i < steps; i += stride) {
        const uint32_t c = gi + i;
        ok = mbar_wait_warp(&sh.sc_full[c & 3], (c >> 2) & 1, p.status, 0x2D) &&
             mbar_wait_warp(&sh.s_full[t], s_phase, p.status, 0x29);
        if (!ok) break;
        s_phase ^= 1u;
        tc_fence_after();
        if (i == i0) mul = sh.row_mul[seg & 1][row - sg.r0];
        const Scales& sc = sh.scales[c & 3];
        const int key0 = (j0 + i) * kBlockKeys;
        float sv[kBlockKeys];
        {
          uint32_t rr[kBlockKeys];
#pragma unroll
          for (int c0 = 0; c0 < kBlockKeys; c0 += 32)
            tmem_ld32(tS + c0, *reinterpret_cast<uint32_t(*)[32]>(rr + c0));
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < kBlockKeys; ++k) sv[k] = __uint_as_float(rr[k]);
        }
        if (__builtin_expect(key0 + kBlockKeys > least, 0)) {
          const int seen = lim - key0;
#pragma unroll
          for (int k = 0; k < kBlockKeys; ++k)
            if (k >= seen) sv[k] = -INFINITY;
        }
        const float mx = uniform ? block_max<1>(sv, sc, mul) : block_max<kGroups>(sv, sc, mul);
        float alpha = 1.0f;
        if (mx - m > kRaise) {
          const float mn = mx - kTop, half = ex2(0.5f * (m - mn));
          alpha = half * half;
          m = mn;
          l = l * half * half;
        }
        // Seldom both: in one branch, and far rows change their scores there, so that the common blocks
        // pay little (a second way through the exponentials cost 2048 rows 7 us of 221, 48 rows 3 of 79).
        const bool far = real && fabsf(m) > kExactShift && m != kNoMax;
        if (__builtin_expect(__any_sync(0xFFFFFFFFu, alpha != 1.0f || far), 0)) {
#pragma unroll 1
          for (int c0 = i == i0 ? D : 0; c0 < D; c0 += 16) {  // no O yet at the first block
            uint32_t rr[16];
            tmem_ld16(tO + c0, rr);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 16; ++k) rr[k] = __float_as_uint(__uint_as_float(rr[k]) * alpha);
            tmem_st16(tO + c0, rr);
          }
          if (far) shift_far(sv, sc, mul, m);
        }
        if (i < both && (t == 1 || i > 0)) {
          ok = mbar_wait_warp(&sh.turn[t], turn_phase, p.status, 0x3A);
          if (!ok) break;
          turn_phase ^= 1u;
        }
        const float from = far ? 0.0f : m;
        l += uniform ? block_probs<1, C::kPair>(sv, sc, mul, from, tS)
                     : block_probs<kGroups, C::kPair>(sv, sc, mul, from, tS);
        __syncwarp();
        if (lane == 0 && i + t < both) mbar_arrive(&sh.turn[t ^ 1]);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[t]);
      }
      if (!ok) break;
      if (have) {
        ok = mbar_wait_warp(&sh.o_done[t], o_phase, p.status, 0x2A);
        if (!ok) break;
        o_phase ^= 1u;
        tc_fence_after();
      }
      const bool handed = split && ((sg.j0 + 1) & 1) < sg.steps;  // tile 1 has a state to hand over
      float4* hand_z = reinterpret_cast<float4*>(
          p.part_z + (static_cast<int64_t>(2 * p.ctas + blockIdx.x) * kRows) * D) + r;
      float2* hand_lm = reinterpret_cast<float2*>(p.part_lm) + static_cast<int64_t>(2 * p.ctas + blockIdx.x) * kRows + r;
      if (split && t == 1) {
        if (have) {
          ok = mbar_wait_warp(&sh.h_free, h_phase ^ 1u, p.status, 0x2E);
          if (!ok) break;
          h_phase ^= 1u;
#pragma unroll 1
          for (int c0 = 0; c0 < D; c0 += 32) {
            uint32_t rr[32];
            tmem_ld32(tO + c0, rr);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              hand_z[(c0 + k) / 4 * kRows] = make_float4(__uint_as_float(rr[k]), __uint_as_float(rr[k + 1]),
                                                         __uint_as_float(rr[k + 2]), __uint_as_float(rr[k + 3]));
          }
          *hand_lm = make_float2(l, m);
          tc_fence_before();
          __threadfence_block();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sh.h_full);
            mbar_arrive(&sh.o_read[t]);
          }
        }
      } else {
        float f0 = 1.0f, f1 = 0.0f;  // factors of this tile's z and of the one handed over
        if (handed) {
          ok = mbar_wait_warp(&sh.h_full, h_phase, p.status, 0x2F);
          if (!ok) break;
          h_phase ^= 1u;
          const float2 lm = __ldcg(hand_lm);
          const float mx = fmaxf(m, lm.y);
          const float h0 = ex2(0.5f * (m - mx)), h1 = ex2(0.5f * (lm.y - mx));
          f0 = h0 * h0;
          f1 = h1 * h1;
          l = l * h0 * h0 + lm.x * h1 * h1;
          m = mx;
        }
        // A masked block's V held NaN codes, which were kept out of the product: the columns of
        // the keys this row sees are NaN.
        uint32_t bad[D / 32];
#pragma unroll
        for (int i = 0; i < D / 32; ++i) bad[i] = 0;
        if (__builtin_expect((have || handed) && sh.nan_seen[seg & 3] != 0, 0)) {
          const int all = min(sg.least[0], sg.least[1]);
          const int k0 = max(all / kBlockKeys, sg.j0) * kBlockKeys;
          const int k1 = min(lim, (sg.j0 + sg.steps) * kBlockKeys);
          const uint32_t* vw = reinterpret_cast<const uint32_t*>(
              p.v8 + ((static_cast<int64_t>(sg.b) * geo.Hk + sg.hk) * geo.cap) * D);
          for (int key = k0; key < k1; ++key)
            for (int w = 0; w < D / 4; ++w) {
              const uint32_t x = __ldg(vw + static_cast<int64_t>(key) * (D / 4) + w);
              const uint32_t eq = __vcmpeq4(x & 0x7F7F7F7Fu, 0x7F7F7F7Fu) & 0x08040201u;
              const uint32_t bits = ((eq | eq >> 8 | eq >> 16 | eq >> 24) & 0xFu) << (4 * (w % 8));
#pragma unroll
              for (int i = 0; i < D / 32; ++i)
                if (i == w / 8) bad[i] |= bits;
            }
        }
        const bool write = row < geo.R;
        const bool none = l == 0.0f || !real;  // a padding row, or one that sees no key
        const float inv = kLiftFactor / l;
        const int64_t orow = geo.row_offset(sg.b, sg.hk, row);
        const int64_t prow = static_cast<int64_t>(sg.slot) * geo.tile + (row - sg.r0);
#pragma unroll 1
        for (int c0 = 0; c0 < D; c0 += 32) {
          uint32_t rr[32];
          __syncwarp();
          if (have) {
            tmem_ld32(tO + c0, rr);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int k = 0; k < 32; ++k) rr[k] = 0u;
          }
          if (handed) {
#pragma unroll
            for (int k = 0; k < 32; k += 4) {
              const float4 h = __ldcg(hand_z + (c0 + k) / 4 * kRows);
              rr[k] = __float_as_uint(fmaf(__uint_as_float(rr[k]), f0, h.x * f1));
              rr[k + 1] = __float_as_uint(fmaf(__uint_as_float(rr[k + 1]), f0, h.y * f1));
              rr[k + 2] = __float_as_uint(fmaf(__uint_as_float(rr[k + 2]), f0, h.z * f1));
              rr[k + 3] = __float_as_uint(fmaf(__uint_as_float(rr[k + 3]), f0, h.w * f1));
            }
          }
          uint32_t nan = 0;
#pragma unroll
          for (int i = 0; i < D / 32; ++i)
            if (i == c0 / 32) nan = bad[i];
          if (nan) {
#pragma unroll
            for (int k = 0; k < 32; ++k)
              if (nan >> k & 1u) rr[k] = 0x7FC00000u;
          }
          if (write && sg.whole) {
            uint4 w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t h[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                h[i] = none ? 0u : pack2<kBf16>(__uint_as_float(rr[8 * k + 2 * i]) * inv,
                                                __uint_as_float(rr[8 * k + 2 * i + 1]) * inv);
              w[k] = make_uint4(h[0], h[1], h[2], h[3]);
              *reinterpret_cast<uint4*>(p.o + orow * D + c0 + 8 * k) = w[k];
            }
          } else if (write) {
#pragma unroll
            for (int k = 0; k < 32; k += 4)
              *reinterpret_cast<float4*>(p.part_z + prow * D + c0 + k) =
                  make_float4(__uint_as_float(rr[k]), __uint_as_float(rr[k + 1]), __uint_as_float(rr[k + 2]),
                              __uint_as_float(rr[k + 3]));
          }
        }
        if (write && sg.whole) {
          p.lse[orow] = none ? -INFINITY : row_lse(l, m);
          if (none && real) raise_empty_row(p.status);
        }
        if (write && !sg.whole) *reinterpret_cast<float2*>(p.part_lm + prow * 2) = make_float2(l, m);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (have) mbar_arrive(&sh.o_read[t]);
          if (handed) mbar_arrive(&sh.h_free);
        }
      }
      gi += sg.steps;
      const bool last = sg.last;
      done_seg(seg);
      if (last) break;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmem);
  }
}

}  // namespace tc
}  // namespace kv8

template <bool kBf16, int D>
cudaError_t launch_kv8_tc(kv8::AttendParams<kv8::ByHead>& p, cudaStream_t s) {
  using C = kv8::tc::Config<kBf16, D>;
  auto* kernel = kv8::tc::attend_tc_kernel<kBf16, D>;
  constexpr size_t smem = C::kOffShared + sizeof(kv8::tc::Shared);
  static_assert(smem <= 227 * 1024, "shared memory overflow");
  CUtensorMap tm_k, tm_v;
  const uint64_t heads = static_cast<uint64_t>(p.geo.B) * p.geo.Hk;
  if (!encode_byte_map(&tm_k, p.k8, heads, p.geo.cap, D, kv8::kBlockKeys, D) ||
      !encode_byte_map(&tm_v, p.v8, heads, p.geo.cap, D, kv8::kBlockKeys, D))
    return cudaErrorInvalidValue;
  // The registers dealt inside the kernel are those it is launched with: were a compiler to give
  // it fewer, the warpgroups that ask for more would wait for ever.
  static const int regs = [&] {
    cudaFuncAttributes attr;
    return cudaFuncGetAttributes(&attr, kernel) == cudaSuccess ? attr.numRegs : 0;
  }();
  if (4 * regs < kv8::tc::kRegsIssue + 2 * kv8::tc::kRegsSoftmax + kv8::tc::kRegsConvert)
    return cudaErrorInvalidConfiguration;
  static std::atomic<uint64_t> allowed{0};
  cudaError_t e = kv8::allow_smem(reinterpret_cast<const void*>(kernel), smem, allowed);
  if (e != cudaSuccess) return e;
  void* args[] = {&tm_k, &tm_v, &p};
  e = cudaLaunchKernel(reinterpret_cast<const void*>(kernel), dim3(p.ctas), dim3(kv8::tc::kThreads), args,
                       smem, s);
  if (e != cudaSuccess) return e;
  return kv8::launch_join<kBf16, D>(p, s);
}

}  // namespace ea
