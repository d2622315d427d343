// Which drafted tokens of a tree the target's probabilities accept, and the token after them.
//
// At a node with p and q the target's and the draft's probabilities after it, the children are asked
// in order.  Children drawn from q: child x_k is accepted with probability min(1, r_k(x) / q(x)), and
// a refusal leaves the residual r_{k+1} = max(r_k - q, 0) over its mass, r_0 = p.  Kept without the
// division, t_k = W_k r_k with W_k its mass, the steps fold into one number:
//     t_{k+1} = max(t_k - W_k q, 0) = max(p - S q, 0),   S = W_0 + .. + W_k,  W_0 = 1
// (where t_k is 0, p <= S q holds already for the smaller S).  So x is accepted iff
//     u q(x) W < max(p(x) - S q(x), 0),
// and a refusal costs one sum over the vocabulary, of t, which is also what the last token is
// drawn from: the least v whose cumulative t passes u_0 times the sum.  Children that were not drawn
// have q(x) = 1 at their own token: accepted iff u W < t(x), else t(x) = 0 and W loses it; no sum.
//
// A cluster of CTAs takes a sequence.  Its first CTA gathers the nodes' few probabilities and walks
// the tree; the others only follow its commands (so that all take the same way whatever the inputs
// do meanwhile): sum the masses at a node, each warp a contiguous share of the vocabulary.  After
// the last sum every CTA looks for the share that the drawn number falls in, and the one that has it
// for the token.
//
// The device has two 64-bit units a multiprocessor, and a dependent 64-bit step of a warp takes about a
// hundred cycles: walk, sums and scans in 64 bits took 37 us where these take 24 (32 trees of 32 nodes over
// 131072 values).  So sums are pairs of float32 values, by Knuth's and Dekker's error-free sums and products,
// two elements an instruction, and a child's test is float32 unless its sides lie within 10^-6.  Of a row of
// mass 1 the pairs' second values round off at most 2^-42 + V 2^-48: an element's two additions 2^-49 while its
// accumulator holds less than 2^-5, and 2^-44 of what it holds beyond that, so 2^-48 together (Sum); fifteen
// additions of pairs above one another 1.5 2^-47 each.
#include <cooperative_groups.h>

#include <type_traits>
#include <utility>

#include "draft.h"
#include "kv8_common.cuh"

namespace ea {
namespace draft {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMostRanks = 8;  // CTAs of a cluster (the portable size)

struct VerifyParams {
  int n, V;
  const void* target;
  const void* draft;
  const int32_t* tokens;
  const int32_t* parents;
  const int32_t* counts;
  const float* uniforms;
  int32_t* path;
  int32_t* accepted;
  int32_t* next_token;
  uint32_t* status;
};

struct Command {  // of the first CTA to all
  bool done;      // nothing more to do
  bool refusing;  // the sum is a refusal's: it counts only if it is not 0
  bool last;      // no child is left: the token is drawn from the sum's shares
  int node;
  int refused;  // tokens taken out of the target's probabilities (drafts that were not drawn)
  float2 S;     // (as a Pair)
};

struct Shared {
  Command cmd;
  float2 mass[kMostRanks * kWarps];  // of each warp's share (first CTA; all of them for the last sum)
  float2 tile[kWarps];
  float2 goal, below;                // drawing the token: what the cumulative sum has to pass, and
  int from;                          // the warp whose share it passes it in, with the sum before that
  float p[kMostNodes], q[kMostNodes], u[kMostNodes];
  int up[kMostNodes], token[kMostNodes];
  int refused[kMostNodes];
};

// A value as the unevaluated sum of two float32 values.  (Explicit roundings: a product and a sum made
// one by the compiler would no longer be error-free.)
struct Pair {
  float hi, lo;
  __device__ __forceinline__ Pair() : hi(0.0f), lo(0.0f) {}
  __device__ __forceinline__ Pair(float h, float l) : hi(h), lo(l) {}
  __device__ __forceinline__ explicit Pair(float2 x) : hi(x.x), lo(x.y) {}
  __device__ __forceinline__ float2 raw() const { return make_float2(hi, lo); }
  __device__ __forceinline__ double value() const { return static_cast<double>(hi) + static_cast<double>(lo); }
  __device__ __forceinline__ bool positive() const { return hi > 0.0f; }
};
__device__ __forceinline__ Pair norm(Pair x) {  // |lo| at most half of hi's last place
  const float s = __fadd_rn(x.hi, x.lo);
  return {s, __fsub_rn(x.lo, __fsub_rn(s, x.hi))};
}
__device__ __forceinline__ Pair operator+(Pair a, Pair x) {
  const float s = __fadd_rn(a.hi, x.hi), b = __fsub_rn(s, a.hi);
  const float e = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, b)), __fsub_rn(x.hi, b));
  return norm({s, __fadd_rn(__fadd_rn(a.lo, x.lo), e)});
}
__device__ __forceinline__ Pair operator*(float u, Pair x) {
  const float h = __fmul_rn(u, x.hi);
  return norm({h, fmaf(u, x.lo, fmaf(u, x.hi, -h))});
}
__device__ __forceinline__ bool operator>(Pair a, Pair b) { return a.hi > b.hi || (a.hi == b.hi && a.lo > b.lo); }
__device__ __forceinline__ Pair shfl(Pair x, int lane) {
  return {__shfl_sync(0xFFFFFFFFu, x.hi, lane), __shfl_sync(0xFFFFFFFFu, x.lo, lane)};
}
__device__ __forceinline__ Pair shfl_up(Pair x, int by) {
  return {__shfl_up_sync(0xFFFFFFFFu, x.hi, by), __shfl_up_sync(0xFFFFFFFFu, x.lo, by)};
}
// A warp's inclusive sums of x over its lanes.
__device__ __forceinline__ Pair scan(Pair x) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Pair y = shfl_up(x, o);
    if (static_cast<int>(lane_id()) >= o) x = y + x;
  }
  return x;
}

// Two elements at once.
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
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;"
      : "=l"(d)
      : "l"(*reinterpret_cast<const uint64_t*>(&a)), "l"(*reinterpret_cast<const uint64_t*>(&b)));
  return *reinterpret_cast<const float2*>(&d);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return fma2(b, both(-1.0f), a); }  // (one rounding)

__device__ __forceinline__ float2 max2(float2 a, float2 b) { return make_float2(fmaxf(a.x, b.x), fmaxf(a.y, b.y)); }

struct Pair2 {
  float2 hi, lo;
};
// Which residual: the probabilities themselves (S = 0), after a first refusal (S = 1), or after more.
enum Kind : int { kAll, kFirst, kMore };
__device__ __forceinline__ Kind kind_of(Pair S) { return S.hi == 0.0f ? kAll : S.hi == 1.0f && S.lo == 0.0f ? kFirst : kMore; }
// max(p - S q, 0) of two elements, as pairs.  After one refusal, with m = max(p, q) and d = m - q rounded, what
// d leaves is (m - d) - q, exactly, as m >= q.  After more, h = S q is rounded too, and where p lies within a
// few of its last places all that is left may be in what was rounded off: so x = (p - d) - h + (h - S q) joins
// d = p - h before the sign is looked at.  (p - d) - h is exact where p >= h / 2, below that d is negative
// by far more than x; the roundings of x come to 2^-45 of p.
template <int kKind>
__device__ __forceinline__ Pair2 residual(float2 p, float2 q, Pair S) {
  if (kKind == kAll) return {p, both(0.0f)};
  if (kKind == kFirst) {
    const float2 m = max2(p, q), d = sub2(m, q);
    return {d, sub2(sub2(m, d), q)};
  }
  const float2 h = mul2(both(S.hi), q), d = sub2(p, h);
  const float2 x = add2(sub2(sub2(p, d), h), fma2(both(-S.lo), q, fma2(both(-S.hi), q, h)));
  const float2 t = add2(d, x), lo = sub2(x, sub2(t, d));
  return {max2(t, both(0.0f)), make_float2(t.x > 0.0f ? lo.x : 0.0f, t.y > 0.0f ? lo.y : 0.0f)};
}
__device__ __forceinline__ Pair2 residual(float2 p, float2 q, Pair S) {
  const Kind k = kind_of(S);
  return k == kAll ? residual<kAll>(p, q, S) : k == kFirst ? residual<kFirst>(p, q, S) : residual<kMore>(p, q, S);
}

// A sum of nonnegative values.  It starts at kFrom, so that the sum is never below a value of at most kFrom
// and what an addition rounds off comes out of two more (of any value: five).  settle() keeps what was rounded
// off below a last place of the sum: left alone it would grow with a row's length, and be rounded ever more
// coarsely (2^26 equal values: 2^-20 of the mass).
struct Sum {
  static constexpr float kFrom = 1.0f / 64.0f;
  Pair2 x{both(kFrom), both(0.0f)};
  template <bool kSmall>  // values of at most kFrom
  __device__ __forceinline__ void add(const Pair2& v) {
    const float2 s = add2(x.hi, v.hi), b = sub2(s, x.hi);
    const float2 e = kSmall ? sub2(v.hi, b) : add2(sub2(x.hi, sub2(s, b)), sub2(v.hi, b));
    x.lo = add2(add2(x.lo, v.lo), e);
    x.hi = s;
  }
  __device__ __forceinline__ void settle() {
    const float2 s = add2(x.hi, x.lo);
    x.lo = sub2(x.lo, sub2(s, x.hi));
    x.hi = s;
  }
  __device__ __forceinline__ Pair total() const {
    return Pair{__fsub_rn(x.hi.x, kFrom), x.lo.x} + Pair{__fsub_rn(x.hi.y, kFrom), x.lo.y};
  }
};

// A probability as it counts: NaN as 0, and within [0, 1].
__device__ __forceinline__ float prob(float x) { return __saturatef(x); }
template <int kType>
__device__ __forceinline__ float load_prob(const void* x, int64_t i) {
  if constexpr (kType == kProbF32) {
    return prob(__ldg(static_cast<const float*>(x) + i));
  } else {
    const uint32_t w = __ldg(static_cast<const uint16_t*>(x) + i);
    return prob(kv8::unpack16<kType == kProbBf16>(w).x);
  }
}

// 16 bytes of probabilities as they lie in memory.
template <int kType>
struct Vec {
  static constexpr int kN = kType == kProbF32 ? 4 : 8;
  using Word = std::conditional_t<kType == kProbF32, uint32_t, uint16_t>;
  uint4 w;
  __device__ __forceinline__ void load(const void* row, int v) {
    w = __ldg(reinterpret_cast<const uint4*>(static_cast<const Word*>(row) + v));
  }
  // The same at the row's ends: what lies outside [0, V) is 0.
  __device__ __forceinline__ void load_edge(const void* row, int v, int V) {
    uint32_t c[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (v + i >= 0 && v + i < V)
        c[i * 4 / kN] |= static_cast<uint32_t>(__ldg(static_cast<const Word*>(row) + v + i)) << (kN == 4 ? 0 : 16 * (i & 1));
    w = make_uint4(c[0], c[1], c[2], c[3]);
  }
  // The largest value's bits: a probability's are at most kOne; negative values' and NaN's are more.
  __device__ __forceinline__ uint32_t most() const {
    if constexpr (kType == kProbF32) {
      return max(max(w.x, w.y), max(w.z, w.w));
    } else {
      const uint32_t m = __vmaxu2(__vmaxu2(w.x, w.y), __vmaxu2(w.z, w.w));
      return max(m >> 16, m & 0xFFFFu);
    }
  }
  // Bits of 1 and of Sum::kFrom = 2^-6.
  static constexpr uint32_t kOne = kType == kProbF32 ? 0x3F800000u : kType == kProbBf16 ? 0x3F80u : 0x3C00u;
  static constexpr uint32_t kFrom = kType == kProbF32 ? 0x3C800000u : kType == kProbBf16 ? 0x3C80u : 0x2400u;
  // Elements 2i and 2i + 1, as they count if kClamp.
  template <bool kClamp>
  __device__ __forceinline__ float2 values(int i) const {
    const uint32_t c[4] = {w.x, w.y, w.z, w.w};
    const float2 f = kType == kProbF32 ? make_float2(__uint_as_float(c[2 * i & 3]), __uint_as_float(c[(2 * i + 1) & 3]))
                                       : kv8::unpack16<kType == kProbBf16>(c[i & 3]);
    return kClamp ? make_float2(prob(f.x), prob(f.y)) : f;
  }
};

// A warp's share of the vocabulary, in tiles of 32 vectors of 16 bytes.
template <int kType, bool kDrawn>
struct Share {
  static constexpr int kN = Vec<kType>::kN, kTile = 32 * kN;
  const typename Vec<kType>::Word* target;  // the node's rows
  const typename Vec<kType>::Word* draft;   // null where S is 0
  int V;
  int v0, v1;  // vectors start at 16-byte boundaries, so the first may lie before 0, and the last past V
  Pair S;
  const int* refused;  // tokens to be taken out
  int refusals;
  int mine;  // the lane's of them, if they are at most 32

  __device__ __forceinline__ Share(const VerifyParams& p, int b, const Command& c, const int* list, int warp, int warps)
      : V(p.V), S(c.S), refused(list) {
    const int64_t row = (static_cast<int64_t>(b) * p.n + c.node) * V;
    target = static_cast<const typename Vec<kType>::Word*>(p.target) + row;
    const int before = static_cast<int>(row & (kN - 1));  // elements past a 16-byte boundary
    const int tiles = (V + before + kTile - 1) / kTile, per = (tiles + warps - 1) / warps;
    v0 = min(warp * per, tiles) * kTile - before;
    v1 = min((warp + 1) * per, tiles) * kTile - before;
    draft = kDrawn && S.hi != 0.0f ? static_cast<const typename Vec<kType>::Word*>(p.draft) + row : nullptr;
    refusals = kDrawn ? 0 : c.refused;
    mine = static_cast<int>(lane_id()) < refusals ? list[lane_id()] : -1;
  }
  __device__ __forceinline__ bool inside(int v, int tiles) const { return v >= 0 && v + tiles * kTile <= V; }
  // The vectors at v: of a tile inside the row, and of one that reaches past its ends.
  template <bool kBoth>
  __device__ __forceinline__ void load(int v, Vec<kType>& t, Vec<kType>& q) const {
    t.load(target, v);
    q.w = make_uint4(0u, 0u, 0u, 0u);
    if (kBoth) q.load(draft, v);
  }
  template <bool kBoth>
  __device__ __forceinline__ void load_edge(int v, Vec<kType>& t, Vec<kType>& q) const {
    t.load_edge(target, v, V);
    q.w = make_uint4(0u, 0u, 0u, 0u);
    if (kBoth) q.load_edge(draft, v, V);
  }
  // The residuals of the vectors at v, whatever they hold.
  __device__ __forceinline__ void terms(int v, const Vec<kType>& t, const Vec<kType>& q, Pair2 (&r)[kN / 2]) const {
#pragma unroll
    for (int i = 0; i < kN / 2; ++i) {
      const float2 p = t.template values<true>(i);
      r[i] = kDrawn ? residual(p, q.template values<true>(i), S) : Pair2{p, both(0.0f)};
    }
    if constexpr (!kDrawn) {
      for (int k = 0; k < refusals; ++k) {
        const int at = refused[k] - v;
#pragma unroll
        for (int i = 0; i < kN / 2; ++i) {
          if (at == 2 * i) r[i].hi.x = 0.0f;
          if (at == 2 * i + 1) r[i].hi.y = 0.0f;
        }
      }
    }
  }
  // Adds them to a sum, by the whole warp, for the tile at v0: most tiles hold nothing but small
  // probabilities, and no refused token.
  template <int kKind>
  __device__ __forceinline__ void add_to(Sum& sum, int v0, const Vec<kType>& t, const Vec<kType>& q) const {
    const int v = v0 + static_cast<int>(lane_id()) * kN;
    bool odd = t.most() > Vec<kType>::kFrom || (kKind != kAll && q.most() > Vec<kType>::kOne);
    if (!kDrawn) odd |= refusals > 32 || (mine >= v0 && mine < v0 + kTile);
    if (__builtin_expect(__any_sync(0xFFFFFFFFu, odd), 0)) {
      Pair2 r[kN / 2];
      terms(v, t, q, r);
#pragma unroll
      for (int i = 0; i < kN / 2; ++i) sum.template add<false>(r[i]);
      return;
    }
#pragma unroll
    for (int i = 0; i < kN / 2; ++i)
      sum.template add<true>(residual<kKind>(t.template values<false>(i), q.template values<false>(i), S));
  }
};

// The mass of the warp's share (in lane 31).
template <int kKind, int kType, bool kDrawn>
__device__ __forceinline__ Pair share_mass_of(const Share<kType, kDrawn>& s) {
  using S = Share<kType, kDrawn>;
  constexpr int kAhead = kKind == kAll ? 4 : 2;  // tiles whose loads are in flight together
  const int mine = static_cast<int>(lane_id()) * S::kN;
  Sum sum;
  for (int v = s.v0; v < s.v1;) {
    Vec<kType> t[kAhead], q[kAhead];
    if (v + kAhead * S::kTile <= s.v1 && s.inside(v, kAhead)) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) s.template load<kKind != kAll>(v + i * S::kTile + mine, t[i], q[i]);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) s.template add_to<kKind>(sum, v + i * S::kTile, t[i], q[i]);
      v += kAhead * S::kTile;
    } else {
      if (s.inside(v, 1)) {
        s.template load<kKind != kAll>(v + mine, t[0], q[0]);
      } else {
        s.template load_edge<kKind != kAll>(v + mine, t[0], q[0]);
      }
      s.template add_to<kKind>(sum, v, t[0], q[0]);
      v += S::kTile;
    }
    sum.settle();
  }
  return scan(sum.total());
}
template <int kType, bool kDrawn>
__device__ __forceinline__ Pair share_mass(const Share<kType, kDrawn>& s) {
  if constexpr (kDrawn) {
    const Kind k = kind_of(s.S);
    if (k == kFirst) return share_mass_of<kFirst>(s);
    if (k == kMore) return share_mass_of<kMore>(s);
  }
  return share_mass_of<kAll>(s);
}

// The sum of the shares' masses, 4 to a lane: up to each lane, and before each of its four.
struct Masses {
  Pair m[4], upto, before;
  __device__ __forceinline__ Masses(const float2* mass, int warps) {
    const int lane = lane_id();
    Pair x;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (4 * lane + k < warps) m[k] = Pair(mass[4 * lane + k]);
      x = x + m[k];
    }
    upto = scan(x);
    before = shfl_up(upto, 1);
    if (lane == 0) before = Pair();
  }
  __device__ __forceinline__ Pair total() const { return shfl(upto, 31); }
  // The share in which the cumulative sum passes goal, and the sum before it (by one warp).  By roundings
  // it may pass in none: then the last share with any mass.
  __device__ __forceinline__ int find(Pair goal, Pair& below) const {
    bool some = false, passed = false;
    int mine = 0;
    Pair cum = before, at = before;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (!passed && m[k].positive()) {
        some = true;
        mine = 4 * static_cast<int>(lane_id()) + k;
        at = cum;
        passed = cum + m[k] > goal;
      }
      cum = cum + m[k];
    }
    const uint32_t any = __ballot_sync(0xFFFFFFFFu, some), past = __ballot_sync(0xFFFFFFFFu, passed);
    const int lane = past ? __ffs(past) - 1 : any ? 31 - __clz(static_cast<int>(any)) : 0;
    below = shfl(at, lane);
    return __shfl_sync(0xFFFFFFFFu, mine, lane);
  }
};

// The token of that share: the least whose cumulative sum passes goal, or the share's last with any
// residual where by roundings none does.  Executed by all warps of a CTA, a tile each; the one that has
// the token writes it.
template <int kType, bool kDrawn>
__device__ __forceinline__ void find_token(const Share<kType, kDrawn>& s, Shared& sh, int32_t* token) {
  using S = Share<kType, kDrawn>;
  const int lane = lane_id(), warp = warp_id();
  const Pair goal(sh.goal);
  Pair below(sh.below);
  int last = s.v0;  // the last tile with any residual
  for (int g = s.v0;; g += kWarps * S::kTile) {
    const bool over = g >= s.v1;  // past the share: its last token, from one tile that all warps look at
    const int v0 = over ? last : g + warp * S::kTile, v = v0 + lane * S::kN;
    Pair2 r[S::kN / 2];
    Pair x;
#pragma unroll
    for (int i = 0; i < S::kN / 2; ++i) r[i] = {both(0.0f), both(0.0f)};
    if (v0 < s.v1) {
      Vec<kType> t, q;
      const bool two = kDrawn && s.draft;
      if (s.inside(v0, 1)) {
        two ? s.template load<true>(v, t, q) : s.template load<false>(v, t, q);
      } else {
        two ? s.template load_edge<true>(v, t, q) : s.template load_edge<false>(v, t, q);
      }
      s.terms(v, t, q, r);
      Sum sum;
#pragma unroll
      for (int i = 0; i < S::kN / 2; ++i) sum.template add<false>(r[i]);
      x = sum.total();
    }
    const Pair upto = scan(x);
    if (lane == 31) sh.tile[warp] = upto.raw();
    __syncthreads();
    const Pair m = lane < kWarps ? Pair(sh.tile[lane]) : Pair(), cum = below + scan(m);
    const uint32_t some = __ballot_sync(0xFFFFFFFFu, m.positive());
    const uint32_t past = __ballot_sync(0xFFFFFFFFu, m.positive() && cum > goal);
    if (past || over) {
      const int w = over ? 0 : __ffs(past) - 1;
      if (warp != w) return;
      const Pair start = w == 0 ? below : shfl(cum, w - 1), end = start + upto;
      // (Only lanes with a residual: another's sum may pass its neighbour's by roundings alone.)
      const uint32_t lanes = __ballot_sync(0xFFFFFFFFu, x.positive());
      const uint32_t here = __ballot_sync(0xFFFFFFFFu, x.positive() && end > goal);
      const int at = !over && here ? __ffs(here) - 1 : 31 - __clz(static_cast<int>(lanes));
      Pair c = shfl_up(end, 1);
      if (lane == 0) c = start;
      int found = -1;
      bool passed = false;
#pragma unroll
      for (int i = 0; i < S::kN; ++i) {
        const Pair e = norm(i & 1 ? Pair{r[i / 2].hi.y, r[i / 2].lo.y} : Pair{r[i / 2].hi.x, r[i / 2].lo.x});
        c = c + e;
        if (!passed && e.positive()) {
          found = v + i;
          passed = !over && c > goal;
        }
      }
      if (lane == at) *token = found;
      return;
    }
    if (some) last = g + (31 - __clz(static_cast<int>(some))) * S::kTile;
    below = shfl(cum, 31);
    __syncthreads();  // sh.tile is read
  }
}

// Whether u q W < t, t = max(p - S q, 0) (drawn), or u W < t, t = p (q = 1, S = 0).
template <bool kDrawn>
__device__ __forceinline__ bool accepts(float u, float p, float q, Pair S, Pair W) {
  float right = p;
  if constexpr (kDrawn) {
    const Pair2 r = residual(both(p), both(q), S);
    right = r.hi.x + r.lo.x;
  }
  const float left = u * q * W.hi;
  // Both sides are within 2^-22 of theirs, and t besides within 2^-45 of p (residual).
  if (fabsf(left - right) > 1e-6f * (fabsf(left) + right) + 1e-12f * p && fabsf(left) + right > 1e-30f)
    return left < right;
  const double t = fmax(__dsub_rn(p, __dmul_rn(S.value(), q)), 0.0);
  return __dmul_rn(__dmul_rn(u, q), W.value()) < t;
}

template <int kType, bool kDrawn>
__global__ void __launch_bounds__(kThreads, 2) verify_kernel(const VerifyParams p) {
  __shared__ Shared sh;
  const cg::cluster_group cluster = cg::this_cluster();
  const int ranks = cluster.num_blocks(), rank = cluster.block_rank(), b = blockIdx.x / ranks;
  const int lane = lane_id(), warp = warp_id(), warps = ranks * kWarps;
  const Shared* leader = cluster.map_shared_rank(&sh, 0);
  const int64_t nodes = static_cast<int64_t>(b) * p.n;
  const float u0 = __ldg(p.uniforms + nodes);
  int cnt = 0;
  // A CTA's shared memory may be touched by others only once it runs: each says so here, and all wait for
  // it before the first command, behind the first CTA's gather.
  auto running = cluster.barrier_arrive();

  if (rank == 0) {
    uint32_t odd_at = 0, bit = 1;  // of the thread's nodes, those with a token or parent out of range
    for (int i = threadIdx.x; i < p.n; i += kThreads, bit <<= 1) {
      int up = __ldg(p.parents + nodes + i);
      const int x = __ldg(p.tokens + nodes + i);
      const float u = __ldg(p.uniforms + nodes + i);
      const bool known = up >= 0 && up < i, real = x >= 0 && x < p.V;
      if (up < -1 || up >= i || (i > 0 && !real)) odd_at |= bit;
      const int64_t v = known && real ? (nodes + up) * p.V + x : 0;
      sh.up[i] = known ? up : -1;  // -1: no node's child, never asked
      sh.token[i] = real ? x : -1;
      sh.p[i] = known && real ? load_prob<kType>(p.target, v) : 0.0f;
      sh.q[i] = kDrawn && known && real ? load_prob<kType>(p.draft, v) : 0.0f;
      sh.u[i] = u;
    }
    cnt = kv8::seq_count(p.counts, b, p.n);
    bool odd = threadIdx.x == 0 && p.counts && __ldg(p.counts + b) != cnt;
    bit = 1;
    for (int i = threadIdx.x; i < cnt; i += kThreads, bit <<= 1) odd |= (odd_at & bit) != 0;
    if (odd) raise_clamped(p.status);
    __syncthreads();
  }

  // The walk, in warp 0 of the first CTA (whose other warps, like the other CTAs', only follow).
  const bool leads = rank == 0 && warp == 0;
  int node = 0, next = 1, len = cnt > 0 ? 1 : 0, refused = 0;
  Pair S, W{1.0f, 0.0f};
  if (leads && lane == 0 && cnt > 0) p.path[nodes] = 0;
  // The first child of the node at hand from number `from` on; cnt if there is none.
  auto child_from = [&](int from) {
    for (int j0 = from & ~31; j0 < cnt; j0 += 32) {
      const int j = j0 + lane;
      const uint32_t m = __ballot_sync(0xFFFFFFFFu, j >= from && j < cnt && sh.up[j] == node);
      if (m) return j0 + __ffs(m) - 1;
    }
    return cnt;
  };
  int child = leads ? child_from(next) : 0;
  Command cmd;
  cluster.barrier_wait(std::move(running));
  for (;;) {
    if (leads) {
      bool refusing = false;
      while (child < cnt && !refusing) {
        bool gone = false;
        for (int k = lane; k < refused; k += 32) gone |= sh.refused[k] == sh.token[child];
        const float pc = !kDrawn && __any_sync(0xFFFFFFFFu, gone) ? 0.0f : sh.p[child];
        if (accepts<kDrawn>(sh.u[child], pc, kDrawn ? sh.q[child] : 1.0f, S, W)) {
          node = child;
          if (lane == 0) p.path[nodes + len] = child;
          ++len;
          S = Pair(), W = Pair{1.0f, 0.0f}, refused = 0;
        } else if constexpr (kDrawn) {
          refusing = true;
        } else if (pc > 0.0f) {
          W = W + Pair{-pc, 0.0f};
          if (lane == 0) sh.refused[refused] = sh.token[child];
          ++refused;
          __syncwarp();
        }
        child = child_from(child + 1);
      }
      cmd = Command{cnt == 0, refusing, child >= cnt, node, refused, (refusing ? S + W : S).raw()};
      if (lane < ranks) cluster.map_shared_rank(&sh, lane)->cmd = cmd;
    }
    cluster.sync();
    cmd = sh.cmd;
    if (cmd.done) break;
    if (!kDrawn && rank > 0 && cmd.refused > 0) {
      for (int i = threadIdx.x; i < cmd.refused; i += kThreads) sh.refused[i] = leader->refused[i];
      __syncthreads();
    }
    {
      const Share<kType, kDrawn> share(p, b, cmd, sh.refused, rank * kWarps + warp, warps);
      const float2 mass = shfl(share_mass(share), 31).raw();
      if (cmd.last ? lane < ranks : lane == 0)
        cluster.map_shared_rank(&sh, lane)->mass[rank * kWarps + warp] = mass;
    }
    cluster.sync();
    if (cmd.last) {  // every CTA finds the share, and the one that has it the token
      if (warp == 0) {
        const Masses all(sh.mass, warps);
        const Pair total = all.total(), goal = u0 * total;
        Pair below;
        const int from = all.find(goal, below);
        if (lane == 0) sh.goal = goal.raw(), sh.below = below.raw(), sh.from = total.positive() ? from : -1;
      }
      __syncthreads();
      if (sh.from >= 0) {
        if (sh.from / kWarps == rank) {
          const Share<kType, kDrawn> share(p, b, cmd, sh.refused, sh.from, warps);
          find_token(share, sh, p.next_token + b);
        }
        break;
      }
      if (!cmd.refusing) break;  // no residual at all
      continue;                  // the refusal leaves nothing, and so the residual as it was
    }
    if (leads) {
      const Pair mass = Masses(sh.mass, warps).total();
      if (mass.positive()) {
        S = Pair(cmd.S);
        W = mass;
      }
    }
  }
  if (leads) {
    for (int i = len + lane; i < p.n; i += 32) p.path[nodes + i] = -1;
    if (lane == 0) {
      p.accepted[b] = len;
      if (cmd.done || sh.from < 0) {
        p.next_token[b] = -1;
        if (cnt > 0) raise_empty_row(p.status);
      }
    }
  }
  cluster.sync();  // no CTA leaves while its list may be read
}

template <int kType, bool kDrawn>
cudaError_t launch(const DraftVerifyArgs& a, cudaStream_t s) {
  VerifyParams p{a.n, a.V, a.target, a.draft, a.tokens, a.parents, a.counts, a.uniforms, a.path, a.accepted,
                 a.next_token, a.status};
  // CTAs of a cluster: doubled while each warp has more than one tile of the vocabulary and the device
  // holds the clusters of all sequences at once (two CTAs a multiprocessor).  us with 2, 4 and 8: 64 sequences
  // of 100003 bf16 values 14.8, 14.8, 21.2 (4 fill the device); with 4 and 8: 32 of 131072 float32 values
  // 30.1, 25.2 (8); with 1, 2 and 4: 150 of 32000 bf16 values 28.6, 23.0, 31.9 (2).
  const int tiles = (a.V + Share<kType, kDrawn>::kTile - 1) / Share<kType, kDrawn>::kTile;
  int ranks = 1;
  while (ranks < kMostRanks && tiles > ranks * kWarps && ranks * static_cast<int64_t>(a.B) <= a.sms) ranks *= 2;
  void* args[] = {&p};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {static_cast<unsigned>(ranks), 1, 1};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B) * ranks);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(verify_kernel<kType, kDrawn>), args);
}

}  // namespace draft

int launch_draft_verify(const DraftVerifyArgs& a, cudaStream_t s, std::string& err) {
  using namespace draft;
  cudaError_t e;
  if (a.draft) {
    e = a.type == kProbF32 ? launch<kProbF32, true>(a, s)
        : a.type == kProbF16 ? launch<kProbF16, true>(a, s) : launch<kProbBf16, true>(a, s);
  } else {
    e = a.type == kProbF32 ? launch<kProbF32, false>(a, s)
        : a.type == kProbF16 ? launch<kProbF16, false>(a, s) : launch<kProbBf16, false>(a, s);
  }
  if (e != cudaSuccess) {
    err = std::string("draft verify launch: ") + cudaGetErrorString(e);
    return -5;
  }
  return 0;
}

}  // namespace ea
