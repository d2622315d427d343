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
// do meanwhile): sum the masses at a node, each warp a contiguous share of the vocabulary, and, by the
// one warp whose share the drawn number falls in, find the token.
//
// Decisions are taken in 64 bits.  Sums over the vocabulary would be bound by the device's few 64-bit
// units, so their terms and partial sums are pairs of float32 values (error-free sums and products),
// about 2^-46 relative; each warp's is rounded to 64 bits once.
#include <cooperative_groups.h>

#include <type_traits>

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

enum Op : int { kSum, kFind, kDone };

struct Command {  // of the first CTA to all
  int op, node;
  int warp;           // kFind: of the cluster
  int refused;        // tokens taken out of the target's probabilities (drafts that were not drawn)
  double S;
  double goal, below;  // kFind: what the cumulative sum has to pass, and where the warp's share starts
};

struct Shared {
  Command cmd;
  double mass[kMostRanks * kWarps];  // first CTA: of each warp's share
  float p[kMostNodes], q[kMostNodes], u[kMostNodes];
  int up[kMostNodes], token[kMostNodes];
  int refused[kMostNodes];
};

// A value as the unevaluated sum of two float32 values.
struct Pair {
  float hi, lo;
  __device__ __forceinline__ double value() const { return static_cast<double>(hi) + static_cast<double>(lo); }
};
__device__ __forceinline__ void add(Pair& a, Pair x) {
  const float s = a.hi + x.hi, b = s - a.hi;
  a.lo += ((a.hi - (s - b)) + (x.hi - b)) + x.lo;
  a.hi = s;
}
// max(p - S q, 0), S = sh + sl.
__device__ __forceinline__ Pair residual(float p, float q, float sh, float sl) {
  const float h = sh * q, e = fmaf(sl, q, fmaf(sh, q, -h));
  const float d = p - h, b = d - p;
  const float lo = ((p - (d - b)) - (h + b)) - e;
  const float hi = d + lo;
  if (!(hi > 0.0f)) return {0.0f, 0.0f};
  return {hi, lo - (hi - d)};
}

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
  __device__ __forceinline__ void values(float (&x)[kN]) const {
    const uint32_t c[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kType == kProbF32) {
        x[i] = prob(__uint_as_float(c[i]));
      } else {
        const float2 f = kv8::unpack16<kType == kProbBf16>(c[i]);
        x[2 * i] = prob(f.x), x[2 * i + 1] = prob(f.y);
      }
    }
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
  float sh, sl;  // S
  const int* refused;
  int refusals;  // tokens to be taken out; 0 if none lies in the share

  __device__ __forceinline__ Share(const VerifyParams& p, int b, const Command& c, const int* list, int warp, int warps)
      : V(p.V), refused(list) {
    const int64_t row = (static_cast<int64_t>(b) * p.n + c.node) * V;
    target = static_cast<const typename Vec<kType>::Word*>(p.target) + row;
    const int before = static_cast<int>(row & (kN - 1));  // elements past a 16-byte boundary
    const int tiles = (V + before + kTile - 1) / kTile, per = (tiles + warps - 1) / warps;
    v0 = min(warp * per, tiles) * kTile - before;
    v1 = min((warp + 1) * per, tiles) * kTile - before;
    sh = static_cast<float>(c.S);
    sl = static_cast<float>(c.S - static_cast<double>(sh));
    draft = kDrawn && sh != 0.0f ? static_cast<const typename Vec<kType>::Word*>(p.draft) + row : nullptr;
    refusals = 0;
    if constexpr (!kDrawn) {
      bool here = false;
      for (int i = lane_id(); i < c.refused; i += 32) here |= list[i] >= v0 && list[i] < v1;
      if (__any_sync(0xFFFFFFFFu, here)) refusals = c.refused;
    }
  }
  __device__ __forceinline__ bool inside(int v, int tiles) const { return v >= 0 && v + tiles * kTile <= V; }
  // The vectors at v: of a tile inside the row, and of one that reaches past its ends.
  __device__ __forceinline__ void load(int v, Vec<kType>& t, Vec<kType>& q) const {
    t.load(target, v);
    q.w = make_uint4(0u, 0u, 0u, 0u);
    if (kDrawn && draft) q.load(draft, v);
  }
  __device__ __forceinline__ void load_edge(int v, Vec<kType>& t, Vec<kType>& q) const {
    t.load_edge(target, v, V);
    q.w = make_uint4(0u, 0u, 0u, 0u);
    if (kDrawn && draft) q.load_edge(draft, v, V);
  }
  // The residuals of the vectors at v.
  __device__ __forceinline__ void terms(int v, const Vec<kType>& t, const Vec<kType>& q, Pair (&r)[kN]) const {
    float x[kN], y[kN];
    t.values(x);
    if (kDrawn) q.values(y);
#pragma unroll
    for (int i = 0; i < kN; ++i) r[i] = kDrawn ? residual(x[i], y[i], sh, sl) : Pair{x[i], 0.0f};
    if constexpr (!kDrawn) {
      for (int k = 0; k < refusals; ++k) {
        const int at = refused[k] - v;
#pragma unroll
        for (int i = 0; i < kN; ++i)
          if (at == i) r[i].hi = 0.0f;
      }
    }
  }
};

// A warp's inclusive sums of x over its lanes.
__device__ __forceinline__ double scan(double x) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (static_cast<int>(lane_id()) >= o) x += y;
  }
  return x;
}

// The mass of the warp's share.
template <int kType, bool kDrawn>
__device__ __forceinline__ double share_mass(const Share<kType, kDrawn>& s) {
  using S = Share<kType, kDrawn>;
  constexpr int kAhead = 4;  // tiles whose loads are in flight together
  const int mine = static_cast<int>(lane_id()) * S::kN;
  Pair sum{0.0f, 0.0f};
  auto take = [&](int v, const Vec<kType>& t, const Vec<kType>& q) {
    Pair r[S::kN];
    s.terms(v, t, q, r);
#pragma unroll
    for (int i = 0; i < S::kN; ++i) add(sum, r[i]);
  };
  for (int v = s.v0; v < s.v1;) {
    Vec<kType> t[kAhead], q[kAhead];
    if (v + kAhead * S::kTile <= s.v1 && s.inside(v, kAhead)) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) s.load(v + i * S::kTile + mine, t[i], q[i]);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) take(v + i * S::kTile + mine, t[i], q[i]);
      v += kAhead * S::kTile;
    } else {
      if (s.inside(v, 1)) {
        s.load(v + mine, t[0], q[0]);
      } else {
        s.load_edge(v + mine, t[0], q[0]);
      }
      take(v + mine, t[0], q[0]);
      v += S::kTile;
    }
  }
  double x = sum.value();
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
  return x;
}

// The least token of the share whose cumulative residual, `below` before the share, passes goal; by
// roundings at the share's end there may be none, and the last with any residual is it.
template <int kType, bool kDrawn>
__device__ __forceinline__ int share_find(const Share<kType, kDrawn>& s, double goal, double below) {
  using S = Share<kType, kDrawn>;
  int last = -1;
  for (int v0 = s.v0; v0 < s.v1; v0 += S::kTile) {
    const int v = v0 + static_cast<int>(lane_id()) * S::kN;
    Vec<kType> t, q;
    Pair r[S::kN];
    if (s.inside(v0, 1)) {
      s.load(v, t, q);
    } else {
      s.load_edge(v, t, q);
    }
    s.terms(v, t, q, r);
    double x = 0.0;
#pragma unroll
    for (int i = 0; i < S::kN; ++i) {
      x += r[i].value();
      if (r[i].hi > 0.0f) last = v + i;
    }
    const double upto = below + scan(x);
    // (x > 0: a lane's sum may pass its neighbour's by roundings alone.)
    const uint32_t past = __ballot_sync(0xFFFFFFFFu, x > 0.0 && upto > goal);
    if (past) {
      double cum = __shfl_up_sync(0xFFFFFFFFu, upto, 1);
      if (lane_id() == 0) cum = below;
      int found = -1;
      bool done = false;
#pragma unroll
      for (int i = 0; i < S::kN; ++i) {
        cum += r[i].value();
        if (!done && r[i].hi > 0.0f) {
          found = v + i;
          done = cum > goal;
        }
      }
      return __shfl_sync(0xFFFFFFFFu, found, __ffs(past) - 1);
    }
    below = __shfl_sync(0xFFFFFFFFu, upto, 31);
  }
  return __reduce_max_sync(0xFFFFFFFFu, last);
}

template <int kType, bool kDrawn>
__global__ void __launch_bounds__(kThreads, 2) verify_kernel(const VerifyParams p) {
  __shared__ Shared sh;
  const cg::cluster_group cluster = cg::this_cluster();
  const int ranks = cluster.num_blocks(), rank = cluster.block_rank(), b = blockIdx.x / ranks;
  const int lane = lane_id(), warp = warp_id();
  const Shared* leader = cluster.map_shared_rank(&sh, 0);
  const int cnt = kv8::seq_count(p.counts, b, p.n);

  if (rank == 0) {
    const int64_t at = static_cast<int64_t>(b) * p.n;
    bool odd = threadIdx.x == 0 && p.counts && __ldg(p.counts + b) != cnt;
    for (int i = 1 + static_cast<int>(threadIdx.x); i < cnt; i += kThreads) {
      int up = __ldg(p.parents + at + i);
      const int x = __ldg(p.tokens + at + i);
      const bool known = up >= 0 && up < i, real = x >= 0 && x < p.V;
      odd |= !real || up < -1 || up >= i;
      if (!known) up = -1;  // no node's child: never asked
      const int64_t v = known && real ? (at + up) * p.V + x : 0;
      sh.up[i] = up;
      sh.token[i] = real ? x : -1;
      sh.p[i] = known && real ? load_prob<kType>(p.target, v) : 0.0f;
      sh.q[i] = kDrawn && known && real ? load_prob<kType>(p.draft, v) : 0.0f;
      sh.u[i] = __ldg(p.uniforms + at + i);
    }
    if (odd) raise_clamped(p.status);
    __syncthreads();
  }

  // The walk, in warp 0 of the first CTA (whose other warps, like the other CTAs', only follow).
  const bool leads = rank == 0 && warp == 0;
  int node = 0, next = 1, len = 0, refused = 0;
  double S = 0.0, W = 1.0, total = 0.0;
  bool summed = false;    // sh.mass holds the shares of the residual at (node, S)
  bool refusing = false;  // the sum asked for is a refusal's, at S + W
  Command cmd;
  if (leads && cnt > 0) {
    if (lane == 0) p.path[static_cast<int64_t>(b) * p.n] = 0;
    len = 1;
  }
  for (;;) {
    if (leads) {
      cmd = Command{kSum, node, 0, refused, S, 0.0, 0.0};
      if (cnt == 0) {
        cmd.op = kDone;
      } else {
        bool over = false;  // no child left to ask
        for (;;) {
          int child = cnt;
          for (int j0 = next & ~31; j0 < cnt; j0 += 32) {
            const int j = j0 + lane;
            const uint32_t m = __ballot_sync(0xFFFFFFFFu, j >= next && j < cnt && sh.up[j] == node);
            if (m) {
              child = j0 + __ffs(m) - 1;
              break;
            }
          }
          if (child >= cnt) {
            over = true;
            break;
          }
          next = child + 1;
          const double pc = sh.p[child], qc = sh.q[child], u = sh.u[child];
          double t;
          bool yes;
          if constexpr (kDrawn) {
            t = fmax(__dsub_rn(pc, __dmul_rn(S, qc)), 0.0);
            yes = __dmul_rn(__dmul_rn(u, qc), W) < t;
          } else {
            bool gone = false;
            for (int k = lane; k < refused; k += 32) gone |= sh.refused[k] == sh.token[child];
            t = __any_sync(0xFFFFFFFFu, gone) ? 0.0 : pc;
            yes = __dmul_rn(u, W) < t;
          }
          if (yes) {
            node = child;
            if (lane == 0) p.path[static_cast<int64_t>(b) * p.n + len] = child;
            ++len;
            S = 0.0, W = 1.0, refused = 0, summed = false;
          } else if constexpr (kDrawn) {
            refusing = true;
            break;
          } else if (t > 0.0) {
            W = __dsub_rn(W, t);
            if (lane == 0) sh.refused[refused] = sh.token[child];
            ++refused;
            __syncwarp();
          }
        }
        cmd.node = node;
        cmd.refused = refused;
        cmd.S = refusing ? __dadd_rn(S, W) : S;
        if (over && summed && !(total > 0.0)) {
          cmd.op = kDone;
        } else if (over && summed) {
          // The token: the warp whose share the drawn number falls in finds it.
          const int warps = ranks * kWarps;
          double m[4], x = 0.0;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            m[k] = 4 * lane + k < warps ? sh.mass[4 * lane + k] : 0.0;
            x += m[k];
          }
          const double upto = scan(x), goal = __dmul_rn(static_cast<double>(__ldg(p.uniforms + static_cast<int64_t>(b) * p.n)), total);
          double cum = __shfl_up_sync(0xFFFFFFFFu, upto, 1);
          if (lane == 0) cum = 0.0;
          uint32_t past = __ballot_sync(0xFFFFFFFFu, x > 0.0 && upto > goal);
          // By roundings there may be none: the last with any mass.
          if (!past) past = 0x80000000u >> __clz(static_cast<int>(__ballot_sync(0xFFFFFFFFu, x > 0.0)));
          int mine = 0;
          double below = cum;
          bool done = false;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if (!done && m[k] > 0.0) {
              mine = 4 * lane + k;
              below = cum;
              done = cum + m[k] > goal;
            }
            cum += m[k];
          }
          const int from = __ffs(past) - 1;
          cmd.op = kFind;
          cmd.warp = __shfl_sync(0xFFFFFFFFu, mine, from);
          cmd.below = __shfl_sync(0xFFFFFFFFu, below, from);
          cmd.goal = goal;
        }
      }
      if (lane < ranks) cluster.map_shared_rank(&sh, lane)->cmd = cmd;
    }
    cluster.sync();
    cmd = sh.cmd;
    if (cmd.op == kDone) break;
    const Share<kType, kDrawn> share(p, b, cmd, leader->refused, rank * kWarps + warp, ranks * kWarps);
    if (cmd.op == kFind) {
      if (cmd.warp == rank * kWarps + warp) {
        const int token = share_find(share, cmd.goal, cmd.below);
        if (lane == 0) p.next_token[b] = token;
      }
      break;
    }
    const double mass = share_mass(share);
    if (lane == 0) cluster.map_shared_rank(&sh, 0)->mass[rank * kWarps + warp] = mass;
    cluster.sync();
    if (leads) {
      double x = 0.0;
#pragma unroll
      for (int k = 0; k < 4; ++k) x += 4 * lane + k < ranks * kWarps ? sh.mass[4 * lane + k] : 0.0;
      const double sum = __shfl_sync(0xFFFFFFFFu, scan(x), 31);
      summed = true;
      if (!refusing) {
        total = sum;
      } else if (sum > 0.0) {
        S = cmd.S;
        W = total = sum;
      } else {
        summed = false;  // a refusal that would leave nothing leaves the residual as it was
      }
      refusing = false;
    }
  }
  if (leads) {
    for (int i = len + lane; i < p.n; i += 32) p.path[static_cast<int64_t>(b) * p.n + i] = -1;
    if (lane == 0) {
      p.accepted[b] = len;
      if (cmd.op == kDone) {
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
  // CTAs of a cluster: doubled while each warp has more than two tiles of the vocabulary.
  const int tiles = (a.V + Share<kType, kDrawn>::kTile - 1) / Share<kType, kDrawn>::kTile;
  int ranks = 1;
  while (ranks < kMostRanks && tiles > 2 * ranks * kWarps) ranks *= 2;
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
