// Which rows and keys a call has, and how its work is cut into equal runs on the device.
//
// A key/value head's R = G n rows (G query heads, n queries) are taken in tiles, a tile's keys in
// chunks.  The work list is every chunk of every (sequence, head, row tile) in that order; each CTA
// takes an equal run of it, whatever the sequences' lengths, which only the device knows.
#pragma once
#include "kv8_common.cuh"

namespace ea {
namespace kv8 {

constexpr int kChunk = 32;       // keys of a warp's step (few rows)
constexpr int kBlockKeys = 128;  // keys of a step of the tcgen05 kernels (many rows)

struct Geometry {
  int B, Hk, G, n, cap, R, tile, tiles;  // tiles of `tile` rows
  bool causal;
  const int32_t* lengths;
  const int32_t* counts;
  bool all_keys;  // the work list covers every held key, not only those some row sees
};

// Rows ordered by query: row r is query i = r / G of head r % G.  For few rows: one tile holds all of
// a head's.
struct ByQuery : Geometry {
  static constexpr int kStep = kChunk;
  __device__ __forceinline__ int query(int r) const { return r / G; }
  // Row of q and o, [B][Hk G][n][D].
  __device__ __forceinline__ int64_t row_offset(int b, int hk, int r) const {
    return (static_cast<int64_t>(b) * Hk * G + static_cast<int64_t>(hk) * G + r % G) * n + r / G;
  }
  // Least and greatest query of the tile's rows that is below cnt; false if there is none.
  __device__ __forceinline__ bool span(int, int, int cnt, int& lo, int& hi) const {
    lo = 0;
    hi = cnt - 1;
    return cnt > 0;
  }
};

// Rows ordered as they lie in memory: row r is query r % n of head r / n.
struct ByHead : Geometry {
  static constexpr int kStep = kBlockKeys;
  __device__ __forceinline__ int query(int r) const { return r % n; }
  __device__ __forceinline__ int64_t row_offset(int b, int hk, int r) const {
    return (static_cast<int64_t>(b) * Hk + hk) * R + r;
  }
  // As above, for rows r0 .. r1 - 1.
  __device__ __forceinline__ bool span(int r0, int r1, int cnt, int& lo, int& hi) const {
    const int a = r0 % n, z = (r1 - 1) % n;
    const bool wraps = r1 - r0 >= n || a > z;  // past a head's last query to the next's first
    lo = wraps ? 0 : a;
    hi = wraps ? (r1 - r0 >= n || a < cnt ? cnt - 1 : min(z, cnt - 1)) : min(z, cnt - 1);
    return lo < cnt && hi >= lo;
  }
};

// Keys query i sees: 0 for a padding row.
__device__ __forceinline__ int query_keys(const Geometry& g, int len, int cnt, int i) {
  if (i >= cnt) return 0;
  return g.causal ? min(max(len - cnt + i + 1, 0), len) : len;
}
// Keys any row of row tile rt sees (its last real query's).
template <class Geo>
__device__ __forceinline__ int tile_keys(const Geo& g, int len, int cnt, int rt) {
  if (g.all_keys) return len;
  int lo, hi;
  if (!g.span(rt * g.tile, min((rt + 1) * g.tile, g.R), cnt, lo, hi)) return 0;
  return query_keys(g, len, cnt, hi);
}
template <class Geo>
__device__ __forceinline__ int chunks_of(const Geo&, int keys) {
  return (keys + Geo::kStep - 1) / Geo::kStep;
}

// Chunks of all row tiles of one head of sequence b.
template <class Geo>
__device__ __forceinline__ int head_chunks(const Geo& g, int b) {
  const int len = seq_len(g.lengths, b, g.cap), cnt = seq_count(g.counts, b, g.n);
  if (g.tiles == 1) return chunks_of(g, tile_keys(g, len, cnt, 0));
  int u = 0;
  for (int rt = 0; rt < g.tiles; ++rt) u += chunks_of(g, tile_keys(g, len, cnt, rt));
  return u;
}

__device__ __forceinline__ int warp_sum(int v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

struct Place {
  int b, hk, rt;
  int keys;   // keys of the tile
  int start;  // work-list index of the tile's first chunk
};

// Whether a call's work list could outgrow the 32-bit arithmetic on it (its chunks if every
// sequence were full; far more than a cache in memory has, unless its queries are many).
inline bool list_too_long(int B, int Hk, int tiles, int cap, int step) {
  return static_cast<double>(B) * Hk * tiles * ((cap + step - 1) / step) >= static_cast<double>(1 << 30);
}

__device__ __forceinline__ int run_length(int total, int ctas, int min_chunks) {
  const int per = (total + ctas - 1) / ctas;
  return per < min_chunks ? min_chunks : per;
}

// The run of CTA `cta` (u0 .. u1 - 1, empty for u0 >= u1) and the tile u0 lies in.  Executed by
// whole warps; lanes take a sequence each.
template <class Geo>
__device__ __forceinline__ Place plan_run(const Geo& g, int cta, int ctas, int min_chunks,
                                          int& u0, int& u1) {
  const int lane = lane_id();
  const int v0 = lane < g.B ? head_chunks(g, lane) * g.Hk : 0;
  int sum = v0;
  for (int b = lane + 32; b < g.B; b += 32) sum += head_chunks(g, b) * g.Hk;
  const int total = warp_sum(sum);
  const int per = run_length(total, ctas, min_chunks);
  u0 = cta * per;
  u1 = min(u0 + per, total);
  Place p{0, 0, 0, 0, 0};
  if (u0 >= u1) return p;
  int base = 0, head = 0;
  for (int b0 = 0; b0 < g.B; b0 += 32) {
    const int v = b0 == 0 ? v0 : b0 + lane < g.B ? head_chunks(g, b0 + lane) * g.Hk : 0;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    const uint32_t past = __ballot_sync(0xFFFFFFFFu, base + x > u0);
    if (past) {
      const int l = __ffs(past) - 1;
      p.b = b0 + l;
      head = __shfl_sync(0xFFFFFFFFu, v, l) / g.Hk;
      base += __shfl_sync(0xFFFFFFFFu, x - v, l);
      break;
    }
    base += __shfl_sync(0xFFFFFFFFu, x, 31);
  }
  const int len = seq_len(g.lengths, p.b, g.cap), cnt = seq_count(g.counts, p.b, g.n);
  p.hk = (u0 - base) / head;
  base += p.hk * head;
  for (;; ++p.rt) {
    p.keys = tile_keys(g, len, cnt, p.rt);
    const int c = chunks_of(g, p.keys);
    if (u0 < base + c || p.rt + 1 >= g.tiles) break;
    base += c;
  }
  p.start = base;
  return p;
}

// The next tile of the list with at least one chunk (the caller knows that there is one).
template <class Geo>
__device__ __forceinline__ void next_place(const Geo& g, Place& p) {
  p.start += chunks_of(g, p.keys);
  for (;;) {
    if (++p.rt == g.tiles) {
      p.rt = 0;
      if (++p.hk == g.Hk) {
        p.hk = 0;
        if (++p.b == g.B) return;
      }
    }
    p.keys = tile_keys(g, seq_len(g.lengths, p.b, g.cap), seq_count(g.counts, p.b, g.n), p.rt);
    if (p.keys > 0) return;
  }
}

}  // namespace kv8
}  // namespace ea
