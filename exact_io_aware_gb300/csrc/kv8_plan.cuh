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
  static constexpr int kTurn = 10, kParts = 2, kLongRun = 60;  // (plan_trees)
  __device__ __forceinline__ int row_tiles(int cnt) const { return cnt > 0 ? 1 : 0; }
  static constexpr bool kPacked = false;
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
  static constexpr bool kPacked = false;
  __device__ __forceinline__ int rows(int) const { return R; }
  __device__ __forceinline__ int query(int r) const { return r % n; }
  __device__ __forceinline__ int query(int r, int) const { return query(r); }
  __device__ __forceinline__ int64_t row_offset(int b, int hk, int r, int) const { return row_offset(b, hk, r); }
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

// Real rows alone, in the order they lie in memory: row r is query r % cnt of head r / cnt.  For a tree's
// rows, which all see every tile's keys up to the sequence's end: padding would cost what real rows do
// (4 x 8 heads of four times 128 to 256 rows over 16384 keys, d = 64, fp16: 280 us with it, 247 packed).
struct ByNode : Geometry {
  static constexpr int kStep = kBlockKeys;
  static constexpr bool kPacked = true;
  static constexpr int kTurn = 7, kParts = 3, kLongRun = 1 << 30;  // (plan_trees)
  __device__ __forceinline__ int row_tiles(int cnt) const { return (G * cnt + tile - 1) >> (31 - __clz(tile)); }
  __device__ __forceinline__ int rows(int cnt) const { return G * cnt; }
  __device__ __forceinline__ int query(int r, int cnt) const { return r % cnt; }
  __device__ __forceinline__ int64_t row_offset(int b, int hk, int r, int cnt) const {
    return (static_cast<int64_t>(b) * Hk * G + static_cast<int64_t>(hk) * G + r / cnt) * n + r % cnt;
  }
  __device__ __forceinline__ bool span(int r0, int, int cnt, int& lo, int& hi) const {
    lo = 0;
    hi = cnt - 1;
    return r0 < G * cnt;
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

// The same for a tree's rows, all of whose tiles of a sequence have its every chunk.  Equal runs across the list
// cut tiles where they happen to end, and a run has the end of one tile and the start of another; so where the
// tiles are no more than the CTAs, a CTA takes one tile or an equal part of one, if the parts are not much longer than
// runs would be; and where there are more and all are alike, whole ones.  In chunks of work, what a tile's
// start and end cost is kTurn, what parts and their join cost kParts.  us in equal runs and so, d = 128:
//   256 rows (kTurn: 13 us)   128 heads of 1024 keys 51, 33, of 6144 112, 103; 32 of 4096 41, 33; 512 of 1024 145,
//                             123; 24 of 1024 to 4096 37, 27; 16 of 49152 101, 94
//   16 rows (4 us)            32 heads of 4096 keys 21.4, 17.3, of 16384 40.2, 36.5; 256 of 1024 26.2, 21.4; 8 of 256 to
//                             1024 14.8, 11.3; runs longer than kLongRun gain nothing (64 heads of 16384 58.2, 58.5)
template <class Geo>
__device__ __forceinline__ Place plan_trees(const Geo& g, int cta, int ctas, int min_chunks, int& u0, int& u1) {
  constexpr int kTurn = Geo::kTurn, kParts = Geo::kParts;
  const int lane = lane_id();
  // Row tiles of a head of sequence b, and chunks of each.
  auto tiles_of = [&](int b, int& c) {
    c = 0;
    if (b >= g.B) return 0;
    c = chunks_of(g, seq_len(g.lengths, b, g.cap));
    return c > 0 ? g.row_tiles(seq_count(g.counts, b, g.n)) : 0;
  };
  int c0;
  const int t0 = tiles_of(lane, c0);  // the lane's first sequence's
  // Over all heads, tiles cut into parts of at most `part` chunks.
  auto parts_of = [&](int part) {
    int sum = t0 * ((c0 + part - 1) / part), c;
    for (int b = lane + 32; b < g.B; b += 32) sum += tiles_of(b, c) * ((c + part - 1) / part);
    return __reduce_add_sync(0xFFFFFFFFu, sum) * g.Hk;
  };
  int total = t0 * c0, tiles = t0, least = t0 > 0 ? c0 : 1 << 30, most = t0 > 0 ? c0 : 0;
  for (int b = lane + 32; b < g.B; b += 32) {
    int c;
    const int t = tiles_of(b, c);
    total += t * c;
    tiles += t;
    if (t > 0) least = min(least, c), most = max(most, c);
  }
  total = __reduce_add_sync(0xFFFFFFFFu, total) * g.Hk;
  tiles = __reduce_add_sync(0xFFFFFFFFu, tiles) * g.Hk;
  least = __reduce_min_sync(0xFFFFFFFFu, least);
  most = __reduce_max_sync(0xFFFFFFFFu, most);
  int per = run_length(total, ctas, min_chunks);
  int part = 0;  // > 0: a CTA takes one part, of at most so many chunks, of a tile
  if (per > Geo::kLongRun) {
  } else if (tiles <= ctas) {
    // The least part (at least `per`) at which there are no more of them than CTAs.
    int lo = per, hi = min(per + kTurn + kParts, max(most, per));
    if (least == most) lo = hi = min(max((most + ctas / tiles - 1) / (ctas / tiles), per), hi);
    if (parts_of(hi) <= ctas) {
      while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (parts_of(mid) <= ctas) {
          hi = mid;
        } else {
          lo = mid + 1;
        }
      }
      if (lo <= per + kTurn + (lo < most ? 0 : kParts)) part = lo;
    }
  } else if (least == most) {
    const int whole = (tiles + ctas - 1) / ctas;
    if (whole * (most + kTurn) <= per + kTurn * (1 + whole) + kParts) per = whole * most;
  }
  u0 = part > 0 ? cta : cta * per;  // the first part or chunk: find its sequence
  u1 = part > 0 ? cta + 1 : min(u0 + per, total);
  Place p{0, 0, 0, 0, 0};
  if (u0 >= u1) return p;
  int base = 0, t = 0, units = 0;  // of the sequence: tiles of a head, and parts or chunks of a tile
  for (int b0 = 0;; b0 += 32) {
    if (b0 >= g.B) {  // more CTAs than parts
      u0 = u1 = 0;
      return p;
    }
    int c = c0;
    const int mine = b0 == 0 ? t0 : tiles_of(b0 + lane, c), each = part > 0 ? (c + part - 1) / part : c, v = mine * each * g.Hk;
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
      t = __shfl_sync(0xFFFFFFFFu, mine, l);
      units = __shfl_sync(0xFFFFFFFFu, each, l);
      base += __shfl_sync(0xFFFFFFFFu, x - v, l);
      break;
    }
    base += __shfl_sync(0xFFFFFFFFu, x, 31);
  }
  const int tile = (u0 - base) / units;
  p.hk = tile / t;
  p.rt = tile % t;
  p.keys = seq_len(g.lengths, p.b, g.cap);
  if (part > 0) {  // a list of this tile alone
    u0 = (u0 - base) % units * part;
    u1 = min(u0 + part, chunks_of(g, p.keys));
  } else {
    p.start = base + tile * units;
  }
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
