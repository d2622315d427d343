// Attention over the 8-bit cache: which kernel a call takes, and the work its CTAs are given.
#include <type_traits>

#include "kv8_attend.cuh"

namespace ea {

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
  return R <= 8 ? 8 : R <= 16 ? 16 : 32;
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
  p.tree = a.tree;
  p.tree_words = (a.n + 31) / 32;
  p.part_z = static_cast<float*>(a.workspace);
  p.part_lm = p.part_z + rows * a.d;
  p.runs = reinterpret_cast<int2*>(p.part_lm + rows * 2);
  p.ctas = ctas;
  p.min_chunks = min_chunks;
  p.status = a.status;
  return p;
}

}  // namespace

namespace {

template <bool kTree>
cudaError_t dispatch(const Kv8Args& a, bool many, cudaStream_t s) {
  if (many) {
    using Geo = std::conditional_t<kTree, kv8::ByNode, kv8::ByHead>;
    auto p = attend_params<Geo>(a, a.sms, 2);
    if (a.bf16)
      return a.d == 128 ? launch_kv8_tc<true, 128>(p, s) : launch_kv8_tc<true, 64>(p, s);
    return a.d == 128 ? launch_kv8_tc<false, 128>(p, s) : launch_kv8_tc<false, 64>(p, s);
  }
  const auto p = attend_params<kv8::ByQuery>(a, kv8::kMostCtas * a.sms, 2 * kv8::kAttendWarps);
  if (a.bf16)
    return a.d == 128 ? launch_kv8_few<true, 128, kTree>(p, a.sms, s) : launch_kv8_few<true, 64, kTree>(p, a.sms, s);
  return a.d == 128 ? launch_kv8_few<false, 128, kTree>(p, a.sms, s) : launch_kv8_few<false, 64, kTree>(p, a.sms, s);
}

}  // namespace

int launch_kv8_attend(const Kv8Args& a, cudaStream_t s, std::string& err) {
  const int64_t R = static_cast<int64_t>(a.G) * a.n;
  const int tiles = static_cast<int>((R + rows_per_tile(R, a.d) - 1) / rows_per_tile(R, a.d));
  if (too_long(a.B, a.Hk, tiles, R, a.d, a.cap)) {
    err = "B * H * n_q * cap is too large for one call";
    return -2;
  }
  const bool many = R > few_rows(a.d);
  const cudaError_t e = a.tree ? dispatch<true>(a, many, s) : dispatch<false>(a, many, s);
  if (e != cudaSuccess) {
    err = std::string("kv8 attention launch: ") + cudaGetErrorString(e);
    return -5;
  }
  return 0;
}

}  // namespace ea
