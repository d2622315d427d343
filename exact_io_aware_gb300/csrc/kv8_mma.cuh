// Warp-level products of the 8-bit cache with a few query rows (mma.sync, fp16 operands).
//
// Scores are formed transposed, S^T = K Q^T: the 16 rows of the instruction's A operand are
// keys and its 8 columns are query rows, so one to eight rows of a key/value head cost one
// instruction column block, and O^T = V^T P^T likewise has the value columns as its rows.  Both
// operands that come from the cache are E4M3 codes widened to fp16, which is exact.
//
// A warp walks chunks of 32 keys staged in shared memory by its own 16-byte asynchronous copies
// (chunk rows past the sequence's end are zero-filled).  The index an instruction sums over may
// be permuted if both operands agree, and so may the keys of a score block; both freedoms are
// used so that a lane reads whole 16-byte pieces of its rows without bank conflicts:
//   * lane (g, t) = (lane / 4, lane % 4) holds bytes 16 t .. 16 t + 15 of 64-column halves of K
//     rows g and g + 8 (slots), four bytes a step;
//   * slot s of a group of 8 keys is key key_of_slot(s);
//   * of V it holds columns D/8 g .. of the rows of slots 2t, 2t + 1, 2t + 8, 2t + 9.
#pragma once
#include "kv8_plan.cuh"

namespace ea {
namespace kv8 {

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void cp_async16(uint32_t sdst, const void* gsrc, uint32_t src_bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sdst), "l"(gsrc), "r"(src_bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t sdst, const void* gsrc) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(sdst), "l"(gsrc) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Layout of a chunk of 32 rows of D codes: 16-byte pieces permuted within 128-byte lines.
template <int D>
struct Chunk;
template <>
struct Chunk<128> {
  static constexpr int kBytes = kChunk * 128;
  __device__ static __forceinline__ uint32_t at(int row, int piece) {
    return row * 128 + ((piece ^ (row & 7)) << 4);
  }
  // Slots 0 .. 7 -> keys 0 4 2 6 5 1 7 3.  Eight lanes that load together hold two slots 2i,
  // 2i + 1 (keys 4 apart: different halves of a line) for K and slots 2t or 2t + 1 of two
  // neighbouring pieces for V (keys whose XOR with 0, 1 covers a line): no bank conflicts.
  __device__ static __forceinline__ int key_of_slot(int s) { return (0x37156240u >> (4 * s)) & 7; }
};
template <>
struct Chunk<64> {
  static constexpr int kBytes = kChunk * 64;
  __device__ static __forceinline__ uint32_t at(int row, int piece) {
    const int line = row >> 1;
    return line * 128 + (((((row & 1) << 2) | piece) ^ (line & 7)) << 4);
  }
  // Slots 0 .. 7 -> keys 0 1 3 2 4 5 7 6, by the same argument for two rows a line.
  __device__ static __forceinline__ int key_of_slot(int s) { return (0x67542310u >> (4 * s)) & 7; }
};

// Issues the copies of one chunk of K (or V): rows key0 .. key0 + 31 of `src`, zeros from `len`.
template <int D>
__device__ __forceinline__ void load_chunk(uint32_t sdst, const uint8_t* src, int key0, int len) {
  constexpr int kPieces = D / 16;
  const int lane = lane_id();
#pragma unroll
  for (int i = 0; i < kPieces; ++i) {
    const int idx = i * 32 + lane, row = idx / kPieces, piece = idx % kPieces;
    const int key = key0 + row;
    const bool in = key < len;
    cp_async16(sdst + Chunk<D>::at(row, piece),
               src + static_cast<int64_t>(in ? key : 0) * D + piece * 16, in ? 16u : 0u);
  }
}

// Eight query rows as the B operand of S^T = K Q^T.
template <int D>
struct QFrag {
  uint32_t b[D / 16][2];
};

// The lane's share of row `row` (null: zeros): columns 64 h + 16 t .. + 15 of each half h.
template <bool kBf16, int D>
__device__ __forceinline__ void load_q_row(const uint16_t* row, float (&x)[D / 4]) {
  const int t = lane_id() & 3;
#pragma unroll
  for (int h = 0; h < D / 64; ++h) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      uint4 u = make_uint4(0, 0, 0, 0);
      if (row) u = __ldg(reinterpret_cast<const uint4*>(row + h * 64 + t * 16 + e * 8));
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpack16<kBf16>(w[i]);
        x[h * 16 + e * 8 + 2 * i] = f.x;
        x[h * 16 + e * 8 + 2 * i + 1] = f.y;
      }
    }
  }
}

// Exponent that brings a row's largest finite |q| to 2^14 .. 2^15: queries enter the products as
// fp16 times a power of two of their own, so bf16 rows keep their range whatever the other rows
// hold, and values down to 2^-31 of the row's largest keep all of their bits.  (At most 2^126, so
// that the power and the inverse are normal values: rows below 2^-112 come to less than 2^14.)
__device__ __forceinline__ int q_exp(float amax) {
  const int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
  return min(14 - e, 126);
}

// The lane's share `x` of its row (lane / 4 of eight) as a fragment, and in kmul the factors of the
// scores of rows 2t and 2t + 1 (those of the lane's accumulators): c2 over the rows' powers of two.
template <int D>
__device__ __forceinline__ void pack_q(const float (&x)[D / 4], float c2, QFrag<D>& f, float (&kmul)[2]) {
  float amax = 0.0f;
#pragma unroll
  for (int e = 0; e < D / 4; ++e) amax = fmaxf(amax, finite_abs(x[e]));
  amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, 2));
  const float mul = pow2(q_exp(amax)), factor = c2 / mul;
#pragma unroll
  for (int s = 0; s < D / 16; ++s) {
    f.b[s][0] = pack_f16(x[4 * s] * mul, x[4 * s + 1] * mul);
    f.b[s][1] = pack_f16(x[4 * s + 2] * mul, x[4 * s + 3] * mul);
  }
  const int t = lane_id() & 3;
#pragma unroll
  for (int c = 0; c < 2; ++c) kmul[c] = __shfl_sync(0xFFFFFFFFu, factor, (2 * t + c) * 4);
}

// Scores of 16 keys (slots g and g + 8 of half `mt` of the chunk) with NT blocks of 8 rows:
// acc[j][0], [1]: slot g with rows 8j + 2t, 2t + 1; acc[j][2], [3]: slot g + 8.
template <int D, int NT>
__device__ __forceinline__ void scores16(const uint8_t* kbase, int mt, const QFrag<D> (&q)[NT],
                                         float (&acc)[NT][4]) {
  const int lane = lane_id(), g = lane >> 2, t = lane & 3;
  const int r0 = mt * 16 + Chunk<D>::key_of_slot(g);
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[j][e] = 0.0f;
#pragma unroll
  for (int h = 0; h < D / 64; ++h) {
    const uint4 u = *reinterpret_cast<const uint4*>(kbase + Chunk<D>::at(r0, h * 4 + t));
    const uint4 v = *reinterpret_cast<const uint4*>(kbase + Chunk<D>::at(r0 + 8, h * 4 + t));
    const uint32_t a[4] = {u.x, u.y, u.z, u.w}, b[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const uint32_t a0 = lo_codes(a[s]), a1 = lo_codes(b[s]), a2 = hi_codes(a[s]),
                     a3 = hi_codes(b[s]);
#pragma unroll
      for (int j = 0; j < NT; ++j)
        mma_f16(acc[j], a0, a1, a2, a3, q[j].b[h * 4 + s][0], q[j].b[h * 4 + s][1]);
    }
  }
}

}  // namespace kv8
}  // namespace ea
