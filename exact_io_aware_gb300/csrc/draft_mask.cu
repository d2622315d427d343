// The words of a tree of drafted tokens: row i has a bit for node i and for each of its ancestors.
//
// One CTA a sequence.  Nodes come after their parents, so a node's ancestors in its own group of 32 are
// found by doubling (the bits of a node and of the node 1, 2, 4 .. steps up), all groups at once, along
// with the first ancestor outside the group; the words below the group's are then that ancestor's row,
// copied group by group.  A walk up the parents instead would take a chain of n nodes n dependent
// reads.  Bound by the launch and a few dependent steps: one tree of 16 nodes 1.6 us, 128 of 256 nodes 3.5 us.
#include <cuda_runtime.h>

#include "draft.h"
#include "kv8_common.cuh"

namespace ea {
namespace draft {

constexpr int kMaskThreads = 256;

__global__ void __launch_bounds__(kMaskThreads)
    tree_mask_kernel(int n, int words, const int32_t* __restrict__ parents, const int32_t* __restrict__ counts,
                     uint32_t* __restrict__ tree, uint32_t* status) {
  extern __shared__ uint32_t rows[];  // [nodes][words], then the first ancestor outside each node's group
  int* out_of = reinterpret_cast<int*>(rows + static_cast<size_t>(words) * 32 * words);
  const int b = blockIdx.x, lane = lane_id();
  const int cnt = kv8::seq_count(counts, b, n);
  parents += static_cast<int64_t>(b) * n;
  tree += static_cast<int64_t>(b) * n * words;
  bool odd = counts && threadIdx.x == 0 && __ldg(counts + b) != cnt;
  const int groups = (cnt + 31) / 32;
  for (int g = warp_id(); g < groups; g += kMaskThreads / 32) {
    const int i = 32 * g + lane;
    int up = i < cnt ? __ldg(parents + i) : -1;
    if (up < -1 || up >= max(i, 0)) {
      odd |= up != -1;
      up = -1;
    }
    uint32_t bits = i < cnt ? 1u << lane : 0u;
    int far = up;  // the ancestor 2^k steps up, or the first outside the group
#pragma unroll
    for (int k = 0; k < 5; ++k) {
      const bool inside = far >= 32 * g;
      const uint32_t more = __shfl_sync(0xFFFFFFFFu, bits, far & 31);
      const int next = __shfl_sync(0xFFFFFFFFu, far, far & 31);
      if (inside) {
        bits |= more;
        far = next;
      }
    }
    rows[i * words + g] = bits;
    out_of[i] = far;
  }
  __syncthreads();
  for (int g = 1; g < groups; ++g) {
    for (int x = threadIdx.x; x < 32 * g; x += kMaskThreads) {
      const int i = 32 * g + x / g, w = x % g, far = out_of[i];
      rows[i * words + w] = far >= 0 && w <= far / 32 ? rows[far * words + w] : 0u;
    }
    __syncthreads();
  }
  for (int x = threadIdx.x; x < n * words; x += kMaskThreads) {
    const int i = x / words, w = x % words;
    tree[x] = i < cnt && w <= i / 32 ? rows[x] : 0u;
  }
  if (odd) raise_clamped(status);
}

}  // namespace draft

int launch_tree_mask(const TreeMaskArgs& a, cudaStream_t s, std::string& err) {
  int words = (a.n + 31) / 32;
  const size_t smem = static_cast<size_t>(words) * 32 * (words + 1) * sizeof(uint32_t);
  static std::atomic<uint64_t> allowed{0};
  constexpr size_t kMost = static_cast<size_t>(kMostNodes) * (kMostNodes / 32 + 1) * sizeof(uint32_t);
  cudaError_t e = kv8::allow_smem(reinterpret_cast<const void*>(draft::tree_mask_kernel), kMost, allowed);
  int n = a.n;
  const int32_t* parents = a.parents;
  const int32_t* counts = a.counts;
  uint32_t* tree = a.tree;
  uint32_t* status = a.status;
  void* args[] = {&n, &words, &parents, &counts, &tree, &status};
  if (e == cudaSuccess)
    e = cudaLaunchKernel(reinterpret_cast<const void*>(draft::tree_mask_kernel), dim3(a.B),
                         dim3(draft::kMaskThreads), args, smem, s);
  if (e != cudaSuccess) {
    err = std::string("tree mask launch: ") + cudaGetErrorString(e);
    return -5;
  }
  return 0;
}

}  // namespace ea
