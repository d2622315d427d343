// C entry points of the operators on trees of drafted tokens: argument checks and dispatch.
// See include/exactattn.h for the contract.
#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>
#include <string>

#include "draft.h"
#include "entry.h"

namespace {

using ea::entry;
using ea::fail;
using ea::misaligned;
using ea::outcome;
using ea::overlap;

int check_tree(int B, int n, std::initializer_list<const void*> words, const int32_t* counts) {
  if (B < 1 || n < 1) return fail(ATTN_ERR_INVALID_ARG, "B and n must be positive");
  if (n > ea::kMostNodes) return fail(ATTN_ERR_UNSUPPORTED, "n must be at most 1024");
  if (B > (1 << 24)) return fail(ATTN_ERR_UNSUPPORTED, "B must be at most 2^24");
  for (const void* p : words) {
    if (!p) return fail(ATTN_ERR_INVALID_ARG, "null pointer");
    if (misaligned(p, 4)) return fail(ATTN_ERR_ALIGNMENT, "float32 and int32 arrays must be 4-byte aligned");
  }
  if (misaligned(counts, 4)) return fail(ATTN_ERR_ALIGNMENT, "counts must be 4-byte aligned");
  return ATTN_OK;
}

}  // namespace

extern "C" {

int attn_tree_mask(int B, int n, const int32_t* parents, const int32_t* counts, uint32_t* tree,
                   void* stream) {
  return entry("attn_tree_mask", [&]() -> int {
    if (int rc = check_tree(B, n, {parents, tree}, counts)) return rc;
    const size_t seqs = static_cast<size_t>(B) * 4, bytes = seqs * n * ((n + 31) / 32);
    if (overlap(tree, bytes, parents, seqs * n) || (counts && overlap(tree, bytes, counts, seqs)))
      return fail(ATTN_ERR_INVALID_ARG, "tree must not overlap the inputs");
    ea::TreeMaskArgs a{B, n, parents, counts, tree, nullptr};
    if (int rc = ea::device_status_word(&a.status)) return rc;
    std::string err;
    const int rc = ea::launch_tree_mask(a, static_cast<cudaStream_t>(stream), err);
    return outcome(rc, err);
  });
}

int attn_draft_verify(int dtype, int B, int n, int V, const void* target, const void* draft,
                      const int32_t* tokens, const int32_t* parents, const int32_t* counts,
                      const float* uniforms, int32_t* path, int32_t* accepted, int32_t* next_token,
                      void* stream) {
  return entry("attn_draft_verify", [&]() -> int {
    if (dtype < ATTN_F32 || dtype > ATTN_BF16) return fail(ATTN_ERR_INVALID_ARG, "unknown dtype");
    if (int rc = check_tree(B, n, {tokens, parents, uniforms, path, accepted, next_token}, counts)) return rc;
    if (V < 1) return fail(ATTN_ERR_INVALID_ARG, "V must be positive");
    if (V > (1 << 30)) return fail(ATTN_ERR_UNSUPPORTED, "V must be at most 2^30");
    if (!target) return fail(ATTN_ERR_INVALID_ARG, "null pointer");
    if (misaligned(target, 16) || misaligned(draft, 16))
      return fail(ATTN_ERR_ALIGNMENT, "target and draft must be 16-byte aligned");
    const size_t seqs = static_cast<size_t>(B) * 4;
    const size_t probs = static_cast<size_t>(B) * n * V * (dtype == ATTN_F32 ? 4 : 2);
    struct Range { const void* p; size_t n; };
    const Range all[] = {{path, seqs * n}, {accepted, seqs}, {next_token, seqs},
                         {target, probs}, {draft, draft ? probs : 0}, {tokens, seqs * n},
                         {parents, seqs * n}, {counts, counts ? seqs : 0}, {uniforms, seqs * n}};
    for (int i = 0; i < 3; ++i)  // what is written against all that comes after it
      for (int j = i + 1; j < 9; ++j)
        if (all[j].n && overlap(all[i].p, all[i].n, all[j].p, all[j].n))
          return fail(ATTN_ERR_INVALID_ARG, "the outputs must not overlap the inputs or one another");
    const int type = dtype == ATTN_F32 ? ea::kProbF32 : dtype == ATTN_F16 ? ea::kProbF16 : ea::kProbBf16;
    ea::DraftVerifyArgs a{type, B, n, V, target, draft, tokens, parents, counts, uniforms,
                          path, accepted, next_token, nullptr, ea::device_sm_count()};
    if (int rc = ea::device_status_word(&a.status)) return rc;
    std::string err;
    const int rc = ea::launch_draft_verify(a, static_cast<cudaStream_t>(stream), err);
    return outcome(rc, err);
  });
}

}  // extern "C"
