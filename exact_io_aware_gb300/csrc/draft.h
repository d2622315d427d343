// Internal interface of the operators on trees of drafted tokens (draft_api.cu and the kernels).
#pragma once
#include <cuda_runtime.h>

#include <cstdint>
#include <string>

namespace ea {

constexpr int kMostNodes = 1024;  // of a sequence's tree

struct TreeMaskArgs {
  int B, n;
  const int32_t* parents;
  const int32_t* counts;  // null: n nodes in every sequence
  uint32_t* tree;
  uint32_t* status;
};

enum ProbType : int { kProbF32 = 0, kProbF16 = 1, kProbBf16 = 2 };

struct DraftVerifyArgs {
  int type;  // ProbType
  int B, n, V;
  const void* target;
  const void* draft;  // null: drafts that were not drawn
  const int32_t* tokens;
  const int32_t* parents;
  const int32_t* counts;
  const float* uniforms;
  int32_t* path;
  int32_t* accepted;
  int32_t* next_token;
  uint32_t* status;
  int sms;
};

// Each launcher returns 0 or a negative ATTN_ERR_* code and fills `err` on failure.
int launch_tree_mask(const TreeMaskArgs& a, cudaStream_t s, std::string& err);
int launch_draft_verify(const DraftVerifyArgs& a, cudaStream_t s, std::string& err);

}  // namespace ea
