// Verification of drafted tokens: parameter blocks and launchers shared by the C ABI layer (abi_tree.cu) and the kernels.
#pragma once
#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

namespace mlaq {

constexpr int kMaxTreeRows = 256;  // nodes of a tree, at most: four words of 64 bits in its masks

struct VerifyParams {
  const void* target;   // [rows][vocab] probabilities (float32), or logits of `type`
  const float* draft;   // [rows][vocab], or nullptr: the drafts were picked without chance
  int64_t target_stride, draft_stride;  // elements from row to row
  const int32_t *tokens, *cu_rows;
  const uint32_t* mask;  // [rows][mask_words], or nullptr: every row's parent is the row before it
  const float *u_accept, *u_sample;
  int32_t *kept, *new_tokens, *n_kept;
  int32_t* err;
  int B, n_rows, vocab, max_rows, mask_words, type;
};
cudaError_t launch_verify_sampled(const VerifyParams& p, cudaStream_t stream);
cudaError_t launch_verify_greedy(const VerifyParams& p, cudaStream_t stream);

// Masks [rows][mask_words] of rows whose parents are given.
struct TreeMaskParams {
  const int32_t *parents, *cu_rows;
  uint32_t* mask;
  int32_t* err;
  int B, n_rows, max_rows, mask_words;
};
cudaError_t launch_tree_mask(const TreeMaskParams& p, cudaStream_t stream);

}  // namespace mlaq
