// C ABI entry points of the verification of drafted tokens (declared in include/mla_qcache.h): host-side validation and
// kernel launches on the caller's stream. No allocation, no synchronization.
#include <cstdint>

#include <cuda_runtime.h>

#include "kernels.cuh"
#include "mla_qcache.h"
#include "verify.cuh"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct Span {
  uintptr_t lo, hi;
};
Span span_of(const void* p, int64_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return {a, a + static_cast<uintptr_t>(bytes)};
}
bool overlap(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }

// What both ways of verifying take; p.B and the pointers of the results are set.
int check(mlaq::VerifyParams& p, const uint64_t* tree_mask, int32_t mask_words, int64_t row_bytes, int64_t target_align) {
  if (p.B < 1 || p.B > (1 << 20) || p.n_rows < 0 || p.n_rows > 0x7fffffff - (1 << 20) || p.vocab < 1 || p.max_rows < 1 ||
      p.max_rows > mlaq::kMaxTreeRows)
    return MLA_QCACHE_ERR_SHAPE;
  if (tree_mask && (mask_words < 1 || mask_words > mlaq::kMaxTreeRows / 64 || p.max_rows > 64 * mask_words)) return MLA_QCACHE_ERR_SHAPE;
  constexpr int64_t kMost = int64_t{1} << 58;  // elements from the first row to the last: far beyond any memory
  if (p.target_stride < 0 || p.target_stride > kMost / (p.n_rows + 1ll) || p.draft_stride < 0 || p.draft_stride > kMost / (p.n_rows + 1ll))
    return MLA_QCACHE_ERR_SHAPE;
  if (!p.cu_rows || !p.kept || !p.new_tokens || !p.n_kept || !p.err || (p.n_rows > 0 && (!p.target || !p.tokens)))
    return MLA_QCACHE_ERR_NULL;
  if (!aligned(p.target, target_align) || !aligned(p.draft, 4) || !aligned(p.tokens, 4) || !aligned(p.cu_rows, 4) ||
      !aligned(tree_mask, 8) || !aligned(p.u_accept, 4) || !aligned(p.u_sample, 4) || !aligned(p.kept, 4) ||
      !aligned(p.new_tokens, 4) || !aligned(p.n_kept, 4) || !aligned(p.err, 4))
    return MLA_QCACHE_ERR_ALIGN;
  const int64_t lists = 4 * static_cast<int64_t>(p.B) * p.max_rows, rows = p.n_rows;
  const Span out[3] = {span_of(p.kept, lists), span_of(p.new_tokens, lists), span_of(p.n_kept, 4 * static_cast<int64_t>(p.B))};
  const int64_t target_bytes = rows ? (rows - 1) * p.target_stride * target_align + row_bytes : 0;
  const Span in[7] = {span_of(p.target, target_bytes),
                      span_of(p.draft, p.draft && rows ? ((rows - 1) * p.draft_stride + p.vocab) * 4 : 0),
                      span_of(p.tokens, 4 * rows),
                      span_of(p.cu_rows, 4 * (static_cast<int64_t>(p.B) + 1)),
                      span_of(tree_mask, tree_mask ? 8 * rows * mask_words : 0),
                      span_of(p.u_accept, p.u_accept ? 4 * rows : 0),
                      span_of(p.u_sample, p.u_sample ? 4 * static_cast<int64_t>(p.B) : 0)};
  for (int i = 0; i < 3; ++i) {
    if (overlap(out[i], span_of(p.err, 4))) return MLA_QCACHE_ERR_SHAPE;
    for (const Span& x : in)
      if (overlap(out[i], x)) return MLA_QCACHE_ERR_SHAPE;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return MLA_QCACHE_ERR_SHAPE;
  }
  if (tree_mask) {  // read as words of 32 bits, the low half of each first
    p.mask = reinterpret_cast<const uint32_t*>(tree_mask);
    p.mask_words = 2 * mask_words;
  }
  return MLA_QCACHE_OK;
}

}  // namespace

extern "C" {

int mla_qcache_verify_sampled(int32_t B, int32_t n_rows, int32_t vocab, const float* target, int64_t target_stride,
                              const float* draft, int64_t draft_stride, const int32_t* tokens, const int32_t* cu_rows,
                              int32_t max_rows, const uint64_t* tree_mask, int32_t mask_words, const float* u_accept,
                              const float* u_sample, int32_t* kept, int32_t* new_tokens, int32_t* n_kept, int32_t* err_word,
                              void* stream) {
  mlaq::VerifyParams p{};
  p.target = target;
  p.draft = draft;
  p.target_stride = target_stride;
  p.draft_stride = draft ? draft_stride : 0;
  p.tokens = tokens;
  p.cu_rows = cu_rows;
  p.u_accept = u_accept;
  p.u_sample = u_sample;
  p.kept = kept;
  p.new_tokens = new_tokens;
  p.n_kept = n_kept;
  p.err = err_word;
  p.B = B;
  p.n_rows = n_rows;
  p.vocab = vocab;
  p.max_rows = max_rows;
  const int st = check(p, tree_mask, mask_words, static_cast<int64_t>(vocab) * 4, 4);
  if (st != MLA_QCACHE_OK) return st;
  if (!u_sample || (n_rows > 0 && !u_accept)) return MLA_QCACHE_ERR_NULL;
  return mlaq::launch_verify_sampled(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MLA_QCACHE_OK : MLA_QCACHE_ERR_CUDA;
}

int mla_qcache_verify_greedy(int32_t B, int32_t n_rows, int32_t vocab, int32_t dtype, const void* logits, int64_t logits_stride,
                             const int32_t* tokens, const int32_t* cu_rows, int32_t max_rows, const uint64_t* tree_mask,
                             int32_t mask_words, int32_t* kept, int32_t* new_tokens, int32_t* n_kept, int32_t* err_word,
                             void* stream) {
  if (dtype != MLA_QCACHE_BF16 && dtype != MLA_QCACHE_FP16 && dtype != MLA_QCACHE_FP32) return MLA_QCACHE_ERR_CONFIG;
  mlaq::VerifyParams p{};
  p.target = logits;
  p.target_stride = logits_stride;
  p.tokens = tokens;
  p.cu_rows = cu_rows;
  p.kept = kept;
  p.new_tokens = new_tokens;
  p.n_kept = n_kept;
  p.err = err_word;
  p.B = B;
  p.n_rows = n_rows;
  p.vocab = vocab;
  p.max_rows = max_rows;
  p.type = dtype;
  const int size = dtype == MLA_QCACHE_FP32 ? 4 : 2;
  const int st = check(p, tree_mask, mask_words, static_cast<int64_t>(vocab) * size, size);
  if (st != MLA_QCACHE_OK) return st;
  return mlaq::launch_verify_greedy(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MLA_QCACHE_OK : MLA_QCACHE_ERR_CUDA;
}

int mla_qcache_tree_mask(int32_t B, int32_t n_rows, const int32_t* parents, const int32_t* cu_rows, int32_t max_rows,
                         int32_t mask_words, uint64_t* mask, int32_t* err_word, void* stream) {
  if (B < 1 || B > (1 << 20) || n_rows < 0 || n_rows > 0x7fffffff - (1 << 20) || mask_words < 1 || mask_words > mlaq::kMaxTreeRows / 64 ||
      max_rows < 1 || max_rows > 64 * mask_words)
    return MLA_QCACHE_ERR_SHAPE;
  if (n_rows == 0) return MLA_QCACHE_OK;
  if (!parents || !cu_rows || !mask || !err_word) return MLA_QCACHE_ERR_NULL;
  if (!aligned(parents, 4) || !aligned(cu_rows, 4) || !aligned(mask, 8) || !aligned(err_word, 4)) return MLA_QCACHE_ERR_ALIGN;
  const Span out = span_of(mask, 8 * static_cast<int64_t>(n_rows) * mask_words);
  if (overlap(out, span_of(parents, 4 * static_cast<int64_t>(n_rows))) || overlap(out, span_of(cu_rows, 4 * (static_cast<int64_t>(B) + 1))) ||
      overlap(out, span_of(err_word, 4)))
    return MLA_QCACHE_ERR_SHAPE;
  mlaq::TreeMaskParams p{};
  p.parents = parents;
  p.cu_rows = cu_rows;
  p.mask = reinterpret_cast<uint32_t*>(mask);
  p.err = err_word;
  p.B = B;
  p.n_rows = n_rows;
  p.max_rows = max_rows;
  p.mask_words = 2 * mask_words;
  return mlaq::launch_tree_mask(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MLA_QCACHE_OK : MLA_QCACHE_ERR_CUDA;
}

}  // extern "C"
