// What the attention kernels know of a tree of drafted tokens: the tokens from the base on are its nodes, node j at base + j. A
// row's mask names the nodes that it sees (its ancestors and itself); its position, for a sliding window, is as many tokens
// behind the base as that are.
#pragma once
#include <cstdint>

#include "kernels.cuh"
#include "kv4.cuh"

namespace mlaq {

// Tokens before sequence b's tree; out of [0, T]: the sequence is read as empty.
__device__ __forceinline__ int tree_base(const Kv4AttnParams& p, int b, int& T, int n, int& flags) {
  const int base = p.tree_base ? __ldg(p.tree_base + b) : T - n;
  if (base < 0 || base > T) {
    flags |= kErrSeqOverflow;
    T = 0;
    return 0;
  }
  return base;
}

// Tokens that some row may see: [x, y). A row sees at least one node, or none and then is placed one before the base.
__device__ __forceinline__ int2 tree_tokens(const Kv4AttnParams& p, int T, int base) {
  const int end = static_cast<int>(min(static_cast<int64_t>(T), static_cast<int64_t>(base) + 32 * p.mask_words));
  return make_int2(p.window && base > p.window ? base - p.window : 0, end);
}
// Tokens that every row sees: [x, y). A row is placed at most as many tokens behind the base as its mask has bits.
__device__ __forceinline__ int2 tree_tokens_of_all(const Kv4AttnParams& p, int T, int base) {
  const int64_t lo = p.window ? static_cast<int64_t>(base) + 32 * p.mask_words - p.window : 0;
  return make_int2(static_cast<int>(max(min(lo, static_cast<int64_t>(base)), static_cast<int64_t>(0))), base);
}

// Which of the tokens first .. first + 31 row r of the call sees.
__device__ __forceinline__ uint32_t tree_bits(const Kv4AttnParams& p, int r, int T, int base, int first) {
  const uint32_t* const mask = p.tree_mask + static_cast<size_t>(r) * p.mask_words;
  const int k = first - base;  // the first token's node; those below 0 stand before the tree
  uint32_t bits = ~0u;
  if (k > -32) {
    const int i = k >> 5;
    const uint32_t lo = i < 0 ? ~0u : i < p.mask_words ? __ldg(mask + i) : 0u;
    const uint32_t hi = i + 1 < p.mask_words ? __ldg(mask + i + 1) : 0u;
    bits = __funnelshift_r(lo, hi, k & 31);
  }
  if (T - first < 32) bits &= T > first ? (1u << (T - first)) - 1u : 0u;
  if (p.window && k < 0) {
    int seen = 0;
    for (int i = 0; i < p.mask_words; ++i) seen += __popc(__ldg(mask + i));
    const int64_t lo = min(static_cast<int64_t>(base), static_cast<int64_t>(base) + seen - p.window) - first;
    if (lo >= 32) bits = 0;
    else if (lo > 0) bits &= ~0u << lo;
  }
  return bits;
}

}  // namespace mlaq
