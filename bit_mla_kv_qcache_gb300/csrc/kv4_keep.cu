// The accepted nodes of a tree of drafted tokens move to the places behind the tokens before it, in the 4-bit grouped-query cache.
//
// A CTA takes one kv head of a sequence. Nodes move towards the front past one another's places, so all that it moves is read
// into registers (at most 256 tokens of 64 + 64 + 32 bytes) before anything is stored: one barrier, no scratch memory, and no
// order among CTAs, whose heads lie apart. Bound: three dependent loads (the lists, page ids, tokens) and a store.
#include "append.cuh"
#include "kernels.cuh"
#include "kv4.cuh"
#include "verify.cuh"

namespace mlaq {
namespace {

constexpr int kThreads = 256;
static_assert(kThreads == kMaxTreeRows, "a thread to a node");

template <int D, int NG>
__global__ void __launch_bounds__(kThreads) kv4_keep_kernel(const Kv4KeepParams p) {
  __shared__ int64_t s_from[kMaxTreeRows], s_to[kMaxTreeRows];  // page and token as one number, -1: the token stays
  const int tid = threadIdx.x, b = static_cast<int>(blockIdx.x) / p.Hkv, h = static_cast<int>(blockIdx.x) - b * p.Hkv;
  const int n = __ldg(p.n_kept + b), base = __ldg(p.tree_base + b);
  int mine = -1, before = -1;
  if (tid < p.max_kept) {
    mine = __ldg(p.kept + static_cast<size_t>(b) * p.max_kept + tid);
    if (tid > 0) before = __ldg(p.kept + static_cast<size_t>(b) * p.max_kept + tid - 1);
  }
  const int64_t room = static_cast<int64_t>(p.max_pages) << p.p_shift;
  int flags = 0;
  if (n < 0 || n > p.max_kept) {
    flags = kErrRows;
  } else if (base < 0) {
    flags = kErrSeqOverflow;
  } else if (tid < n) {
    if (mine <= before || mine < 0) flags = kErrRows;
    if (static_cast<int64_t>(base) + max(mine, tid) >= room) flags |= kErrSeqOverflow;
  }
  if (base >= 0 && base > room) flags |= kErrSeqOverflow;
  const int bad = __syncthreads_or(flags);
  if (bad) {  // the sequence stays as it is
    if (h == 0 && flags) atomicOr(p.err, flags);
    return;
  }
  if (tid < n) {
    int64_t from = -1, to = -1;
    if (mine != tid) {
      const int32_t* table = p.page_table + static_cast<size_t>(b) * p.max_pages;
      const int32_t x = __ldg(table + ((base + mine) >> p.p_shift)), y = __ldg(table + ((base + tid) >> p.p_shift));
      if (x >= 0 && x < p.n_pages && y >= 0 && y < p.n_pages) {
        from = (static_cast<int64_t>(x) << p.p_shift) + ((base + mine) & (p.P - 1));
        to = (static_cast<int64_t>(y) << p.p_shift) + ((base + tid) & (p.P - 1));
      } else {
        flags |= kErrBadPage;
      }
    }
    s_from[tid] = from;
    s_to[tid] = to;
  }
  if (h == 0 && flags) atomicOr(p.err, flags);
  if (h == 0 && tid == 0) p.seq_lens[b] = base + n;
  __syncthreads();
  constexpr int kChunks = D / 16;  // 16-byte chunks of a token: keys, then values
  constexpr int kMost = kChunks * kMaxTreeRows / kThreads, kNumbers = NG * kMaxTreeRows / kThreads;
  const int64_t region = static_cast<int64_t>(h) * kv4_head_bytes(D, NG, p.P);
  auto chunk_at = [&](int64_t at, int c) {
    const int64_t t = at & (p.P - 1);
    return reinterpret_cast<uint4*>(p.pool + (at >> p.p_shift) * p.page_bytes + region + (c >= kChunks / 2 ? p.P * (D / 2) : 0) + t * (D / 2)) +
           c % (kChunks / 2);
  };
  auto numbers_at = [&](int64_t at, int g) {
    return reinterpret_cast<uint2*>(p.pool + (at >> p.p_shift) * p.page_bytes + region + p.P * D + (at & (p.P - 1)) * (8 * NG)) + g;
  };
  uint4 x[kMost];
  uint2 y[kNumbers];
#pragma unroll
  for (int k = 0; k < kMost; ++k) {
    const int e = tid + k * kThreads, i = e / kChunks;
    if (i < n && s_from[i] >= 0) x[k] = *chunk_at(s_from[i], e % kChunks);
  }
#pragma unroll
  for (int k = 0; k < kNumbers; ++k) {
    const int e = tid + k * kThreads, i = e / NG;
    if (i < n && s_from[i] >= 0) y[k] = *numbers_at(s_from[i], e % NG);
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kMost; ++k) {
    const int e = tid + k * kThreads, i = e / kChunks;
    if (i < n && s_to[i] >= 0) *chunk_at(s_to[i], e % kChunks) = x[k];
  }
#pragma unroll
  for (int k = 0; k < kNumbers; ++k) {
    const int e = tid + k * kThreads, i = e / NG;
    if (i < n && s_to[i] >= 0) *numbers_at(s_to[i], e % NG) = y[k];
  }
}

template <int D, int NG>
cudaError_t launch(const Kv4KeepParams& p, cudaStream_t stream) {
  kv4_keep_kernel<D, NG><<<static_cast<unsigned>(p.B) * p.Hkv, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv4_keep(const Kv4KeepParams& p, int D, int n_groups, cudaStream_t stream) {
  if (D == 128) {
    if (n_groups == 1) return launch<128, 1>(p, stream);
    if (n_groups == 2) return launch<128, 2>(p, stream);
    return launch<128, 4>(p, stream);
  }
  return n_groups == 1 ? launch<64, 1>(p, stream) : launch<64, 2>(p, stream);
}

}  // namespace mlaq
