// Attention over the 4-bit grouped-query cache for few query rows per kv head: nodes of trees of drafted tokens, BF16.
#include "kv4_attn.cuh"

namespace mlaq {

cudaError_t launch_kv4_decode_tree(const Kv4AttnParams& p, int D, int n_groups, int num_sms, cudaStream_t stream) {
  return p.f16 ? launch_kv4_decode_tree_f16(p, D, n_groups, num_sms, stream) : launch_decode_kernel<true, false>(p, D, n_groups, num_sms, stream);
}

}  // namespace mlaq
