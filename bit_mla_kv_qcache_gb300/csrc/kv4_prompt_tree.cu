// Attention over the 4-bit grouped-query cache for many query rows per kv head: nodes of trees of drafted tokens.
#include "kv4_prompt.cuh"

namespace mlaq {

cudaError_t launch_kv4_prompt_tree(const Kv4AttnParams& p, const Kv4PromptPlan& z, int D, int n_groups, cudaStream_t stream) {
  return p.f16 ? launch_kv4_prompt_tree_f16(p, z, D, n_groups, stream) : launch_prompt_kernel<true, false>(p, z, D, n_groups, stream);
}

}  // namespace mlaq
