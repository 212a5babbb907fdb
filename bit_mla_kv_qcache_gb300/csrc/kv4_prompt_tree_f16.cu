// As kv4_prompt_tree.cu, for FP16 outputs: weights in two parts.
#include "kv4_prompt.cuh"

namespace mlaq {

cudaError_t launch_kv4_prompt_tree_f16(const Kv4AttnParams& p, const Kv4PromptPlan& z, int D, int n_groups, cudaStream_t stream) {
  return launch_prompt_kernel<true, true>(p, z, D, n_groups, stream);
}

}  // namespace mlaq
