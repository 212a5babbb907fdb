// As kv4_attn_tree.cu, for FP16 rows.
#include "kv4_attn.cuh"

namespace mlaq {

cudaError_t launch_kv4_decode_tree_f16(const Kv4AttnParams& p, int D, int n_groups, int num_sms, cudaStream_t stream) {
  return launch_decode_kernel<true, true>(p, D, n_groups, num_sms, stream);
}

}  // namespace mlaq
