// Attention over the 4-bit grouped-query cache for few query rows per kv head: rows of a sequence's last positions.
#include "kv4_attn.cuh"

namespace mlaq {

int kv4_decode_rows(int max_q, int G) { return static_cast<int64_t>(max_q) * G <= 8 ? 8 : 16; }
int kv4_decode_ctas(int num_sms) { return std::min(2 * num_sms, static_cast<int>(kKv4CounterBytes / 4)); }
size_t kv4_decode_workspace_bytes(int rows, int D, int num_sms) {
  const size_t ctas = kv4_decode_ctas(num_sms);
  return kKv4CounterBytes + 2 * ctas * rows * (static_cast<size_t>(D) + 2) * sizeof(float);
}

cudaError_t launch_kv4_decode(const Kv4AttnParams& p, int D, int n_groups, int num_sms, cudaStream_t stream) {
  return launch_decode_kernel<false>(p, D, n_groups, num_sms, stream);
}

}  // namespace mlaq
