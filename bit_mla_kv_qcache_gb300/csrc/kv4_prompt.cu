// Attention over the 4-bit grouped-query cache for many query rows per kv head: rows of a sequence's last positions.
#include "kv4_prompt.cuh"

namespace mlaq {

bool kv4_uses_prompt(int max_q, int G) { return static_cast<int64_t>(max_q) * G > 32; }

// An item is worth cutting, which costs a schedule, a second store and a join, when its tokens are many. 48 items
// of 256 rows, one CTA each against cut: 2K tokens 39 and 43 us, 3K 53 and 47, 8K 122 and 72; four of 40 rows: 1K 20 and 25, 2K 30
// and 26. Between a half and all of the SMs whole items fill one wave and a cut makes two (96 items, 8K: 123 and 126 us).
// Up to twice the SMs a cut fills the second wave: 192 items, 4K: 103 and 104, 8K: 215 and 173 us. The lengths are on
// the device: the room of the page table stands for them here, and there short items stay whole.
Kv4PromptPlan kv4_prompt_plan(int B, int Hkv, int n_rows, int max_q, int64_t max_tokens, int G, int num_sms) {
  Kv4PromptPlan z;
  const int64_t rows = static_cast<int64_t>(std::min(max_q, n_rows)) * G;
  z.rows = rows > 128 ? 256 : rows > 64 ? 128 : 64;
  const int64_t items = static_cast<int64_t>(B) * Hkv * ((rows + z.rows - 1) / z.rows);
  const int64_t blocks = (rows + z.rows - 1) / z.rows;
  const bool cut = 2 * items <= num_sms ? max_tokens > 2048 : items > num_sms && items < 2 * num_sms && max_tokens > 4096;
  z.line = cut && B * blocks <= kThreads ? static_cast<int>(blocks) : 0;
  z.ctas = z.line ? std::min(num_sms, static_cast<int>(kKv4CounterBytes / 4)) : items;
  return z;
}

size_t kv4_prompt_workspace_bytes(const Kv4PromptPlan& z, int D) {
  return kKv4CounterBytes + (z.line ? 2 * static_cast<size_t>(z.ctas) * z.rows * (static_cast<size_t>(D) + 2) * sizeof(float) : 0);
}

cudaError_t launch_kv4_prompt(const Kv4AttnParams& p, const Kv4PromptPlan& z, int D, int n_groups, cudaStream_t stream) {
  return launch_prompt_kernel<false>(p, z, D, n_groups, stream);
}

}  // namespace mlaq
