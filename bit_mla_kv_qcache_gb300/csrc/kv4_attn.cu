// Attention over the 4-bit grouped-query cache for few query rows per kv head: rows of a sequence's last positions, BF16.
#include "kv4_attn.cuh"

namespace mlaq {

// 9 to 32 rows in blocks of eight, as long as these are few and short: the blocks of a head read its tokens each for itself, but
// eight warps go through a block of eight at twice the pace, there are more parts to share out, and less to join. Blocks of eight and
// of 16, 8 kv heads, D = 128: 32 rows of one sequence, 1K tokens 10.5 and 16.7 us, 4K 13.8 and 20.2, 16K 25.0 and 31.3; of four, 4K 26.2
// and 28.6, 8K 42.4 and 42.3, 16K 73.6 and 67.9; of eight, 2K 24.0 and 28.4, 8K 71.5 and 68.0. 16 rows of eight, 2K 18.1 and 21.8, 16K
// 73.3 and 68.2; of 32, 1K 36.2 and 25.7 (more blocks than CTAs). The lengths are on the device: the room of the page table stands for them.
int kv4_decode_rows(int B, int Hkv, int max_q, int G, int64_t max_tokens, int num_sms) {
  const int64_t rows = static_cast<int64_t>(max_q) * G, items = (rows + 7) / 8 * B * Hkv;
  return rows <= 8 || (items <= kv4_decode_ctas(num_sms) && items * max_tokens <= (1 << 20)) ? 8 : 16;
}
// Trees of 33 to 128 rows stay here where their blocks of eight are few and short: the kernel for many rows starts and ends for ~18 us.
// Here and there, 8 kv heads, D = 128: 40 rows of one sequence, 1K tokens 12.0 and 22.6 us, 8K 19.4 and 22.9, 16K 29.2 and 27.3; 64 rows
// of one, 4K 18.1 and 21.9, 8K 26.2 and 23.2; of four, 1K 16.6 and 23.6, 2K 24.0 and 22.7; 128 rows of one, 2K 18.1 and 24.7, 4K 26.2 and
// 25.4 (of these the bound leaves 40 rows at 8K, 64 at 8K, four times 64 at 2K and 128 at 4K to the other). 56 rows on 2 heads, D = 64: one sequence of 16K 14.0 and 22.3, four of 8K 18.2 and 20.4, eight of 4K 20.1 and 19.7.
bool kv4_tree_stays(int B, int Hkv, int max_q, int G, int64_t max_tokens, int D, int num_sms) {
  const int64_t rows = static_cast<int64_t>(max_q) * G, items = (rows + 7) / 8 * B * Hkv;
  return rows <= 128 && items <= kv4_decode_ctas(num_sms) && items * max_tokens * D <= (9 << 22);
}
int kv4_decode_ctas(int num_sms) { return std::min(2 * num_sms, static_cast<int>(kKv4CounterBytes / 4)); }
size_t kv4_decode_workspace_bytes(int rows, int D, int num_sms) {
  const size_t ctas = kv4_decode_ctas(num_sms);
  return kKv4CounterBytes + 2 * ctas * rows * (static_cast<size_t>(D) + 2) * sizeof(float);
}

cudaError_t launch_kv4_decode(const Kv4AttnParams& p, int D, int n_groups, int num_sms, cudaStream_t stream) {
  return p.f16 ? launch_kv4_decode_f16(p, D, n_groups, num_sms, stream) : launch_decode_kernel<false, false>(p, D, n_groups, num_sms, stream);
}

}  // namespace mlaq
