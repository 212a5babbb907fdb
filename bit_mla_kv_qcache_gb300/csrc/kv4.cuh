// Grouped-query K/V cache in 4 bits: page layout, parameter blocks and launchers shared by the C
// ABI layer (abi_kv4.cu) and the kernels.
#pragma once
#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

namespace mlaq {

// Rows of heads with their strides in elements (a head's channels are contiguous).
struct HeadView {
  const uint16_t* data;
  int64_t row_stride, head_stride;
};

// cos / sin tables [n_pos][rot_dim / 2] of the rotation; rot_dim = 0: no rotation.
struct Rotation {
  const float* cos_tab;
  const float* sin_tab;
  int n_pos, rot_dim, interleaved;
};

// One kv head's region of a page: P rows of key codes, P rows of value codes (D / 2 bytes each),
// then per token and group (key scale, key min, value scale, value min) in FP16.
__host__ __device__ constexpr int kv4_head_bytes(int D, int n_groups, int P) { return P * (D + 8 * n_groups); }

struct Kv4AppendParams {
  HeadView k, v, q;  // q.data == nullptr: no queries to rotate
  Rotation rot;
  uint16_t *q_out, *k_deq, *v_deq;  // [rows][heads][D] contiguous, each optional
  const int32_t *cu_new, *seq_lens, *page_table;
  int32_t* seq_next;
  uint8_t* pool;
  int32_t* err;
  int64_t n_pages, page_bytes;
  int B, n_rows, max_new, max_pages, P, p_shift, Hq, Hkv;
  bool f16;  // FP16 rows (else BF16)
  // Nodes of trees of drafted tokens: rotated to tree_base[b] (nullptr: seq_lens[b]) + bits of the row's mask - 1.
  const uint32_t* tree_mask;  // [rows][mask_words], else nullptr
  const int32_t* tree_base;
  int mask_words;  // of 32 bits
};
cudaError_t launch_kv4_append(const Kv4AppendParams& p, int D, int n_groups, cudaStream_t stream);

struct LatentAppendParams {
  HeadView kv;  // [rows][576]
  HeadView q;   // [rows][H][64] positional part of the queries, or data == nullptr
  Rotation rot;
  const uint16_t* weight;  // [512] BF16, or nullptr: no normalization
  float eps;
  uint16_t *q_out, *c_out, *kr_out;  // contiguous, each optional
  const int32_t *cu_new, *seq_lens, *page_table;
  int32_t* seq_next;
  uint16_t* pool;  // [n_pages][P][576] BF16, or nullptr
  int32_t* err;
  int64_t n_pages;
  int B, n_rows, max_new, max_pages, P, p_shift, H;
};
cudaError_t launch_latent_append(const LatentAppendParams& p, cudaStream_t stream);

// An item that several CTAs took: what the kernel that joins its parts has to know. One place for each CTA, that of the item which
// it begins; parts 0: none. A part whose sum is negative is not there (its CTA's wait ran out).
struct Kv4Joined {
  int h, rb, parts, r0, rows;  // kv head, row block, its parts, the sequence's first row, rows (of all heads of the group)
};
struct Kv4AttnParams {
  HeadView q;
  const int32_t* cu_q;  // [B+1], or nullptr: one row per sequence
  const int32_t *page_table, *seq_lens;
  const uint8_t* pool;
  uint16_t* out;  // [rows][Hq][D]
  float* lse;     // [rows][Hq], or nullptr
  int32_t* err;
  uint32_t* arrive;  // one counter per CTA, zero between calls
  float* part_o;     // [2 * CTAs][rows of a block][D] unnormalized partial outputs
  float* part_ml;    // [2 * CTAs][rows of a block][2] partial (max in log2 units, sum)
  Kv4Joined* joined;  // [CTAs], for many rows
  int64_t n_pages, page_bytes;
  float scale_log2;
  int B, n_rows, max_q, Hq, Hkv, G, max_pages, P, p_shift, window;
  bool causal, f16;
  const uint32_t* tree_mask;  // trees of drafted tokens: [rows][mask_words], else nullptr
  const int32_t* tree_base;   // [B] tokens before the tree, or nullptr: all but the sequence's rows
  int mask_words;             // of 32 bits
};
// The workspace begins with one counter per CTA, at the same place for every problem size (a
// workspace may serve calls of different sizes one after the other).
constexpr size_t kKv4CounterBytes = 8192;
// Rows of one work item of the decode kernel (8 or 16) and the CTAs that it launches.
int kv4_decode_rows(int B, int Hkv, int max_q, int G, int64_t max_tokens, int num_sms);  // of a block
int kv4_decode_ctas(int num_sms);
size_t kv4_decode_workspace_bytes(int rows, int D, int num_sms);
cudaError_t launch_kv4_decode(const Kv4AttnParams& p, int D, int n_groups, int num_sms, cudaStream_t stream);
cudaError_t launch_kv4_decode_f16(const Kv4AttnParams& p, int D, int n_groups, int num_sms, cudaStream_t stream);
cudaError_t launch_kv4_decode_tree(const Kv4AttnParams& p, int D, int n_groups, int num_sms, cudaStream_t stream);
cudaError_t launch_kv4_decode_tree_f16(const Kv4AttnParams& p, int D, int n_groups, int num_sms, cudaStream_t stream);

// Tokens base + kept[i] of a sequence move to base + i, i < n_kept, and its length becomes base + n_kept.
struct Kv4KeepParams {
  const int32_t *kept, *n_kept, *tree_base, *page_table;  // kept: [B][max_kept]
  uint8_t* pool;
  int32_t *seq_lens, *err;
  int64_t n_pages, page_bytes;
  int B, max_kept, max_pages, P, p_shift, Hkv;
};
cudaError_t launch_kv4_keep(const Kv4KeepParams& p, int D, int n_groups, cudaStream_t stream);

// More rows than the decode kernel holds go to the fifth-generation tensor cores: 128 rows of
// queries (or two tiles of 128), one CTA per item or, with few items, the items cut over the SMs.
struct Kv4PromptPlan {
  int line;      // 0: one CTA per item; else the row blocks of the longest sequence
  int rows;      // rows of one item
  int64_t ctas;
};
bool kv4_uses_prompt(int max_q, int G);
bool kv4_tree_stays(int B, int Hkv, int max_q, int G, int64_t max_tokens, int D, int num_sms);  // a tree stays with the kernel for few rows
Kv4PromptPlan kv4_prompt_plan(int B, int Hkv, int n_rows, int max_q, int64_t max_tokens, int G, int num_sms);
size_t kv4_prompt_workspace_bytes(const Kv4PromptPlan& z, int D);
cudaError_t launch_kv4_prompt(const Kv4AttnParams& p, const Kv4PromptPlan& z, int D, int n_groups, cudaStream_t stream);
cudaError_t launch_kv4_join(const Kv4AttnParams& p, const Kv4PromptPlan& z, int D, cudaStream_t stream);  // behind it, where items are cut
cudaError_t launch_kv4_prompt_tree_f16(const Kv4AttnParams& p, const Kv4PromptPlan& z, int D, int n_groups, cudaStream_t stream);
cudaError_t launch_kv4_prompt_tree(const Kv4AttnParams& p, const Kv4PromptPlan& z, int D, int n_groups, cudaStream_t stream);

}  // namespace mlaq
