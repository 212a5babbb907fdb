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
  int64_t n_pages, page_bytes;
  float scale_log2;
  int B, n_rows, max_q, Hq, Hkv, G, max_pages, P, p_shift, window;
  bool causal, f16;
};
// The workspace begins with one counter per CTA, at the same place for every problem size (a
// workspace may serve calls of different sizes one after the other).
constexpr size_t kKv4CounterBytes = 8192;
// Rows of one work item of the decode kernel (8 or 16) and the CTAs that it launches.
int kv4_decode_rows(int max_q, int G);
int kv4_decode_ctas(int num_sms);
size_t kv4_decode_workspace_bytes(int rows, int D, int num_sms);
cudaError_t launch_kv4_decode(const Kv4AttnParams& p, int D, int n_groups, int num_sms, cudaStream_t stream);

// More rows than the decode kernel holds go to the fifth-generation tensor cores: 128 rows of
// queries (or two tiles of 128), one CTA per item or, with few items, the items cut over the SMs.
struct Kv4PromptPlan {
  int line;      // 0: one CTA per item; else the row blocks of the longest sequence
  int rows;      // rows of one item
  int64_t ctas;
};
bool kv4_uses_prompt(int max_q, int G);
Kv4PromptPlan kv4_prompt_plan(int B, int Hkv, int n_rows, int max_q, int64_t max_tokens, int G, int num_sms);
size_t kv4_prompt_workspace_bytes(const Kv4PromptPlan& z, int D);
cudaError_t launch_kv4_prompt(const Kv4AttnParams& p, const Kv4PromptPlan& z, int D, int n_groups, cudaStream_t stream);

}  // namespace mlaq
