// C ABI entry points of the grouped-query cache in 4 bits and of the append to the paged BF16
// latent cache (declared in include/mla_qcache.h): host-side validation, problem decomposition and
// kernel launches on the caller's stream. No allocation, no synchronization.
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "kernels.cuh"
#include "kv4.cuh"
#include "mla_qcache.h"

namespace {

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int check_kv4(const mla_qcache_kv4_config* c) {
  if (!c) return MLA_QCACHE_ERR_NULL;
  if (c->n_kv_heads < 1 || c->n_kv_heads > 256) return MLA_QCACHE_ERR_CONFIG;
  if (c->head_dim != 64 && c->head_dim != 128) return MLA_QCACHE_ERR_CONFIG;
  if ((c->group != 32 && c->group != 64 && c->group != 128) || c->group > c->head_dim) return MLA_QCACHE_ERR_CONFIG;
  const int P = c->page_size;  // a 16-token tile never straddles pages
  if (P != 16 && P != 32 && P != 64 && P != 128 && P != 256) return MLA_QCACHE_ERR_CONFIG;
  return MLA_QCACHE_OK;
}

int64_t kv4_page_bytes(const mla_qcache_kv4_config* c) {
  return static_cast<int64_t>(c->n_kv_heads) *
         mlaq::kv4_head_bytes(c->head_dim, c->head_dim / c->group, c->page_size);
}

int log2_of(int P) {
  int s = 0;
  while ((1 << s) < P) ++s;
  return s;
}

int sm_count(int* out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return MLA_QCACHE_ERR_CUDA;
  if (cudaDeviceGetAttribute(out, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return MLA_QCACHE_ERR_CUDA;
  return MLA_QCACHE_OK;
}

// Strides of whole 16-byte steps, none negative.
int check_view(const mla_qcache_view* v, mlaq::HeadView* out) {
  if (!v || !v->data) return MLA_QCACHE_ERR_NULL;
  if (v->row_stride < 0 || v->head_stride < 0) return MLA_QCACHE_ERR_SHAPE;
  if (!aligned(v->data, 16) || v->row_stride % 8 || v->head_stride % 8) return MLA_QCACHE_ERR_ALIGN;
  *out = mlaq::HeadView{static_cast<const uint16_t*>(v->data), v->row_stride, v->head_stride};
  return MLA_QCACHE_OK;
}

struct Span {
  uintptr_t lo, hi;
};
Span span_of(const mlaq::HeadView& v, int64_t rows, int64_t heads, int64_t dim) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(v.data);
  return {a, a + 2 * static_cast<uintptr_t>((rows - 1) * v.row_stride + (heads - 1) * v.head_stride + dim)};
}
Span span_of(const void* p, int64_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return {a, a + static_cast<uintptr_t>(bytes)};
}
bool overlap(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }

int check_rotation(const mla_qcache_rotation* r, int max_dim, mlaq::Rotation* out) {
  *out = mlaq::Rotation{nullptr, nullptr, 0, 0, 0};
  if (!r) return MLA_QCACHE_OK;
  if (r->rot_dim < 16 || r->rot_dim % 16 || r->rot_dim > max_dim || r->n_pos < 1) return MLA_QCACHE_ERR_SHAPE;
  if (!r->cos_tab || !r->sin_tab) return MLA_QCACHE_ERR_NULL;
  if (!aligned(r->cos_tab, 16) || !aligned(r->sin_tab, 16)) return MLA_QCACHE_ERR_ALIGN;
  *out = mlaq::Rotation{r->cos_tab, r->sin_tab, r->n_pos, r->rot_dim, r->interleaved ? 1 : 0};
  return MLA_QCACHE_OK;
}

// The arrays that both appends take; n_rows == 0 leaves only the lengths to copy (*done).
int check_append(int32_t B, int32_t n_rows, const int32_t* cu_new, const int32_t* seq_lens, int32_t* seq_next,
                 int32_t max_new, const int32_t* page_table, int32_t max_pages, bool paged, const int32_t* err_word,
                 void* stream, bool* done) {
  *done = false;
  if (B < 1 || B > (1 << 20) || n_rows < 0 || n_rows > 0x7fffffff - (1 << 20)) return MLA_QCACHE_ERR_SHAPE;
  if (seq_next && seq_lens && overlap(span_of(seq_lens, 4 * static_cast<int64_t>(B)), span_of(seq_next, 4 * static_cast<int64_t>(B))))
    return MLA_QCACHE_ERR_SHAPE;
  if (!aligned(cu_new, 4) || !aligned(seq_lens, 4) || !aligned(seq_next, 4) || !aligned(page_table, 4) ||
      !aligned(err_word, 4))
    return MLA_QCACHE_ERR_ALIGN;
  if (n_rows == 0) {
    *done = true;
    if (!seq_next) return MLA_QCACHE_OK;
    if (!seq_lens) return MLA_QCACHE_ERR_NULL;
    return cudaMemcpyAsync(seq_next, seq_lens, static_cast<size_t>(B) * sizeof(int32_t), cudaMemcpyDeviceToDevice,
                           static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? MLA_QCACHE_OK
               : MLA_QCACHE_ERR_CUDA;
  }
  if (max_new < 1 || (paged && max_pages < 1)) return MLA_QCACHE_ERR_SHAPE;
  if (!cu_new || !seq_lens || !err_word || (paged && !page_table)) return MLA_QCACHE_ERR_NULL;
  return MLA_QCACHE_OK;
}

}  // namespace

extern "C" {

int mla_qcache_kv4_config_check(const mla_qcache_kv4_config* cfg) { return check_kv4(cfg); }

size_t mla_qcache_kv4_page_bytes(const mla_qcache_kv4_config* cfg) {
  return check_kv4(cfg) == MLA_QCACHE_OK ? static_cast<size_t>(kv4_page_bytes(cfg)) : 0;
}

int mla_qcache_kv4_append(const mla_qcache_kv4_config* cfg, int32_t dtype, int32_t B, int32_t n_rows,
                          const mla_qcache_view* k_new, const mla_qcache_view* v_new, const int32_t* cu_new,
                          const int32_t* seq_lens, int32_t* seq_lens_next, int32_t max_new,
                          const mla_qcache_rotation* rotation, const mla_qcache_view* q, int32_t n_heads, void* q_out,
                          void* k_deq, void* v_deq, const int32_t* page_table, int32_t max_pages, uint8_t* pool,
                          int64_t n_pages, int32_t* err_word, void* stream) {
  int st = check_kv4(cfg);
  if (st != MLA_QCACHE_OK) return st;
  if (dtype != MLA_QCACHE_BF16 && dtype != MLA_QCACHE_FP16) return MLA_QCACHE_ERR_CONFIG;
  bool done = false;
  st = check_append(B, n_rows, cu_new, seq_lens, seq_lens_next, max_new, page_table, max_pages, true, err_word, stream,
                    &done);
  if (st != MLA_QCACHE_OK || done) return st;
  mlaq::Kv4AppendParams p{};
  const int D = cfg->head_dim;
  if ((st = check_view(k_new, &p.k)) != MLA_QCACHE_OK || (st = check_view(v_new, &p.v)) != MLA_QCACHE_OK ||
      (st = check_rotation(rotation, D, &p.rot)) != MLA_QCACHE_OK)
    return st;
  if ((q == nullptr) != (q_out == nullptr) || !pool) return MLA_QCACHE_ERR_NULL;
  if (n_pages < 1) return MLA_QCACHE_ERR_SHAPE;
  if (q) {
    if (n_heads < 1 || n_heads > 4096) return MLA_QCACHE_ERR_SHAPE;
    if ((st = check_view(q, &p.q)) != MLA_QCACHE_OK) return st;
  }
  if (!aligned(q_out, 16) || !aligned(k_deq, 16) || !aligned(v_deq, 16) || !aligned(pool, 16)) return MLA_QCACHE_ERR_ALIGN;
  // outputs must not overlap the rows that are read, nor each other
  const int64_t kv_bytes = static_cast<int64_t>(n_rows) * cfg->n_kv_heads * D * 2;
  const Span in[3] = {span_of(p.k, n_rows, cfg->n_kv_heads, D), span_of(p.v, n_rows, cfg->n_kv_heads, D),
                      q ? span_of(p.q, n_rows, n_heads, D) : Span{0, 0}};
  const Span out[4] = {q ? span_of(q_out, static_cast<int64_t>(n_rows) * n_heads * D * 2) : Span{0, 0},
                       k_deq ? span_of(k_deq, kv_bytes) : Span{0, 0}, v_deq ? span_of(v_deq, kv_bytes) : Span{0, 0},
                       span_of(pool, n_pages * kv4_page_bytes(cfg))};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 3; ++j)
      if (overlap(out[i], in[j])) return MLA_QCACHE_ERR_SHAPE;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return MLA_QCACHE_ERR_SHAPE;
  }
  p.q_out = static_cast<uint16_t*>(q_out);
  p.k_deq = static_cast<uint16_t*>(k_deq);
  p.v_deq = static_cast<uint16_t*>(v_deq);
  p.cu_new = cu_new;
  p.seq_lens = seq_lens;
  p.seq_next = seq_lens_next;
  p.page_table = page_table;
  p.pool = pool;
  p.err = err_word;
  p.n_pages = n_pages;
  p.page_bytes = kv4_page_bytes(cfg);
  p.B = B;
  p.n_rows = n_rows;
  p.max_new = max_new;
  p.max_pages = max_pages;
  p.P = cfg->page_size;
  p.p_shift = log2_of(p.P);
  p.Hq = q ? n_heads : 0;
  p.Hkv = cfg->n_kv_heads;
  p.f16 = dtype == MLA_QCACHE_FP16;
  const cudaError_t e = mlaq::launch_kv4_append(p, D, D / cfg->group, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MLA_QCACHE_OK : MLA_QCACHE_ERR_CUDA;
}

size_t mla_qcache_kv4_workspace_bytes(const mla_qcache_kv4_config* cfg, int32_t B, int32_t n_heads, int32_t max_q,
                                      int32_t max_pages) {
  if (check_kv4(cfg) != MLA_QCACHE_OK || max_pages < 1 || B < 1 || B > (1 << 20) || n_heads < 1 || n_heads > 4096 ||
      n_heads % cfg->n_kv_heads || max_q < 1)
    return 0;
  int sms = 0;
  if (sm_count(&sms) != MLA_QCACHE_OK) return 0;
  const int G = n_heads / cfg->n_kv_heads, D = cfg->head_dim;
  const size_t few = mlaq::kv4_decode_workspace_bytes(mlaq::kv4_decode_rows(max_q, G), D, sms);
  if (!mlaq::kv4_uses_prompt(max_q, G)) return few;
  // the rows of a call, up to max_q per sequence, decide how it is cut: the most that any needs. What a cut
  // takes goes by the rows of an item (64, 128 or 256) alone; whether it is cut, by the number of row blocks.
  const int64_t max_tokens = static_cast<int64_t>(max_pages) * cfg->page_size;
  size_t most = few;
  for (int i = 0; i < 2 * sms + 3; ++i) {
    const int64_t rows = i == 0 ? 1 : i < 3 ? 64 * i / G + 1 : static_cast<int64_t>(i - 2) * 256 / G + 1;
    if (rows > max_q) break;
    const mlaq::Kv4PromptPlan z = mlaq::kv4_prompt_plan(B, cfg->n_kv_heads, static_cast<int>(rows), max_q, max_tokens, G, sms);
    const size_t w = mlaq::kv4_prompt_workspace_bytes(z, D);
    most = most > w ? most : w;
    if (z.line && z.rows == 256) break;
  }
  return most;
}

int mla_qcache_kv4_attn(const mla_qcache_kv4_config* cfg, int32_t dtype, int32_t B, int32_t n_heads, int32_t n_rows,
                        const mla_qcache_view* q, const int32_t* cu_q, int32_t max_q, const int32_t* page_table,
                        int32_t max_pages, const int32_t* seq_lens, const uint8_t* pool, int64_t n_pages,
                        int32_t causal, int32_t window, float softmax_scale, void* out, float* lse, void* workspace,
                        size_t workspace_bytes, int32_t* err_word, void* stream) {
  int st = check_kv4(cfg);
  if (st != MLA_QCACHE_OK) return st;
  if (dtype != MLA_QCACHE_BF16 && dtype != MLA_QCACHE_FP16) return MLA_QCACHE_ERR_CONFIG;
  const float scale_log2 = static_cast<float>(static_cast<double>(softmax_scale) * 1.4426950408889634074);
  if (B < 1 || B > (1 << 20) || n_heads < 1 || n_heads > 4096 || n_heads % cfg->n_kv_heads || n_rows < 0 ||
      static_cast<int64_t>(n_rows) * n_heads > 0x7fffffff || max_q < 1 || max_pages < 1 || n_pages < 1 || window < 0 ||
      (window > 0 && !causal) || !std::isfinite(scale_log2) ||
      static_cast<int64_t>(max_pages) * cfg->page_size > 0x7ffff000)  // positions and steps are counted in 32 bits
    return MLA_QCACHE_ERR_SHAPE;
  if (!cu_q && (max_q != 1 || n_rows != B)) return MLA_QCACHE_ERR_SHAPE;
  if (n_rows == 0) return MLA_QCACHE_OK;
  mlaq::Kv4AttnParams p{};
  if ((st = check_view(q, &p.q)) != MLA_QCACHE_OK) return st;
  if (!page_table || !seq_lens || !pool || !out || !workspace || !err_word) return MLA_QCACHE_ERR_NULL;
  if (!aligned(cu_q, 4) || !aligned(page_table, 4) || !aligned(seq_lens, 4) || !aligned(pool, 16) || !aligned(out, 16) ||
      !aligned(lse, 4) || !aligned(workspace, 16) || !aligned(err_word, 4))
    return MLA_QCACHE_ERR_ALIGN;
  const int D = cfg->head_dim, G = n_heads / cfg->n_kv_heads;
  const int64_t out_rows = static_cast<int64_t>(n_rows) * n_heads;
  const Span os = span_of(out, out_rows * D * 2);
  if (overlap(os, span_of(p.q, n_rows, n_heads, D)) || (lse && overlap(os, span_of(lse, out_rows * 4))))
    return MLA_QCACHE_ERR_SHAPE;
  int sms = 0;
  if ((st = sm_count(&sms)) != MLA_QCACHE_OK) return st;
  const bool prompt = mlaq::kv4_uses_prompt(max_q, G);
  const mlaq::Kv4PromptPlan plan =
      mlaq::kv4_prompt_plan(B, cfg->n_kv_heads, n_rows, max_q, static_cast<int64_t>(max_pages) * cfg->page_size, G, sms);
  const size_t rows = prompt ? plan.rows : mlaq::kv4_decode_rows(max_q, G);
  const size_t need = prompt ? mlaq::kv4_prompt_workspace_bytes(plan, D)
                             : mlaq::kv4_decode_workspace_bytes(static_cast<int>(rows), D, sms);
  if (workspace_bytes < need) return MLA_QCACHE_ERR_WORKSPACE;
  if (prompt && plan.ctas > 0x7fffffff) return MLA_QCACHE_ERR_SHAPE;
  const size_t ctas = prompt ? (plan.line ? plan.ctas : 0) : mlaq::kv4_decode_ctas(sms);
  p.cu_q = cu_q;
  p.page_table = page_table;
  p.seq_lens = seq_lens;
  p.pool = pool;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.err = err_word;
  p.arrive = static_cast<uint32_t*>(workspace);
  p.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + mlaq::kKv4CounterBytes);
  p.part_ml = p.part_o + 2 * ctas * rows * D;
  p.n_pages = n_pages;
  p.page_bytes = kv4_page_bytes(cfg);
  p.scale_log2 = scale_log2;
  p.B = B;
  p.n_rows = n_rows;
  p.max_q = max_q;
  p.Hq = n_heads;
  p.Hkv = cfg->n_kv_heads;
  p.G = G;
  p.max_pages = max_pages;
  p.P = cfg->page_size;
  p.p_shift = log2_of(p.P);
  p.window = window;
  p.causal = causal != 0;
  p.f16 = dtype == MLA_QCACHE_FP16;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const cudaError_t e = prompt ? mlaq::launch_kv4_prompt(p, plan, D, D / cfg->group, cs)
                               : mlaq::launch_kv4_decode(p, D, D / cfg->group, sms, cs);
  return e == cudaSuccess ? MLA_QCACHE_OK : MLA_QCACHE_ERR_CUDA;
}

int mla_qcache_append_bf16(int32_t B, int32_t n_rows, const uint16_t* kv_new, int64_t kv_row_stride,
                           const int32_t* cu_new, const int32_t* seq_lens, int32_t* seq_lens_next, int32_t max_new,
                           const uint16_t* norm_weight, float norm_eps, const mla_qcache_rotation* rotation,
                           const mla_qcache_view* q_rope, int32_t n_heads, uint16_t* q_out, uint16_t* c_out,
                           uint16_t* kr_out, const int32_t* page_table, int32_t max_pages, int32_t page_size,
                           uint16_t* kv_pool, int64_t n_pages, int32_t* err_word, void* stream) {
  if (page_size != 32 && page_size != 64 && page_size != 128) return MLA_QCACHE_ERR_CONFIG;
  bool done = false;
  int st = check_append(B, n_rows, cu_new, seq_lens, seq_lens_next, max_new, page_table, max_pages, kv_pool != nullptr,
                        err_word, stream, &done);
  if (st != MLA_QCACHE_OK || done) return st;
  mlaq::LatentAppendParams p{};
  const mla_qcache_view kv{kv_new, kv_row_stride, 0};
  if ((st = check_view(&kv, &p.kv)) != MLA_QCACHE_OK ||
      (st = check_rotation(rotation, mlaq::kRope, &p.rot)) != MLA_QCACHE_OK)
    return st;
  if ((q_rope == nullptr) != (q_out == nullptr) || (!kv_pool && !c_out && !kr_out)) return MLA_QCACHE_ERR_NULL;
  if ((kv_pool && n_pages < 1) || !(norm_eps >= 0.f)) return MLA_QCACHE_ERR_SHAPE;
  if (q_rope) {
    if (n_heads < 1 || n_heads > 4096) return MLA_QCACHE_ERR_SHAPE;
    if ((st = check_view(q_rope, &p.q)) != MLA_QCACHE_OK) return st;
  }
  if (!aligned(norm_weight, 16) || !aligned(q_out, 16) || !aligned(c_out, 16) || !aligned(kr_out, 16) ||
      !aligned(kv_pool, 16))
    return MLA_QCACHE_ERR_ALIGN;
  const int64_t rows = n_rows;
  const Span in[2] = {span_of(p.kv, rows, 1, mlaq::kRow),
                      q_rope ? span_of(p.q, rows, n_heads, mlaq::kRope) : Span{0, 0}};
  const Span out[4] = {q_out ? span_of(q_out, rows * n_heads * mlaq::kRope * 2) : Span{0, 0},
                       c_out ? span_of(c_out, rows * mlaq::kLatent * 2) : Span{0, 0},
                       kr_out ? span_of(kr_out, rows * mlaq::kRope * 2) : Span{0, 0},
                       kv_pool ? span_of(kv_pool, n_pages * page_size * mlaq::kRow * 2) : Span{0, 0}};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < 2; ++j)
      if (overlap(out[i], in[j])) return MLA_QCACHE_ERR_SHAPE;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j])) return MLA_QCACHE_ERR_SHAPE;
  }
  p.weight = norm_weight;
  p.eps = norm_eps;
  p.q_out = q_out;
  p.c_out = c_out;
  p.kr_out = kr_out;
  p.cu_new = cu_new;
  p.seq_lens = seq_lens;
  p.seq_next = seq_lens_next;
  p.page_table = page_table;
  p.pool = kv_pool;
  p.err = err_word;
  p.n_pages = n_pages;
  p.B = B;
  p.n_rows = n_rows;
  p.max_new = max_new;
  p.max_pages = kv_pool ? max_pages : 0x7fffffff;
  p.P = page_size;
  p.p_shift = log2_of(page_size);
  p.H = q_rope ? n_heads : 0;
  const cudaError_t e = mlaq::launch_latent_append(p, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? MLA_QCACHE_OK : MLA_QCACHE_ERR_CUDA;
}

}  // extern "C"
