// Native argument marshalling for the entry points that a decode step calls once per layer: checks of
// the tensors, their pointers, the current stream, the C ABI call. From Python each of these costs
// 20-30 us a call (a dozen attributes per tensor and ctypes conversions), more than the kernels take.
//
// Functions take positional arguments only (binding.py has the keywords and the documentation) and
// return the C ABI's status; a tensor of the wrong kind raises QCacheError, one of the wrong shape
// ValueError, as in binding.py.
#include <Python.h>

#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <initializer_list>
#include <string>

#include "mla_qcache.h"

namespace {

PyObject* g_error = nullptr;  // QCacheError

struct Raised {};  // a Python error is set

[[noreturn]] void raise(PyObject* type, const std::string& what) {
  PyErr_SetString(type, what.c_str());
  throw Raised{};
}
PyObject* error_type() { return g_error ? g_error : PyExc_RuntimeError; }

std::string shape_of(const at::Tensor& t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + ")";
}

int32_t as_bool(PyObject* o) {
  const int v = PyObject_IsTrue(o);
  if (v < 0) throw Raised{};  // a tensor of several values, for one
  return v;
}

// The tensors of one call: on one device, which is the current one.
struct Call {
  c10::Device device{c10::kCPU};

  const at::Tensor& tensor(PyObject* o, const char* name) const {
    if (o == Py_None) raise(error_type(), std::string(name) + " is required");
    if (!THPVariable_Check(o)) raise(PyExc_TypeError, std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
  }
  // The first tensor sets the device.
  const at::Tensor& lead(PyObject* o, const char* name) {
    const at::Tensor& t = tensor(o, name);
    if (!t.is_cuda()) raise(error_type(), std::string(name) + " must be a CUDA tensor");
    device = t.device();
    const int current = c10::cuda::current_device();
    if (device.index() != current)
      raise(error_type(), std::string(name) + " is on " + device.str() + ", the current device is cuda:" + std::to_string(current));
    return t;
  }
  // A contiguous tensor of this type and shape (-1: any extent).
  const at::Tensor& plain(PyObject* o, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape) const {
    const at::Tensor& t = tensor(o, name);
    if (t.device() != device) raise(error_type(), std::string(name) + " must be on " + device.str() + ", got " + t.device().str());
    if (t.scalar_type() != type)
      raise(error_type(), std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
    bool same = t.dim() == static_cast<int64_t>(shape.size());
    int64_t i = 0;
    if (same)
      for (const int64_t n : shape) same = same && (n < 0 || t.size(i) == n), ++i;
    if (!same) {
      std::string want;
      for (const int64_t n : shape) want += (want.empty() ? "" : ", ") + (n < 0 ? std::string("any") : std::to_string(n));
      raise(PyExc_ValueError, std::string(name) + " must be [" + want + "], got " + shape_of(t));
    }
    if (!t.is_contiguous()) raise(error_type(), std::string(name) + " must be contiguous");
    return t;
  }
  void* ptr(PyObject* o, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape) const {
    return plain(o, name, type, shape).data_ptr();
  }
  void* optional(PyObject* o, const char* name, at::ScalarType type, std::initializer_list<int64_t> shape) const {
    return o == Py_None ? nullptr : ptr(o, name, type, shape);
  }
  // Rows of heads [rows, heads, dim], channels contiguous; heads < 0: any number.
  mla_qcache_view view(PyObject* o, const char* name, at::ScalarType type, int64_t rows, int64_t heads, int64_t dim) const {
    const at::Tensor& t = tensor(o, name);
    if (t.device() != device || t.scalar_type() != type)
      raise(error_type(), std::string(name) + " must be " + c10::toString(type) + " on " + device.str() + ", got " +
                              c10::toString(t.scalar_type()) + " on " + t.device().str());
    if (t.dim() != 3 || t.size(0) != rows || t.size(2) != dim || (heads >= 0 && t.size(1) != heads))
      raise(PyExc_ValueError, std::string(name) + " must be [" + std::to_string(rows) + ", " +
                                  (heads >= 0 ? std::to_string(heads) : "heads") + ", " + std::to_string(dim) + "], got " + shape_of(t));
    if (t.numel() > 0 && t.stride(2) != 1) raise(error_type(), std::string(name) + ": the channels of a head must be contiguous");
    return {t.data_ptr(), rows > 1 ? t.stride(0) : 0, t.size(1) > 1 ? t.stride(1) : 0};
  }
  // cos and sin tables [positions, rot_dim / 2]; false: no rotation.
  bool rotation(PyObject* cos, PyObject* sin, PyObject* interleaved, mla_qcache_rotation* out) const {
    if (cos == Py_None && sin == Py_None) return false;
    if (cos == Py_None || sin == Py_None) raise(PyExc_ValueError, "cos and sin must both be [positions, rot_dim / 2] tables");
    const at::Tensor& c = plain(cos, "cos", at::kFloat, {-1, -1});
    const void* s = ptr(sin, "sin", at::kFloat, {c.size(0), c.size(1)});
    if (c.size(0) > INT32_MAX || c.size(1) > INT32_MAX / 2) raise(PyExc_ValueError, "cos: too large a table");
    *out = {static_cast<const float*>(c.data_ptr()), static_cast<const float*>(s), static_cast<int32_t>(c.size(0)),
            static_cast<int32_t>(2 * c.size(1)), as_bool(interleaved)};
    return true;
  }
  // Masks [rows] or [rows, words] of trees of drafted tokens; false: none.
  bool tree(PyObject* mask, PyObject* base, int64_t rows, int64_t B, mla_qcache_tree* out) const {
    if (mask == Py_None) {
      if (base != Py_None) raise(PyExc_ValueError, "tree_base needs a tree_mask");
      return false;
    }
    const at::Tensor& m = tensor(mask, "tree_mask");
    if (m.dim() == 1) plain(mask, "tree_mask", at::kLong, {rows});
    else plain(mask, "tree_mask", at::kLong, {rows, -1});
    const int64_t words = m.dim() == 1 ? 1 : m.size(1);
    if (words > INT32_MAX) raise(PyExc_ValueError, "tree_mask: too many words");
    *out = {static_cast<const uint64_t*>(m.data_ptr()), static_cast<int32_t>(words),
            static_cast<const int32_t*>(optional(base, "tree_base", at::kInt, {B}))};
    return true;
  }
  // Rows [rows, any] with contiguous entries, strided from row to row.
  const at::Tensor& strided(PyObject* o, const char* name, at::ScalarType type, int64_t rows, int64_t width) const {
    const at::Tensor& t = tensor(o, name);
    if (t.device() != device || t.scalar_type() != type)
      raise(error_type(), std::string(name) + " must be " + c10::toString(type) + " on " + device.str() + ", got " +
                              c10::toString(t.scalar_type()) + " on " + t.device().str());
    if (t.dim() != 2 || (rows >= 0 && t.size(0) != rows) || (width >= 0 && t.size(1) != width))
      raise(PyExc_ValueError, std::string(name) + " must be [rows, vocab], got " + shape_of(t));
    if (t.numel() > 0 && t.size(1) > 1 && t.stride(1) != 1) raise(error_type(), std::string(name) + ": the entries of a row must be contiguous");
    return t;
  }
  void* stream(PyObject* o) const {
    if (o != Py_None) {
      void* p = PyLong_AsVoidPtr(o);
      if (PyErr_Occurred()) throw Raised{};
      return p;
    }
    return c10::cuda::getCurrentCUDAStream(device.index()).stream();
  }
};

int32_t as_int(PyObject* o, const char* name) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Raised{};
  if (v < INT32_MIN || v > INT32_MAX) raise(PyExc_ValueError, std::string(name) + " does not fit 32 bits");
  return static_cast<int32_t>(v);
}
float as_float(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Raised{};
  return static_cast<float>(v);
}
int32_t extent(int64_t n, const char* name) {
  if (n > INT32_MAX) raise(PyExc_ValueError, std::string(name) + " is too large");
  return static_cast<int32_t>(n);
}
int32_t row_type(const at::Tensor& t, const char* name) {
  if (t.scalar_type() == at::kBFloat16) return MLA_QCACHE_BF16;
  if (t.scalar_type() == at::kHalf) return MLA_QCACHE_FP16;
  raise(error_type(), std::string(name) + " must be bfloat16 or float16, got " + c10::toString(t.scalar_type()));
}

// The mla_qcache_kv4_config behind a ctypes structure.
struct Config {
  Py_buffer buf{};
  const mla_qcache_kv4_config* p = nullptr;
  explicit Config(PyObject* o) {
    if (PyObject_GetBuffer(o, &buf, PyBUF_SIMPLE) != 0) throw Raised{};
    if (buf.len != static_cast<Py_ssize_t>(sizeof(mla_qcache_kv4_config))) {
      PyBuffer_Release(&buf);
      raise(PyExc_TypeError, "cfg must be a KV4Config");
    }
    p = static_cast<const mla_qcache_kv4_config*>(buf.buf);
  }
  ~Config() { PyBuffer_Release(&buf); }
  Config(const Config&) = delete;
};

template <typename F>
PyObject* guarded(PyObject* const* a, Py_ssize_t got, Py_ssize_t want, F f) {
  if (got != want) {
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, got);
    return nullptr;
  }
  try {
    return PyLong_FromLong(f(a));
  } catch (const Raised&) {
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
  }
  return nullptr;
}

PyObject* kv4_append(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(args, n, 20, [](PyObject* const* a) {
    const Config cfg(a[0]);
    const int64_t Hkv = cfg.p->n_kv_heads, D = cfg.p->head_dim;
    Call c;
    const at::Tensor& k = c.lead(a[1], "k_new");
    const at::ScalarType type = k.scalar_type();
    const int32_t dtype = row_type(k, "k_new");
    if (k.dim() != 3) raise(PyExc_ValueError, "k_new must be [rows, kv heads, D], got " + shape_of(k));
    const int64_t rows = k.size(0);
    const mla_qcache_view kv = c.view(a[1], "k_new", type, rows, Hkv, D), vv = c.view(a[2], "v_new", type, rows, Hkv, D);
    const at::Tensor& lens = c.plain(a[4], "seq_lens", at::kInt, {-1});
    const int64_t B = lens.size(0);
    const void* cu = c.ptr(a[3], "cu_new", at::kInt, {B + 1});
    const int32_t max_new = as_int(a[5], "max_new");
    const at::Tensor& table = c.plain(a[6], "page_table", at::kInt, {B, -1});
    const at::Tensor& pool = c.plain(a[7], "pool", at::kByte, {-1, static_cast<int64_t>(mla_qcache_kv4_page_bytes(cfg.p))});
    void* err = c.ptr(a[8], "err_word", at::kInt, {1});
    mla_qcache_rotation rot;
    const bool rotated = c.rotation(a[9], a[10], a[11], &rot);
    if ((a[12] == Py_None) != (a[13] == Py_None)) raise(error_type(), "q and q_out go together");
    mla_qcache_view qv{};
    int64_t heads = 0;
    void* q_out = nullptr;
    if (a[12] != Py_None) {
      qv = c.view(a[12], "q", type, rows, -1, D);
      heads = THPVariable_Unpack(a[12]).size(1);
      q_out = c.ptr(a[13], "q_out", type, {rows, heads, D});
    }
    void* k_deq = c.optional(a[14], "k_deq", type, {rows, Hkv, D});
    void* v_deq = c.optional(a[15], "v_deq", type, {rows, Hkv, D});
    void* next = c.optional(a[16], "seq_lens_next", at::kInt, {B});
    const bool in_place = next && next == lens.data_ptr();
    mla_qcache_tree tree{};
    const bool of_tree = c.tree(a[18], a[19], rows, B, &tree);
    void* stream = c.stream(a[17]);
    const int32_t* const cu32 = static_cast<const int32_t*>(cu);
    const int32_t* const lens32 = static_cast<const int32_t*>(lens.data_ptr());
    int32_t* const next32 = in_place ? nullptr : static_cast<int32_t*>(next);
    const int32_t* const table32 = static_cast<const int32_t*>(table.data_ptr());
    const int32_t pages = extent(table.size(1), "page_table");
    uint8_t* const bytes = static_cast<uint8_t*>(pool.data_ptr());
    const int status =
        of_tree ? mla_qcache_kv4_append_tree(cfg.p, dtype, extent(B, "B"), extent(rows, "rows"), &kv, &vv, cu32, lens32, next32, max_new,
                                             rotated ? &rot : nullptr, q_out ? &qv : nullptr, extent(heads, "heads"), q_out, k_deq,
                                             v_deq, table32, pages, bytes, pool.size(0), &tree, static_cast<int32_t*>(err), stream)
                : mla_qcache_kv4_append(cfg.p, dtype, extent(B, "B"), extent(rows, "rows"), &kv, &vv, cu32, lens32, next32, max_new,
                                        rotated ? &rot : nullptr, q_out ? &qv : nullptr, extent(heads, "heads"), q_out, k_deq, v_deq,
                                        table32, pages, bytes, pool.size(0), static_cast<int32_t*>(err), stream);
    if (status != MLA_QCACHE_OK || !in_place) return status;
    return mla_qcache_advance(static_cast<const int32_t*>(cu), static_cast<int32_t*>(lens.data_ptr()), extent(B, "B"), stream);
  });
}

// With a tree (kv4_attn_tree) the arguments 12 .. 14 are its mask and base and the window, else causal and the window.
template <bool kTree>
int attn(PyObject* const* a) {
  const Config cfg(a[0]);
  const int64_t D = cfg.p->head_dim;
  Call c;
  const at::Tensor& q = c.lead(a[1], "q");
  const at::ScalarType type = q.scalar_type();
  const int32_t dtype = row_type(q, "q");
  if (q.dim() != 3) raise(PyExc_ValueError, "q must be [rows, heads, D], got " + shape_of(q));
  const int64_t rows = q.size(0), heads = q.size(1);
  const mla_qcache_view qv = c.view(a[1], "q", type, rows, heads, D);
  const at::Tensor& lens = c.plain(a[3], "seq_lens", at::kInt, {-1});
  const int64_t B = lens.size(0);
  const at::Tensor& table = c.plain(a[2], "page_table", at::kInt, {B, -1});
  const at::Tensor& pool = c.plain(a[4], "pool", at::kByte, {-1, static_cast<int64_t>(mla_qcache_kv4_page_bytes(cfg.p))});
  const float scale = as_float(a[5]);
  void* out = c.ptr(a[6], "out", type, {rows, heads, D});
  const at::Tensor& ws = c.plain(a[7], "workspace", at::kByte, {-1});
  int32_t* const err = static_cast<int32_t*>(c.ptr(a[8], "err_word", at::kInt, {1}));
  const int32_t* const cu = static_cast<const int32_t*>(c.optional(a[9], "cu_q", at::kInt, {B + 1}));
  float* const lse = static_cast<float*>(c.optional(a[11], "lse", at::kFloat, {rows, heads}));
  const int32_t* const table32 = static_cast<const int32_t*>(table.data_ptr());
  const int32_t* const lens32 = static_cast<const int32_t*>(lens.data_ptr());
  const uint8_t* const bytes = static_cast<const uint8_t*>(pool.data_ptr());
  const int32_t pages = extent(table.size(1), "page_table"), max_q = as_int(a[10], "max_q");
  if constexpr (kTree) {
    mla_qcache_tree tree{};
    if (!c.tree(a[12], a[13], rows, B, &tree)) raise(error_type(), "tree_mask is required");
    return mla_qcache_kv4_attn_tree(cfg.p, dtype, extent(B, "B"), extent(heads, "heads"), extent(rows, "rows"), &qv, cu, max_q, &tree,
                                    table32, pages, lens32, bytes, pool.size(0), as_int(a[14], "window"), scale, out, lse,
                                    ws.data_ptr(), static_cast<size_t>(ws.size(0)), err, c.stream(a[15]));
  }
  return mla_qcache_kv4_attn(cfg.p, dtype, extent(B, "B"), extent(heads, "heads"), extent(rows, "rows"), &qv, cu, max_q, table32,
                             pages, lens32, bytes, pool.size(0), as_bool(a[12]), as_int(a[13], "window"), scale, out, lse,
                             ws.data_ptr(), static_cast<size_t>(ws.size(0)), err, c.stream(a[14]));
}
PyObject* kv4_attn(PyObject*, PyObject* const* args, Py_ssize_t n) { return guarded(args, n, 15, attn<false>); }
PyObject* kv4_attn_tree(PyObject*, PyObject* const* args, Py_ssize_t n) { return guarded(args, n, 16, attn<true>); }

PyObject* kv4_keep(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(args, n, 9, [](PyObject* const* a) {
    const Config cfg(a[0]);
    Call c;
    const at::Tensor& kept = c.lead(a[1], "kept");
    c.plain(a[1], "kept", at::kInt, {-1, -1});
    const int64_t B = kept.size(0);
    const void* count = c.ptr(a[2], "n_kept", at::kInt, {B});
    const void* base = c.ptr(a[3], "tree_base", at::kInt, {B});
    const at::Tensor& table = c.plain(a[4], "page_table", at::kInt, {B, -1});
    const at::Tensor& pool = c.plain(a[5], "pool", at::kByte, {-1, static_cast<int64_t>(mla_qcache_kv4_page_bytes(cfg.p))});
    void* lens = c.ptr(a[6], "seq_lens", at::kInt, {B});
    void* err = c.ptr(a[7], "err_word", at::kInt, {1});
    return mla_qcache_kv4_keep(cfg.p, extent(B, "B"), static_cast<const int32_t*>(kept.data_ptr()), extent(kept.size(1), "kept"),
                               static_cast<const int32_t*>(count), static_cast<const int32_t*>(base),
                               static_cast<const int32_t*>(table.data_ptr()), extent(table.size(1), "page_table"),
                               static_cast<uint8_t*>(pool.data_ptr()), pool.size(0), static_cast<int32_t*>(lens),
                               static_cast<int32_t*>(err), c.stream(a[8]));
  });
}

// What both ways of verifying take beside the rows: tokens, offsets, masks, results.
struct Drafts {
  const int32_t *tokens, *cu;
  mla_qcache_tree tree{};
  int32_t B, rows, max_rows, *kept, *news, *count, *err;
  Drafts(const Call& c, int64_t n, PyObject* tokens_, PyObject* cu_, PyObject* max_rows_, PyObject* mask, PyObject* kept_,
         PyObject* new_, PyObject* count_, PyObject* err_) {
    const at::Tensor& k = c.plain(kept_, "kept", at::kInt, {-1, -1});
    B = extent(k.size(0), "B"), rows = extent(n, "rows"), max_rows = as_int(max_rows_, "max_rows");
    if (k.size(1) != max_rows) raise(PyExc_ValueError, "kept must be [B, max_rows], got " + shape_of(k));
    tokens = static_cast<const int32_t*>(c.ptr(tokens_, "tokens", at::kInt, {n}));
    cu = static_cast<const int32_t*>(c.ptr(cu_, "cu_rows", at::kInt, {B + 1ll}));
    c.tree(mask, Py_None, n, B, &tree);
    kept = static_cast<int32_t*>(k.data_ptr());
    news = static_cast<int32_t*>(c.ptr(new_, "new_tokens", at::kInt, {B, max_rows}));
    count = static_cast<int32_t*>(c.ptr(count_, "n_kept", at::kInt, {B}));
    err = static_cast<int32_t*>(c.ptr(err_, "err_word", at::kInt, {1}));
  }
};

PyObject* verify_sampled(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(args, n, 13, [](PyObject* const* a) {
    Call c;
    const at::Tensor& p = c.lead(a[0], "target_probs");
    c.strided(a[0], "target_probs", at::kFloat, -1, -1);
    const int64_t rows = p.size(0), vocab = p.size(1);
    const at::Tensor* const q = a[1] == Py_None ? nullptr : &c.strided(a[1], "draft_probs", at::kFloat, rows, vocab);
    const Drafts d(c, rows, a[2], a[3], a[4], a[5], a[8], a[9], a[10], a[11]);
    const void* ua = c.ptr(a[6], "u_accept", at::kFloat, {rows});
    const void* us = c.ptr(a[7], "u_sample", at::kFloat, {d.B});
    return mla_qcache_verify_sampled(d.B, d.rows, extent(vocab, "vocab"), static_cast<const float*>(p.data_ptr()),
                                     rows > 1 ? p.stride(0) : 0, q ? static_cast<const float*>(q->data_ptr()) : nullptr,
                                     q && rows > 1 ? q->stride(0) : 0, d.tokens, d.cu, d.max_rows, d.tree.mask, d.tree.mask_words,
                                     static_cast<const float*>(ua), static_cast<const float*>(us), d.kept, d.news, d.count, d.err,
                                     c.stream(a[12]));
  });
}

PyObject* verify_greedy(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(args, n, 10, [](PyObject* const* a) {
    Call c;
    const at::Tensor& x = c.lead(a[0], "logits");
    const int32_t dtype = x.scalar_type() == at::kFloat ? MLA_QCACHE_FP32 : row_type(x, "logits");
    c.strided(a[0], "logits", x.scalar_type(), -1, -1);
    const int64_t rows = x.size(0);
    const Drafts d(c, rows, a[1], a[2], a[3], a[4], a[5], a[6], a[7], a[8]);
    return mla_qcache_verify_greedy(d.B, d.rows, extent(x.size(1), "vocab"), dtype, x.data_ptr(), rows > 1 ? x.stride(0) : 0, d.tokens,
                                    d.cu, d.max_rows, d.tree.mask, d.tree.mask_words, d.kept, d.news, d.count, d.err, c.stream(a[9]));
  });
}

PyObject* tree_mask(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(args, n, 6, [](PyObject* const* a) {
    Call c;
    const at::Tensor& parents = c.lead(a[0], "parents");
    c.plain(a[0], "parents", at::kInt, {-1});
    const int64_t rows = parents.size(0);
    const at::Tensor& cu = c.plain(a[1], "cu_rows", at::kInt, {-1});
    if (cu.size(0) < 2) raise(PyExc_ValueError, "cu_rows must be [B + 1], got " + shape_of(cu));
    mla_qcache_tree tree{};
    if (!c.tree(a[3], Py_None, rows, 0, &tree)) raise(error_type(), "mask is required");
    void* err = c.ptr(a[4], "err_word", at::kInt, {1});
    return mla_qcache_tree_mask(extent(cu.size(0) - 1, "B"), extent(rows, "rows"), static_cast<const int32_t*>(parents.data_ptr()),
                                static_cast<const int32_t*>(cu.data_ptr()), as_int(a[2], "max_rows"), tree.mask_words,
                                const_cast<uint64_t*>(tree.mask), static_cast<int32_t*>(err), c.stream(a[5]));
  });
}

PyObject* append_bf16(PyObject*, PyObject* const* args, Py_ssize_t n) {
  return guarded(args, n, 18, [](PyObject* const* a) {
    const at::ScalarType bf = at::kBFloat16;
    Call c;
    const at::Tensor& kv = c.lead(a[0], "kv_new");
    if (kv.scalar_type() != bf || kv.dim() != 2 || kv.size(1) != 576 || kv.stride(1) != 1)
      raise(PyExc_ValueError, std::string("kv_new must be BFloat16 [rows, 576] with contiguous rows, got ") +
                                  c10::toString(kv.scalar_type()) + " " + shape_of(kv));
    const int64_t rows = kv.size(0);
    const at::Tensor& lens = c.plain(a[2], "seq_lens", at::kInt, {-1});
    const int64_t B = lens.size(0);
    const void* cu = c.ptr(a[1], "cu_new", at::kInt, {B + 1});
    const int32_t max_new = as_int(a[3], "max_new");
    const void* table = nullptr;
    void* pool = nullptr;
    int64_t pages = 1, n_pages = 0, P = 64;
    if (a[5] != Py_None) {
      const at::Tensor& t = c.plain(a[4], "page_table", at::kInt, {B, -1});
      const at::Tensor& q = c.plain(a[5], "kv_pool", bf, {-1, -1, 576});
      table = t.data_ptr(), pages = t.size(1);
      pool = q.data_ptr(), n_pages = q.size(0), P = q.size(1);
    }
    void* err = c.ptr(a[6], "err_word", at::kInt, {1});
    const void* weight = c.optional(a[7], "norm_weight", bf, {512});
    const float eps = as_float(a[8]);
    mla_qcache_rotation rot;
    const bool rotated = c.rotation(a[9], a[10], a[11], &rot);
    if ((a[12] == Py_None) != (a[13] == Py_None)) raise(error_type(), "q_rope and q_out go together");
    mla_qcache_view qv{};
    int64_t heads = 0;
    void* q_out = nullptr;
    if (a[12] != Py_None) {
      qv = c.view(a[12], "q_rope", bf, rows, -1, 64);
      heads = THPVariable_Unpack(a[12]).size(1);
      q_out = c.ptr(a[13], "q_out", bf, {rows, heads, 64});
    }
    void* c_out = c.optional(a[14], "c_out", bf, {rows, 512});
    void* kr_out = c.optional(a[15], "kr_out", bf, {rows, 64});
    void* next = c.optional(a[16], "seq_lens_next", at::kInt, {B});
    return mla_qcache_append_bf16(extent(B, "B"), extent(rows, "rows"), static_cast<const uint16_t*>(kv.data_ptr()),
                                  rows > 1 ? kv.stride(0) : 0, static_cast<const int32_t*>(cu),
                                  static_cast<const int32_t*>(lens.data_ptr()), static_cast<int32_t*>(next), max_new,
                                  static_cast<const uint16_t*>(weight), eps, rotated ? &rot : nullptr, q_out ? &qv : nullptr,
                                  extent(heads, "heads"), static_cast<uint16_t*>(q_out), static_cast<uint16_t*>(c_out),
                                  static_cast<uint16_t*>(kr_out), static_cast<const int32_t*>(table), extent(pages, "page_table"),
                                  extent(P, "page size"), static_cast<uint16_t*>(pool), n_pages, static_cast<int32_t*>(err),
                                  c.stream(a[17]));
  });
}

PyObject* set_error(PyObject*, PyObject* type) {
  Py_XINCREF(type);
  Py_XDECREF(g_error);
  g_error = type;
  Py_RETURN_NONE;
}

#define FASTCALL(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f)), METH_FASTCALL, nullptr
PyMethodDef kMethods[] = {{"kv4_append", FASTCALL(kv4_append)},
                          {"kv4_attn", FASTCALL(kv4_attn)},
                          {"kv4_attn_tree", FASTCALL(kv4_attn_tree)},
                          {"kv4_keep", FASTCALL(kv4_keep)},
                          {"verify_sampled", FASTCALL(verify_sampled)},
                          {"verify_greedy", FASTCALL(verify_greedy)},
                          {"tree_mask", FASTCALL(tree_mask)},
                          {"append_bf16", FASTCALL(append_bf16)},
                          {"set_error", set_error, METH_O, nullptr},
                          {nullptr, nullptr, 0, nullptr}};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_fastcall", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fastcall() { return PyModule_Create(&kModule); }
