// binding.cpp -- tensors into the argument blocks of the language-model
// operators (include/dc.h).
//
// A small call's time is mostly its checks: read from Python, the properties
// of seven tensors cost 5 of the 8 microseconds of a paged attention call.
// This extension module reads them in C++ and calls the library.  It holds no
// state but the library's entry points, and does no work of its own: every
// function returns the library's status.  What a call has written counts as
// changed in place (its version moves on), so that autograd notices where it
// had kept those numbers.
#include <Python.h>

#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <exception>
#include <string>

#include "dc.h"

namespace {

decltype(&dc_token_logprobs) g_score = nullptr;
decltype(&dc_token_logprobs_backward) g_grad = nullptr;
decltype(&dc_kv_append) g_append = nullptr;
decltype(&dc_paged_attention) g_attend = nullptr;

// A refusal: the Python exception is set.
struct Refused {};

[[noreturn]] void refuse(PyObject* kind, const std::string& text) {
  PyErr_SetString(kind, text.c_str());
  throw Refused{};
}
[[noreturn]] void wrong(const std::string& text) { refuse(PyExc_ValueError, text); }

std::string text(const at::Tensor& t) {
  std::string s = "(";
  for (int64_t i = 0; i < t.dim(); ++i) s += (i ? ", " : "") + std::to_string(t.size(i));
  return s + (t.dim() == 1 ? ",)" : ")");
}
std::string indexed(const char* what, int64_t i) {
  return i < 0 ? std::string(what) : std::string(what) + "[" + std::to_string(i) + "]";
}
const char* dtype_name(at::ScalarType t) {
  switch (t) {
    case at::kBFloat16: return "torch.bfloat16";
    case at::kHalf: return "torch.float16";
    case at::kFloat: return "torch.float32";
    case at::kInt: return "torch.int32";
    case at::kLong: return "torch.int64";
    default: return c10::toString(t);
  }
}

// The dc_dtype_t of a floating type, -1 if it has none.
int code_of(at::ScalarType t) {
  return t == at::kBFloat16 ? DC_BF16 : t == at::kHalf ? DC_F16 : t == at::kFloat ? DC_F32 : -1;
}

struct Call {
  int device;    // the current device, where the library launches
  dc_stream_t stream;
};

const at::Tensor& tensor(PyObject* o, const char* what, int64_t i = -1) {
  if (!THPVariable_Check(o)) refuse(PyExc_TypeError, indexed(what, i) + " must be a tensor");
  return THPVariable_Unpack(o);
}

// The tensor, on the current device and of the given type.
const at::Tensor& on(const Call& c, PyObject* o, const char* what, at::ScalarType type, int64_t i = -1) {
  const at::Tensor& t = tensor(o, what, i);
  if (!t.is_cuda())
    wrong(indexed(what, i) + " must be a CUDA tensor (got device " + t.device().str() + ")");
  if (t.get_device() != c.device)
    wrong(indexed(what, i) + " is on " + t.device().str() + ", but the current device is cuda:" + std::to_string(c.device) +
          "; make it current (torch.cuda.set_device) or move the tensor");
  if (t.scalar_type() != type)
    wrong(indexed(what, i) + " has dtype " + dtype_name(t.scalar_type()) + ", expected " + dtype_name(type));
  return t;
}

// A tensor of int32 or int64 indexes.
const at::Tensor& indexes(const Call& c, PyObject* o, const char* what) {
  const at::Tensor& t = tensor(o, what);
  const at::ScalarType s = t.scalar_type();
  if (s != at::kInt && s != at::kLong)
    wrong(std::string(what) + " has dtype " + dtype_name(s) + ", expected torch.int64 or torch.int32");
  return on(c, o, what, s);
}

void shaped(const at::Tensor& t, const char* what, int64_t n) {
  if (t.dim() != 1 || t.size(0) != n)
    wrong(std::string(what) + " has shape " + text(t) + ", expected (" + std::to_string(n) + ",)");
  if (!t.is_contiguous()) wrong(std::string(what) + " must be contiguous");
}

// Contiguous [n] vectors; NULL for None where that is allowed.
const void* vector(const Call& c, PyObject* o, const char* what, int64_t n, at::ScalarType type, bool optional = false) {
  if (optional && o == Py_None) return nullptr;
  const at::Tensor& t = on(c, o, what, type);
  shaped(t, what, n);
  return t.const_data_ptr();
}

// The call's device and stream; `first` is its first tensor: if that is on no
// GPU the checks refuse it without touching CUDA.
Call call_of(const at::Tensor& first, PyObject* stream) {
  Call c{-2, nullptr};
  if (!first.is_cuda()) return c;
  c.device = static_cast<int>(c10::cuda::current_device());
  if (stream == Py_None) {
    c.stream = reinterpret_cast<dc_stream_t>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(c.device)).stream());
    return c;
  }
  PyObject* handle = PyLong_Check(stream) ? Py_NewRef(stream) : PyObject_GetAttrString(stream, "cuda_stream");
  if (!handle) throw Refused{};
  c.stream = reinterpret_cast<dc_stream_t>(PyLong_AsVoidPtr(handle));
  Py_DECREF(handle);
  if (PyErr_Occurred()) throw Refused{};
  return c;
}

int64_t integer(PyObject* o) {
  const long long v = PyLong_AsLongLong(o);
  if (v == -1 && PyErr_Occurred()) throw Refused{};
  return v;
}
int32_t small(PyObject* o, const char* what) {
  const int64_t v = integer(o);
  if (v < INT32_MIN || v > INT32_MAX) refuse(PyExc_OverflowError, std::string(what) + " is out of range");
  return static_cast<int32_t>(v);
}
double number(PyObject* o) {
  const double v = PyFloat_AsDouble(o);
  if (v == -1.0 && PyErr_Occurred()) throw Refused{};
  return v;
}

// A sequence's items while in scope.
struct Items {
  PyObject* fast;
  explicit Items(PyObject* o, const char* what) : fast(PySequence_Fast(o, what)) {
    if (!fast) throw Refused{};
  }
  ~Items() { Py_DECREF(fast); }
  Items(const Items&) = delete;
  Py_ssize_t size() const { return PySequence_Fast_GET_SIZE(fast); }
  PyObject* operator[](Py_ssize_t i) const { return PySequence_Fast_GET_ITEM(fast, i); }
};

// The tensors that a call writes.
struct Written {
  const at::Tensor* t[DC_MAX_RANKS];
  int n = 0;
  const at::Tensor& operator()(const at::Tensor& x) {
    if (n < DC_MAX_RANKS) t[n++] = &x;
    return x;
  }
  PyObject* after(dc_status_t status) const {
    for (int i = 0; i < n && status == DC_OK; ++i)
      if (!t[i]->is_inference()) t[i]->unsafeGetTensorImpl()->bump_version();
    return PyLong_FromLong(status);
  }
};

// Ranks' [rows, width] matrices.
struct Matrices {
  const void* data[DC_MAX_RANKS];
  uint64_t width[DC_MAX_RANKS], stride[DC_MAX_RANKS];
  int64_t total = 0;
};
void matrices(const Call& c, const Items& items, const char* what, int64_t rows, at::ScalarType type, Written* w,
              Matrices& m) {
  for (Py_ssize_t r = 0; r < items.size(); ++r) {
    const at::Tensor& t = on(c, items[r], what, type, r);
    if (t.dim() != 2 || t.size(0) != rows)
      wrong(indexed(what, r) + " has shape " + text(t) + ", expected (" + std::to_string(rows) + ", columns)");
    if (t.stride(1) != 1 && t.size(1) > 1) wrong(indexed(what, r) + ": the vocabulary dimension must be contiguous");
    m.total += t.size(1);
    if (r >= DC_MAX_RANKS) continue;  // (the library refuses the count)
    m.data[r] = w ? (*w)(t).mutable_data_ptr() : t.const_data_ptr();
    m.width[r] = static_cast<uint64_t>(t.size(1));
    m.stride[r] = static_cast<uint64_t>(t.stride(0));
  }
}

// The rows and the type of the first shard.
struct Logits {
  int64_t rows;
  at::ScalarType type;
  int code;
};
Logits logits(const Items& shards) {
  if (shards.size() == 0) wrong("need at least one shard");
  const at::Tensor& first = tensor(shards[0], "shards", 0);
  if (first.dim() != 2) wrong("shards[0] has shape " + text(first) + ", expected (rows, columns)");
  const int code = code_of(first.scalar_type());
  if (code < 0) wrong(std::string("logits are bfloat16, float16 or float32 (got ") + dtype_name(first.scalar_type()) + ")");
  return Logits{first.size(0), first.scalar_type(), code};
}

// A contiguous [n] output; NULL for None where that is allowed.
void* out_vector(const Call& c, PyObject* o, const char* what, int64_t n, at::ScalarType type, Written& w,
                 bool optional = false) {
  if (optional && o == Py_None) return nullptr;
  const at::Tensor& t = on(c, o, what, type);
  shaped(t, what, n);
  return w(t).mutable_data_ptr();
}

// A contiguous [rows, k] output; k < 0: any, and it is set.
void* alternatives(const Call& c, PyObject* o, const char* what, int64_t rows, at::ScalarType type, Written& w, int64_t& k) {
  const at::Tensor& t = on(c, o, what, type);
  if (t.dim() != 2 || t.size(0) != rows || (k >= 0 && t.size(1) != k) || !t.is_contiguous())
    wrong(std::string(what) + " must be a contiguous (" + std::to_string(rows) + ", " + (k < 0 ? "k" : std::to_string(k)) +
          ") tensor (got " + text(t) + ")");
  k = t.size(1);
  return w(t).mutable_data_ptr();
}

// token_logprobs(shards, tokens, logprobs, entropy, lse, top_logprobs,
//                top_tokens, vocab, temperature, stream) -> status
PyObject* score(PyObject* const* a) {
  const Items shards(a[0], "shards must be a sequence of tensors");
  const Logits l = logits(shards);
  const Call c = call_of(THPVariable_Unpack(shards[0]), a[9]);
  Written w;
  Matrices m;
  matrices(c, shards, "shards", l.rows, l.type, nullptr, m);
  dc_token_logprobs_t b{};
  b.shards = m.data;
  b.widths = m.width;
  b.row_strides = m.stride;
  const at::Tensor& tokens = indexes(c, a[1], "tokens");
  shaped(tokens, "tokens", l.rows);
  b.tokens = tokens.const_data_ptr();
  b.tokens_64 = tokens.scalar_type() == at::kLong;
  b.logprobs = static_cast<float*>(out_vector(c, a[2], "logprobs", l.rows, at::kFloat, w));
  b.entropy = static_cast<float*>(out_vector(c, a[3], "entropy", l.rows, at::kFloat, w, true));
  b.lse = static_cast<float*>(out_vector(c, a[4], "lse", l.rows, at::kFloat, w, true));
  int64_t top = -1;
  if (a[5] != Py_None)
    b.top_logprobs = static_cast<float*>(alternatives(c, a[5], "top_logprobs", l.rows, at::kFloat, w, top));
  if (a[6] != Py_None) {
    const at::Tensor& t = indexes(c, a[6], "top_tokens");
    b.top_tokens = alternatives(c, a[6], "top_tokens", l.rows, t.scalar_type(), w, top);
    b.top_tokens_64 = t.scalar_type() == at::kLong;
  }
  b.top = top < 0 ? 0 : static_cast<int32_t>(top > 1 << 20 ? 1 << 20 : top);
  b.rows = l.rows;
  b.vocab = a[7] == Py_None ? m.total : integer(a[7]);
  b.temperature = number(a[8]);
  b.ranks = static_cast<int32_t>(shards.size());
  b.dtype = l.code;
  return w.after(g_score(&b, c.stream));
}

// token_logprobs_backward(shards, tokens, lse, grad_logprobs, grads, entropy,
//                         grad_entropy, vocab, temperature, stream) -> status
PyObject* grad(PyObject* const* a) {
  const Items shards(a[0], "shards must be a sequence of tensors"), grads(a[4], "grads must be a sequence of tensors");
  const Logits l = logits(shards);
  const Call c = call_of(THPVariable_Unpack(shards[0]), a[9]);
  if (grads.size() != shards.size())
    wrong("need one gradient per shard (got " + std::to_string(grads.size()) + " for " + std::to_string(shards.size()) + ")");
  Written w;
  Matrices m, g;
  matrices(c, shards, "shards", l.rows, l.type, nullptr, m);
  matrices(c, grads, "grads", l.rows, l.type, &w, g);
  for (Py_ssize_t r = 0; r < shards.size() && r < DC_MAX_RANKS; ++r)
    if (m.width[r] != g.width[r]) wrong("grads must have the shards' shapes");
  if (a[6] != Py_None && a[5] == Py_None) wrong("grad_entropy needs the forward call's entropy");
  dc_token_logprobs_backward_t b{};
  b.shards = m.data;
  b.widths = m.width;
  b.row_strides = m.stride;
  void* out[DC_MAX_RANKS];
  for (Py_ssize_t r = 0; r < grads.size() && r < DC_MAX_RANKS; ++r) out[r] = const_cast<void*>(g.data[r]);
  b.grads = out;
  b.grad_row_strides = g.stride;
  const at::Tensor& tokens = indexes(c, a[1], "tokens");
  shaped(tokens, "tokens", l.rows);
  b.tokens = tokens.const_data_ptr();
  b.tokens_64 = tokens.scalar_type() == at::kLong;
  b.lse = static_cast<const float*>(vector(c, a[2], "lse", l.rows, at::kFloat));
  b.grad_logprobs = static_cast<const float*>(vector(c, a[3], "grad_logprobs", l.rows, at::kFloat, true));
  b.entropy = static_cast<const float*>(vector(c, a[5], "entropy", l.rows, at::kFloat, true));
  b.grad_entropy = static_cast<const float*>(vector(c, a[6], "grad_entropy", l.rows, at::kFloat, true));
  b.rows = l.rows;
  b.vocab = a[7] == Py_None ? m.total : integer(a[7]);
  b.temperature = number(a[8]);
  b.ranks = static_cast<int32_t>(shards.size());
  b.dtype = l.code;
  return w.after(g_grad(&b, c.stream));
}

// A [n, heads, dim] tensor's strides; heads or dim < 0: any.
const at::Tensor& heads_of(const Call& c, PyObject* o, const char* what, int64_t n, int64_t heads, int64_t dim,
                           at::ScalarType type, uint64_t& s0, uint64_t& s1) {
  const at::Tensor& t = on(c, o, what, type);
  if (t.dim() != 3 || t.size(0) != n || (heads >= 0 && t.size(1) != heads) || (dim >= 0 && t.size(2) != dim))
    wrong(std::string(what) + " has shape " + text(t) + ", expected (" + std::to_string(n) + ", " +
          (heads < 0 ? "heads" : std::to_string(heads)) + ", " + (dim < 0 ? "dim" : std::to_string(dim)) + ")");
  if (t.stride(2) != 1 && t.size(2) > 1) wrong(std::string(what) + ": the last dimension must be contiguous");
  s0 = static_cast<uint64_t>(t.stride(0));
  s1 = static_cast<uint64_t>(t.stride(1));
  return t;
}

// The two caches of a call: same shape, any strides.
struct Caches {
  int64_t pages, page_size, heads;
};
Caches caches(const Call& c, PyObject* ko, PyObject* vo, int64_t heads, int64_t dim, at::ScalarType type, Written* w,
              dc_paged_cache_t& k, dc_paged_cache_t& v) {
  Caches r{0, 0, heads};
  for (int i = 0; i < 2; ++i) {
    const char* what = i ? "v_cache" : "k_cache";
    const at::Tensor& t = on(c, i ? vo : ko, what, type);
    if (t.dim() != 4 || (r.heads >= 0 && t.size(2) != r.heads) || t.size(3) != dim ||
        (i && (t.size(0) != r.pages || t.size(1) != r.page_size)))
      wrong(std::string(what) + " has shape " + text(t) + ", expected (" + (i ? std::to_string(r.pages) : "pages") + ", " +
            (i ? std::to_string(r.page_size) : "page size") + ", " + (r.heads < 0 ? "heads" : std::to_string(r.heads)) + ", " +
            std::to_string(dim) + ")");
    if (t.stride(3) != 1 && t.size(3) > 1) wrong(std::string(what) + ": the last dimension must be contiguous");
    r = Caches{t.size(0), t.size(1), t.size(2)};
    dc_paged_cache_t& x = i ? v : k;
    x.data = w ? (*w)(t).mutable_data_ptr() : const_cast<void*>(t.const_data_ptr());
    x.page_stride = static_cast<uint64_t>(t.stride(0));
    x.token_stride = static_cast<uint64_t>(t.stride(1));
    x.head_stride = static_cast<uint64_t>(t.stride(2));
  }
  return r;
}

const at::Tensor& page_table(const Call& c, PyObject* o, int64_t rows) {
  const at::Tensor& t = on(c, o, "page_table", at::kInt);
  if (t.dim() != 2 || (rows >= 0 && t.size(0) != rows))
    wrong("page_table has shape " + text(t) + ", expected (" + (rows < 0 ? "sequences" : std::to_string(rows)) + ", pages)");
  if (t.stride(1) != 1 && t.size(1) > 1) wrong("page_table: rows must be contiguous");
  return t;
}

// kv_append(k, v, positions, seqs, page_table, k_cache, v_cache, q, q_out,
//           cos_sin, interleaved, stream) -> status
PyObject* append(PyObject* const* a) {
  const at::Tensor& first = tensor(a[0], "k");
  const at::ScalarType type = first.scalar_type();
  const int code = code_of(type);
  if (code < 0) wrong(std::string("keys are bfloat16, float16 or float32 (got ") + dtype_name(type) + ")");
  const Call c = call_of(first, a[11]);
  if (first.dim() != 3) wrong("k has shape " + text(first) + ", expected (tokens, heads, dim)");
  const int64_t n = first.size(0), hk = first.size(1), d = first.size(2);
  Written w;
  dc_kv_append_t b{};
  b.k = heads_of(c, a[0], "k", n, hk, d, type, b.k_token_stride, b.k_head_stride).const_data_ptr();
  b.v = heads_of(c, a[1], "v", n, hk, d, type, b.v_token_stride, b.v_head_stride).const_data_ptr();
  int64_t hq = 0;
  if (a[7] != Py_None) {
    if (a[8] == Py_None) wrong("q needs q_out");
    const at::Tensor& q = heads_of(c, a[7], "q", n, -1, d, type, b.q_token_stride, b.q_head_stride);
    hq = q.size(1);
    b.q = q.const_data_ptr();
    b.q_out = w(heads_of(c, a[8], "q_out", n, hq, d, type, b.q_out_token_stride, b.q_out_head_stride)).mutable_data_ptr();
  } else if (a[8] != Py_None) {
    wrong("q_out needs q");
  }
  if (a[9] != Py_None) {
    const at::Tensor& t = tensor(a[9], "cos_sin");
    if (t.scalar_type() != at::kFloat || t.dim() != 2 || !t.is_contiguous())
      wrong(std::string("cos_sin must be a contiguous float32 (positions, rotary_dim) tensor (got ") +
            dtype_name(t.scalar_type()) + " " + text(t) + ")");
    on(c, a[9], "cos_sin", at::kFloat);
    b.cos_sin = static_cast<const float*>(t.const_data_ptr());
    b.cos_sin_rows = t.size(0);
    b.rotary_dim = static_cast<int32_t>(t.size(1) > 1 << 20 ? 1 << 20 : t.size(1));
  }
  const Caches x = caches(c, a[5], a[6], hk, d, type, &w, b.k_cache, b.v_cache);
  const at::Tensor& table = page_table(c, a[4], -1);
  b.positions = static_cast<const int32_t*>(vector(c, a[2], "positions", n, at::kInt));
  b.seqs = static_cast<const int32_t*>(vector(c, a[3], "seqs", n, at::kInt));
  b.page_table = static_cast<const int32_t*>(table.const_data_ptr());
  b.table_rows = table.size(0);
  b.table_width = table.size(1);
  b.table_stride = table.stride(0);
  b.tokens = n;
  b.num_pages = x.pages;
  if (x.page_size > INT32_MAX || hq > INT32_MAX || hk > INT32_MAX || d > INT32_MAX) wrong("a dimension is too large");
  b.page_size = static_cast<int32_t>(x.page_size);
  b.q_heads = static_cast<int32_t>(hq);
  b.kv_heads = static_cast<int32_t>(hk);
  b.dim = static_cast<int32_t>(d);
  const int truth = PyObject_IsTrue(a[10]);
  if (truth < 0) throw Refused{};
  b.interleaved = truth;
  b.dtype = code;
  return w.after(g_append(&b, c.stream));
}

// paged_attention(q, k_cache, v_cache, page_table, lengths, out, workspace,
//                 scale, window, lse, stream) -> status
PyObject* attend(PyObject* const* a) {
  const at::Tensor& first = tensor(a[0], "q");
  const at::ScalarType type = first.scalar_type();
  const int code = code_of(type);
  if (code != DC_BF16 && code != DC_F16) wrong(std::string("queries are bfloat16 or float16 (got ") + dtype_name(type) + ")");
  const Call c = call_of(first, a[10]);
  if (first.dim() != 3) wrong("q has shape " + text(first) + ", expected (sequences, heads, dim)");
  const int64_t n = first.size(0), hq = first.size(1), d = first.size(2);
  Written w;
  dc_paged_attention_t b{};
  b.q = heads_of(c, a[0], "q", n, hq, d, type, b.q_seq_stride, b.q_head_stride).const_data_ptr();
  b.out = w(heads_of(c, a[5], "out", n, hq, d, type, b.out_seq_stride, b.out_head_stride)).mutable_data_ptr();
  const Caches x = caches(c, a[1], a[2], -1, d, type, nullptr, b.k_cache, b.v_cache);
  const at::Tensor& table = page_table(c, a[3], n);
  b.page_table = static_cast<const int32_t*>(table.const_data_ptr());
  b.table_width = table.size(1);
  b.table_stride = table.stride(0);
  b.lengths = static_cast<const int32_t*>(vector(c, a[4], "lengths", n, at::kInt));
  const at::Tensor& ws = tensor(a[6], "workspace");
  on(c, a[6], "workspace", ws.scalar_type());
  if (!ws.is_contiguous()) wrong("workspace must be contiguous");
  b.workspace = ws.mutable_data_ptr();
  b.workspace_bytes = static_cast<uint64_t>(ws.nbytes());
  if (a[9] != Py_None) {
    const at::Tensor& t = tensor(a[9], "lse");
    if (t.scalar_type() != at::kFloat || t.dim() != 2 || t.size(0) != n || t.size(1) != hq || !t.is_contiguous())
      wrong("lse must be a contiguous float32 (" + std::to_string(n) + ", " + std::to_string(hq) + ") tensor (got " +
            dtype_name(t.scalar_type()) + " " + text(t) + ")");
    on(c, a[9], "lse", at::kFloat);
    b.lse = static_cast<float*>(w(t).mutable_data_ptr());
  }
  if (x.page_size > INT32_MAX || hq > INT32_MAX || x.heads > INT32_MAX || d > INT32_MAX) wrong("a dimension is too large");
  b.seqs = n;
  b.num_pages = x.pages;
  b.page_size = static_cast<int32_t>(x.page_size);
  b.q_heads = static_cast<int32_t>(hq);
  b.kv_heads = static_cast<int32_t>(x.heads);
  b.dim = static_cast<int32_t>(d);
  b.window = small(a[8], "window");
  b.dtype = code;
  b.scale = a[7] == Py_None ? static_cast<float>(1.0 / std::sqrt(static_cast<double>(d))) : static_cast<float>(number(a[7]));
  return w.after(g_attend(&b, c.stream));
}

// Counts the arguments and turns C++ exceptions into Python's.
template <PyObject* (*F)(PyObject* const*), int N>
PyObject* entry(PyObject*, PyObject* const* args, Py_ssize_t n) {
  if (n != N) {
    PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", N, n);
    return nullptr;
  }
  if (!g_score) {
    PyErr_SetString(PyExc_RuntimeError, "bind() has not been called");
    return nullptr;
  }
  try {
    return F(args);
  } catch (const Refused&) {
    return nullptr;
  } catch (const std::exception& e) {
    PyErr_SetString(PyExc_RuntimeError, e.what());
    return nullptr;
  }
}

// bind(dc_token_logprobs, dc_token_logprobs_backward, dc_kv_append,
//      dc_paged_attention): the loaded library's entry points, as addresses.
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  void* at[4];
  if (n != 4) {
    PyErr_SetString(PyExc_TypeError, "expected 4 addresses");
    return nullptr;
  }
  for (int i = 0; i < 4; ++i) {
    at[i] = PyLong_AsVoidPtr(args[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  g_score = reinterpret_cast<decltype(g_score)>(at[0]);
  g_grad = reinterpret_cast<decltype(g_grad)>(at[1]);
  g_append = reinterpret_cast<decltype(g_append)>(at[2]);
  g_attend = reinterpret_cast<decltype(g_attend)>(at[3]);
  Py_RETURN_NONE;
}

template <class F>
PyCFunction as_function(F f) {
  return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f));
}

PyMethodDef kMethods[] = {
    {"bind", as_function(&bind), METH_FASTCALL, nullptr},
    {"token_logprobs", as_function(&entry<score, 10>), METH_FASTCALL, nullptr},
    {"token_logprobs_backward", as_function(&entry<grad, 10>), METH_FASTCALL, nullptr},
    {"kv_append", as_function(&entry<append, 12>), METH_FASTCALL, nullptr},
    {"paged_attention", as_function(&entry<attend, 11>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&kModule); }
