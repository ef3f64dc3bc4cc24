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
decltype(&dc_linear_logprobs) g_linear = nullptr;
decltype(&dc_linear_logprobs_backward) g_linear_grad = nullptr;
decltype(&dc_kv_append_norm) g_append_norm = nullptr;
decltype(&dc_qk_norm_rotate) g_norm = nullptr;
decltype(&dc_qk_norm_rotate_backward) g_norm_grad = nullptr;
decltype(&dc_prefix_attention) g_prefix = nullptr;

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

// A call's workspace, whatever its type.
const at::Tensor& workspace_of(const Call& c, PyObject* o) {
  const at::Tensor& t = tensor(o, "workspace");
  on(c, o, "workspace", t.scalar_type());
  if (!t.is_contiguous()) wrong("workspace must be contiguous");
  return t;
}

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

const at::Tensor& page_table(const Call& c, PyObject* o, int64_t rows, const char* what = "page_table") {
  const at::Tensor& t = on(c, o, what, at::kInt);
  if (t.dim() != 2 || (rows >= 0 && t.size(0) != rows))
    wrong(std::string(what) + " has shape " + text(t) + ", expected (" + (rows < 0 ? "sequences" : std::to_string(rows)) + ", pages)");
  if (t.stride(1) != 1 && t.size(1) > 1) wrong(std::string(what) + ": rows must be contiguous");
  return t;
}

const float* angles(const Call& c, PyObject* o, int64_t& rows, int32_t& rotary) {
  if (o == Py_None) return nullptr;
  const at::Tensor& t = tensor(o, "cos_sin");
  if (t.scalar_type() != at::kFloat || t.dim() != 2 || !t.is_contiguous())
    wrong(std::string("cos_sin must be a contiguous float32 (positions, rotary_dim) tensor (got ") +
          dtype_name(t.scalar_type()) + " " + text(t) + ")");
  on(c, o, "cos_sin", at::kFloat);
  rows = t.size(0);
  rotary = static_cast<int32_t>(t.size(1) > 1 << 20 ? 1 << 20 : t.size(1));
  return static_cast<const float*>(t.const_data_ptr());
}

int truth(PyObject* o) {
  const int t = PyObject_IsTrue(o);
  if (t < 0) throw Refused{};
  return t;
}

// The arguments of kv_append, in their order.
Call fill_append(PyObject* const* a, dc_kv_append_t& b, Written& w) {
  const at::Tensor& first = tensor(a[0], "k");
  const at::ScalarType type = first.scalar_type();
  const int code = code_of(type);
  if (code < 0) wrong(std::string("keys are bfloat16, float16 or float32 (got ") + dtype_name(type) + ")");
  const Call c = call_of(first, a[11]);
  if (first.dim() != 3) wrong("k has shape " + text(first) + ", expected (tokens, heads, dim)");
  const int64_t n = first.size(0), hk = first.size(1), d = first.size(2);
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
  b.cos_sin = angles(c, a[9], b.cos_sin_rows, b.rotary_dim);
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
  b.interleaved = truth(a[10]);
  b.dtype = code;
  return c;
}

// kv_append(k, v, positions, seqs, page_table, k_cache, v_cache, q, q_out,
//           cos_sin, interleaved, stream) -> status
PyObject* append(PyObject* const* a) {
  Written w;
  dc_kv_append_t b{};
  const Call c = fill_append(a, b, w);
  return w.after(g_append(&b, c.stream));
}

// The weights of a norm: [dim] in binary32 or the heads' type; `f32` < 0: either.
const void* norm_weight(const Call& c, PyObject* o, const char* what, int64_t dim, at::ScalarType type, int& f32) {
  const at::Tensor& t = tensor(o, what);
  const at::ScalarType s = t.scalar_type();
  if (s != at::kFloat && s != type)
    wrong(std::string(what) + " has dtype " + dtype_name(s) + ", expected torch.float32 or " + dtype_name(type));
  if (f32 >= 0 && f32 != (s == at::kFloat)) wrong("q_norm and k_norm must have one dtype");
  on(c, o, what, s);
  shaped(t, what, dim);
  f32 = s == at::kFloat;
  return t.const_data_ptr();
}

// kv_append_norm(the arguments of kv_append, then q_norm, k_norm, eps) -> status
PyObject* append_norm(PyObject* const* a) {
  Written w;
  dc_kv_append_norm_t b{};
  const Call c = fill_append(a, b.append, w);
  const at::ScalarType type = THPVariable_Unpack(a[0]).scalar_type();
  int f32 = -1;
  if (a[13] == Py_None) wrong("q_norm needs k_norm");
  b.k_norm = norm_weight(c, a[13], "k_norm", b.append.dim, type, f32);
  if (b.append.q_heads || a[12] != Py_None) {
    if (a[12] == Py_None) wrong("k_norm needs q_norm where there are queries");
    b.q_norm = norm_weight(c, a[12], "q_norm", b.append.dim, type, f32);
  }
  b.norm_32 = f32;
  b.eps = static_cast<float>(number(a[14]));
  return w.after(g_append_norm(&b, c.stream));
}

// The tokens, heads and angles of a norm of queries and keys.
struct NormArgs {
  int64_t n, hq, hk, d;
  at::ScalarType type;
  Call call;
};
void heads_in(const NormArgs& s, PyObject* o, const char* what, bool keys, dc_heads_t& h, Written* w) {
  const at::Tensor& t = heads_of(s.call, o, what, s.n, keys ? s.hk : s.hq, s.d, s.type, h.token_stride, h.head_stride);
  h.data = w ? (*w)(t).mutable_data_ptr() : const_cast<void*>(t.const_data_ptr());
}
template <class Block>
NormArgs fill_norm(Block& b, PyObject* const* a, PyObject* eps, PyObject* interleaved, PyObject* stream) {
  const at::Tensor &q = tensor(a[0], "q"), &k = tensor(a[1], "k");
  NormArgs s{};
  s.type = q.scalar_type();
  const int code = code_of(s.type);
  if (code < 0) wrong(std::string("queries are bfloat16, float16 or float32 (got ") + dtype_name(s.type) + ")");
  s.call = call_of(q, stream);
  if (q.dim() != 3) wrong("q has shape " + text(q) + ", expected (tokens, heads, dim)");
  if (k.dim() != 3) wrong("k has shape " + text(k) + ", expected (tokens, heads, dim)");
  s.n = q.size(0);
  s.hq = q.size(1);
  s.hk = k.size(1);
  s.d = q.size(2);
  if (s.hq > INT32_MAX || s.hk > INT32_MAX || s.d > INT32_MAX) wrong("a dimension is too large");
  heads_in(s, a[0], "q", false, b.q, nullptr);
  heads_in(s, a[1], "k", true, b.k, nullptr);
  b.positions = static_cast<const int32_t*>(vector(s.call, a[2], "positions", s.n, at::kInt));
  b.cos_sin = angles(s.call, a[3], b.cos_sin_rows, b.rotary_dim);
  int f32 = -1;
  b.q_norm = norm_weight(s.call, a[4], "q_norm", s.d, s.type, f32);
  b.k_norm = norm_weight(s.call, a[5], "k_norm", s.d, s.type, f32);
  b.norm_32 = f32;
  b.tokens = s.n;
  b.q_heads = static_cast<int32_t>(s.hq);
  b.kv_heads = static_cast<int32_t>(s.hk);
  b.dim = static_cast<int32_t>(s.d);
  b.dtype = code;
  b.eps = static_cast<float>(number(eps));
  b.interleaved = truth(interleaved);
  return s;
}

// qk_norm_rotate(q, k, positions, cos_sin, q_norm, k_norm, q_out, k_out, eps,
//                interleaved, stream) -> status
PyObject* norm(PyObject* const* a) {
  Written w;
  dc_qk_norm_rotate_t b{};
  const NormArgs s = fill_norm(b, a, a[8], a[9], a[10]);
  heads_in(s, a[6], "q_out", false, b.q_out, &w);
  heads_in(s, a[7], "k_out", true, b.k_out, &w);
  return w.after(g_norm(&b, s.call.stream));
}

// qk_norm_rotate_backward(q, k, positions, cos_sin, q_norm, k_norm,
//   grad_q_out, grad_k_out, grad_q, grad_k, grad_q_norm, grad_k_norm,
//   workspace, eps, interleaved, stream) -> status
PyObject* norm_grad(PyObject* const* a) {
  Written w;
  dc_qk_norm_rotate_backward_t b{};
  const NormArgs s = fill_norm(b, a, a[13], a[14], a[15]);
  heads_in(s, a[6], "grad_q_out", false, b.grad_q_out, nullptr);
  heads_in(s, a[7], "grad_k_out", true, b.grad_k_out, nullptr);
  heads_in(s, a[8], "grad_q", false, b.grad_q, &w);
  heads_in(s, a[9], "grad_k", true, b.grad_k, &w);
  const at::ScalarType type = b.norm_32 ? at::kFloat : s.type;
  b.grad_q_norm = out_vector(s.call, a[10], "grad_q_norm", s.d, type, w, true);
  b.grad_k_norm = out_vector(s.call, a[11], "grad_k_norm", s.d, type, w, true);
  if (a[12] != Py_None) {
    const at::Tensor& ws = workspace_of(s.call, a[12]);
    b.workspace = ws.mutable_data_ptr();
    b.workspace_bytes = static_cast<uint64_t>(ws.nbytes());
  }
  return w.after(g_norm_grad(&b, s.call.stream));
}

// The arguments of paged_attention, in their order.
Call fill_attend(PyObject* const* a, dc_paged_attention_t& b, Written& w) {
  const at::Tensor& first = tensor(a[0], "q");
  const at::ScalarType type = first.scalar_type();
  const int code = code_of(type);
  if (code != DC_BF16 && code != DC_F16) wrong(std::string("queries are bfloat16 or float16 (got ") + dtype_name(type) + ")");
  const Call c = call_of(first, a[10]);
  if (first.dim() != 3) wrong("q has shape " + text(first) + ", expected (sequences, heads, dim)");
  const int64_t n = first.size(0), hq = first.size(1), d = first.size(2);
  b.q = heads_of(c, a[0], "q", n, hq, d, type, b.q_seq_stride, b.q_head_stride).const_data_ptr();
  b.out = w(heads_of(c, a[5], "out", n, hq, d, type, b.out_seq_stride, b.out_head_stride)).mutable_data_ptr();
  const Caches x = caches(c, a[1], a[2], -1, d, type, nullptr, b.k_cache, b.v_cache);
  const at::Tensor& table = page_table(c, a[3], n);
  b.page_table = static_cast<const int32_t*>(table.const_data_ptr());
  b.table_width = table.size(1);
  b.table_stride = table.stride(0);
  b.lengths = static_cast<const int32_t*>(vector(c, a[4], "lengths", n, at::kInt));
  const at::Tensor& ws = workspace_of(c, a[6]);
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
  return c;
}

// paged_attention(q, k_cache, v_cache, page_table, lengths, out, workspace,
//                 scale, window, lse, stream) -> status
PyObject* attend(PyObject* const* a) {
  Written w;
  dc_paged_attention_t b{};
  const Call c = fill_attend(a, b, w);
  return w.after(g_attend(&b, c.stream));
}

// prefix_attention(the arguments of paged_attention, then prefix_table,
//                  prefix_lengths) -> status
PyObject* prefix(PyObject* const* a) {
  Written w;
  dc_prefix_attention_t b{};
  const Call c = fill_attend(a, b.own, w);
  const at::Tensor& table = page_table(c, a[11], -1, "prefix_table");
  b.prefix_table = static_cast<const int32_t*>(table.const_data_ptr());
  b.prefixes = table.size(0);
  b.prefix_table_width = table.size(1);
  b.prefix_table_stride = table.stride(0);
  b.prefix_lengths = static_cast<const int32_t*>(vector(c, a[12], "prefix_lengths", b.prefixes, at::kInt));
  return w.after(g_prefix(&b, c.stream));
}

// A head: hidden [rows, size] and its shards [columns, size].
struct HeadArgs {
  int64_t rows, size, columns = 0;
  at::ScalarType type;
  int code;
  Call call;
  const void* weights[DC_MAX_RANKS];
  uint64_t width[DC_MAX_RANKS], stride[DC_MAX_RANKS];
};
const at::Tensor& head_matrix(const Call& c, PyObject* o, const char* what, int64_t i, int64_t rows, int64_t size,
                              at::ScalarType type) {
  const at::Tensor& t = on(c, o, what, type, i);
  if (t.dim() != 2 || (rows >= 0 && t.size(0) != rows) || t.size(1) != size)
    wrong(indexed(what, i) + " has shape " + text(t) + ", expected (" + (rows < 0 ? "columns" : std::to_string(rows)) + ", " +
          std::to_string(size) + ")");
  if (t.stride(1) != 1 && t.size(1) > 1) wrong(indexed(what, i) + ": the hidden dimension must be contiguous");
  return t;
}
void head(PyObject* hidden, const Items& weights, PyObject* stream, HeadArgs& h) {
  const at::Tensor& x = tensor(hidden, "hidden");
  if (x.dim() != 2) wrong("hidden has shape " + text(x) + ", expected (rows, hidden size)");
  h.type = x.scalar_type();
  h.code = code_of(h.type);
  if (h.code != DC_BF16 && h.code != DC_F16)
    wrong(std::string("hidden rows are bfloat16 or float16 (got ") + dtype_name(h.type) + ")");
  h.call = call_of(x, stream);
  h.rows = x.size(0);
  h.size = x.size(1);
  head_matrix(h.call, hidden, "hidden", -1, h.rows, h.size, h.type);
  if (weights.size() == 0) wrong("need at least one shard of the weights");
  for (Py_ssize_t r = 0; r < weights.size(); ++r) {
    const at::Tensor& w = head_matrix(h.call, weights[r], "weights", r, -1, h.size, h.type);
    h.columns += w.size(0);
    if (r >= DC_MAX_RANKS) continue;  // (the library refuses the count)
    h.weights[r] = w.const_data_ptr();
    h.width[r] = static_cast<uint64_t>(w.size(0));
    h.stride[r] = static_cast<uint64_t>(w.stride(0));
  }
}
template <class Block>
void fill_head(Block& b, const HeadArgs& h, PyObject* hidden, const Items& weights, PyObject* tokens_of, PyObject* workspace,
               PyObject* vocab, PyObject* temperature) {
  const at::Tensor& x = THPVariable_Unpack(hidden);
  b.hidden = x.const_data_ptr();
  b.hidden_row_stride = static_cast<uint64_t>(x.stride(0));
  b.weights = h.weights;
  b.widths = h.width;
  b.weight_row_strides = h.stride;
  const at::Tensor& tokens = indexes(h.call, tokens_of, "tokens");
  shaped(tokens, "tokens", h.rows);
  b.tokens = tokens.const_data_ptr();
  b.tokens_64 = tokens.scalar_type() == at::kLong;
  const at::Tensor& ws = workspace_of(h.call, workspace);
  b.workspace = ws.mutable_data_ptr();
  b.workspace_bytes = static_cast<uint64_t>(ws.nbytes());
  b.rows = h.rows;
  b.hidden_size = h.size;
  b.vocab = vocab == Py_None ? h.columns : integer(vocab);
  b.temperature = number(temperature);
  b.ranks = static_cast<int32_t>(weights.size());
  b.dtype = h.code;
}

// linear_logprobs(hidden, weights, tokens, logprobs, workspace, entropy, lse,
//                 vocab, temperature, stream) -> status
PyObject* linear(PyObject* const* a) {
  const Items weights(a[1], "weights must be a sequence of tensors");
  HeadArgs h;
  head(a[0], weights, a[9], h);
  Written w;
  dc_linear_logprobs_t b{};
  fill_head(b, h, a[0], weights, a[2], a[4], a[7], a[8]);
  b.logprobs = static_cast<float*>(out_vector(h.call, a[3], "logprobs", h.rows, at::kFloat, w));
  b.entropy = static_cast<float*>(out_vector(h.call, a[5], "entropy", h.rows, at::kFloat, w, true));
  b.lse = static_cast<float*>(out_vector(h.call, a[6], "lse", h.rows, at::kFloat, w, true));
  return w.after(g_linear(&b, h.call.stream));
}

// linear_logprobs_backward(hidden, weights, tokens, lse, grad_logprobs,
//   grad_hidden, grad_weights, workspace, entropy, grad_entropy, vocab,
//   temperature, stream) -> status
PyObject* linear_grad(PyObject* const* a) {
  const Items weights(a[1], "weights must be a sequence of tensors");
  HeadArgs h;
  head(a[0], weights, a[12], h);
  Written w, w_hidden;
  dc_linear_logprobs_backward_t b{};
  fill_head(b, h, a[0], weights, a[2], a[7], a[10], a[11]);
  if (a[9] != Py_None && a[8] == Py_None) wrong("grad_entropy needs the forward call's entropy");
  b.lse = static_cast<const float*>(vector(h.call, a[3], "lse", h.rows, at::kFloat));
  b.grad_logprobs = static_cast<const float*>(vector(h.call, a[4], "grad_logprobs", h.rows, at::kFloat, true));
  b.entropy = static_cast<const float*>(vector(h.call, a[8], "entropy", h.rows, at::kFloat, true));
  b.grad_entropy = static_cast<const float*>(vector(h.call, a[9], "grad_entropy", h.rows, at::kFloat, true));
  if (a[5] != Py_None) {
    const at::Tensor& g = head_matrix(h.call, a[5], "grad_hidden", -1, h.rows, h.size, h.type);
    b.grad_hidden = w_hidden(g).mutable_data_ptr();
    b.grad_hidden_row_stride = static_cast<uint64_t>(g.stride(0));
  }
  void* out[DC_MAX_RANKS];
  uint64_t stride[DC_MAX_RANKS];
  if (a[6] != Py_None) {
    const Items grads(a[6], "grad_weights must be a sequence of tensors");
    if (grads.size() != weights.size())
      wrong("need one gradient per shard (got " + std::to_string(grads.size()) + " for " + std::to_string(weights.size()) + ")");
    for (Py_ssize_t r = 0; r < grads.size() && r < DC_MAX_RANKS; ++r) {
      const at::Tensor& g = head_matrix(h.call, grads[r], "grad_weights", r, static_cast<int64_t>(h.width[r]), h.size, h.type);
      out[r] = w(g).mutable_data_ptr();
      stride[r] = static_cast<uint64_t>(g.stride(0));
    }
    b.grad_weights = out;
    b.grad_weight_row_strides = stride;
  }
  const dc_status_t status = g_linear_grad(&b, h.call.stream);
  Py_XDECREF(w_hidden.after(status));
  return w.after(status);
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

// bind(...): the loaded library's entry points as addresses, in the order of
// the pointers below.
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
  void** const to[] = {
      reinterpret_cast<void**>(&g_score), reinterpret_cast<void**>(&g_grad), reinterpret_cast<void**>(&g_append),
      reinterpret_cast<void**>(&g_attend), reinterpret_cast<void**>(&g_linear), reinterpret_cast<void**>(&g_linear_grad),
      reinterpret_cast<void**>(&g_append_norm), reinterpret_cast<void**>(&g_norm), reinterpret_cast<void**>(&g_norm_grad),
      reinterpret_cast<void**>(&g_prefix),
  };
  constexpr Py_ssize_t count = sizeof to / sizeof to[0];
  if (n != count) {
    PyErr_Format(PyExc_TypeError, "expected %zd addresses", count);
    return nullptr;
  }
  void* at[count];
  for (Py_ssize_t i = 0; i < count; ++i) {
    at[i] = PyLong_AsVoidPtr(args[i]);
    if (PyErr_Occurred()) return nullptr;
  }
  for (Py_ssize_t i = 0; i < count; ++i) *to[i] = at[i];
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
    {"kv_append_norm", as_function(&entry<append_norm, 15>), METH_FASTCALL, nullptr},
    {"qk_norm_rotate", as_function(&entry<norm, 11>), METH_FASTCALL, nullptr},
    {"qk_norm_rotate_backward", as_function(&entry<norm_grad, 16>), METH_FASTCALL, nullptr},
    {"prefix_attention", as_function(&entry<prefix, 13>), METH_FASTCALL, nullptr},
    {"linear_logprobs", as_function(&entry<linear, 10>), METH_FASTCALL, nullptr},
    {"linear_logprobs_backward", as_function(&entry<linear_grad, 13>), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef kModule = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, kMethods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&kModule); }
