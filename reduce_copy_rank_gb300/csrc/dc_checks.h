// dc_checks.h -- what the argument checks of the language-model operators share:
// spans of memory and whether they meet, strided tensors, paged caches, logits.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <numeric>

#include "dc.h"
#include "dc_host.h"
#include "dc_llm.h"

namespace dc {

constexpr uint64_t kTop = 1ull << 62;  // sizes and strides above this are refused

inline uint64_t addr(const void* p) { return reinterpret_cast<uint64_t>(p); }

// A device array that a call reads or writes: [lo, hi).
struct Span {
  uint64_t lo, hi;
  const char* name;
};

// A list of fixed room: an entry point of the C ABI throws nothing.
template <class T, int N>
struct Few {
  T v[N];
  int n = 0;
  void add(const T& x) {
    if (n < N) v[n++] = x;
  }
  const T* begin() const { return v; }
  const T* end() const { return v + n; }
  const T& operator[](int i) const { return v[i]; }
};
using Spans = Few<Span, 16>;

inline bool meet(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }

// Rejects a written range that meets any other range.
inline dc_status_t check_apart(const Span& out, const Spans& in, int from = 0) {
  for (int i = from; i < in.n; ++i)
    if (meet(out, in[i])) return fail(DC_ERR_OVERLAP, "%s overlaps %s", out.name, in[i].name);
  return DC_OK;
}
inline dc_status_t check_disjoint(const Spans& out, const Spans& in) {
  for (int i = 0; i < out.n; ++i) {
    const dc_status_t st = check_apart(out[i], out, i + 1);
    if (st != DC_OK) return st;
    const dc_status_t st_in = check_apart(out[i], in);
    if (st_in != DC_OK) return st_in;
  }
  return DC_OK;
}

// Checks a pointer and its alignment and sets its span of `bytes`.
inline dc_status_t take(const void* p, const char* name, uint64_t bytes, uint64_t align, Spans& to) {
  if (!p) return fail(DC_ERR_INVALID, "%s is NULL", name);
  if (addr(p) % align) return fail(DC_ERR_ALIGN, "%s must be %llu-byte aligned", name,
                                   static_cast<unsigned long long>(align));
  if (addr(p) + bytes < addr(p)) return fail(DC_ERR_INVALID, "%s wraps around", name);
  to.add(Span{addr(p), addr(p) + bytes, name});
  return DC_OK;
}

#define DC_TRY(expr)                        \
  do {                                      \
    const dc_status_t st_ = (expr);         \
    if (st_ != DC_OK) return st_;           \
  } while (0)

inline dc_status_t device(int* sms) {
  if (launch_failure_injected())
    return fail(DC_ERR_CUDA, "launch failure injected by the test_fail_launch option");
  int dev = 0;
  DC_TRY(current_device(&dev));
  return sm_count(dev, sms);
}

inline int elem_bytes(int dtype) { return dtype == kF32 ? 4 : 2; }

// ------------------------------------------------------ log probabilities ---
// Rows of one shard: `width` elements every `stride` elements.
struct Strided {
  uint64_t base, stride, width;  // bytes
  uint64_t hi;                   // end of the last row
};

using Shards = Few<Strided, kMaxRanks>;

// Whether two strided matrices of `rows` rows share a byte.
inline bool rows_meet(const Strided& a, const Strided& b, uint64_t rows) {
  if (!(a.base < b.hi && b.base < a.hi)) return false;
  if (rows > 1 && a.stride == b.stride) {
    // columns of the same rows: intervals modulo the row length
    const uint64_t d = (b.base >= a.base ? b.base - a.base : a.stride - (a.base - b.base) % a.stride) % a.stride;
    return d < a.width || d + b.width > a.stride;
  }
  return true;
}

inline dc_status_t check_temperature(double temperature) {
  // (the kernels' exponents are in units of log2(e) / temperature, in binary32)
  if (!(temperature > 0.0) || !std::isfinite(temperature) ||
      !std::isfinite(static_cast<float>(1.0 / temperature) * 1.44269504f) || static_cast<float>(1.0 / temperature) < 1e-30f)
    return fail(DC_ERR_INVALID, "temperature %g is not a positive number of usable size", temperature);
  return DC_OK;
}

inline dc_status_t check_logits(const void* const* shards, const uint64_t* widths, const uint64_t* strides, int P,
                         int64_t rows, int64_t vocab, int dtype, double temperature, const char* what,
                         Shards& out) {
  if (P < 1 || P > kMaxRanks) return fail(DC_ERR_INVALID, "ranks = %d is outside 1..%d", P, kMaxRanks);
  if (rows < 0) return fail(DC_ERR_INVALID, "rows = %lld is negative", static_cast<long long>(rows));
  if (vocab < 1 || vocab > kMaxVocab)
    return fail(DC_ERR_INVALID, "vocab = %lld is outside 1..%d", static_cast<long long>(vocab), kMaxVocab);
  if (dtype < kBF16 || dtype > kF32) return fail(DC_ERR_INVALID, "dtype %d is not DC_BF16, DC_F16 or DC_F32", dtype);
  DC_TRY(check_temperature(temperature));
  if (!shards || !widths || !strides) return fail(DC_ERR_INVALID, "%s, widths and strides must not be NULL", what);
  const uint64_t es = static_cast<uint64_t>(elem_bytes(dtype));
  uint64_t sum = 0;
  for (int r = 0; r < P; ++r) {
    if (widths[r] > static_cast<uint64_t>(kMaxVocab))
      return fail(DC_ERR_INVALID, "%s[%d] has %llu columns, more than %d", what, r,
                  static_cast<unsigned long long>(widths[r]), kMaxVocab);
    sum += widths[r];
    if (widths[r] == 0 || rows == 0) {
      out.add(Strided{0, 1, 0, 0});
      continue;
    }
    if (!shards[r]) return fail(DC_ERR_INVALID, "%s[%d] is NULL", what, r);
    if (addr(shards[r]) % es) return fail(DC_ERR_ALIGN, "%s[%d] is not aligned to its element size", what, r);
    if (rows > 1 && strides[r] < widths[r])
      return fail(DC_ERR_INVALID, "%s[%d]: rows of %llu elements every %llu overlap", what, r,
                  static_cast<unsigned long long>(widths[r]), static_cast<unsigned long long>(strides[r]));
    const uint64_t stride = rows > 1 ? strides[r] : widths[r];
    if (stride > kTop / es / static_cast<uint64_t>(rows)) return fail(DC_ERR_INVALID, "%s[%d] is too large", what, r);
    const uint64_t lo = addr(shards[r]), hi = lo + ((static_cast<uint64_t>(rows) - 1) * stride + widths[r]) * es;
    if (hi < lo) return fail(DC_ERR_INVALID, "%s[%d] wraps around", what, r);
    out.add(Strided{lo, stride * es, widths[r] * es, hi});
  }
  if (sum < static_cast<uint64_t>(vocab))
    return fail(DC_ERR_INVALID, "the shards hold %llu columns, fewer than vocab = %lld",
                static_cast<unsigned long long>(sum), static_cast<long long>(vocab));
  if (sum > static_cast<uint64_t>(kMaxVocab))
    return fail(DC_ERR_INVALID, "the shards hold %llu columns, more than %d", static_cast<unsigned long long>(sum),
                kMaxVocab);
  return DC_OK;
}

inline dc_status_t outside_shards(const Spans& out, const Shards& shards, const char* what) {
  for (const Span& o : out)
    for (const Strided& s : shards)
      if (s.width && o.lo < s.hi && s.base < o.hi) return fail(DC_ERR_OVERLAP, "%s overlaps %s", o.name, what);
  return DC_OK;
}

// --------------------------------------------------------- paged tensors ---
inline dc_status_t check_heads(int q_heads, int kv_heads, int dim, bool need_q) {
  if (kv_heads < 1 || kv_heads > 65535) return fail(DC_ERR_INVALID, "kv_heads = %d is outside 1..65535", kv_heads);
  if (q_heads < (need_q ? 1 : 0) || q_heads > 65535)
    return fail(DC_ERR_INVALID, "q_heads = %d is outside %d..65535", q_heads, need_q ? 1 : 0);
  if (dim < 1) return fail(DC_ERR_INVALID, "head dimension %d is not positive", dim);
  return DC_OK;
}

// What the norms of heads add to check_heads.
inline dc_status_t check_norm(int dim, float eps) {
  if (dim > kNormMaxDim) return fail(DC_ERR_INVALID, "normed heads have up to %d elements (got %d)", kNormMaxDim, dim);
  if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(DC_ERR_INVALID, "eps is not a finite number of at least 0");
  return DC_OK;
}

// A [n, heads, dim] tensor with strides in elements, every head 16-byte aligned.
inline dc_status_t check_tokens(const void* p, const char* name, uint64_t n, int heads, int dim, uint64_t tok, uint64_t head,
                         int es, Spans& to) {
  if (tok > kTop / 4 / std::max<uint64_t>(n, 1) || head > kTop / 4 / static_cast<uint64_t>(heads))
    return fail(DC_ERR_INVALID, "%s is too large", name);
  if ((n > 1 && tok * es % 16) || (heads > 1 && head * es % 16))
    return fail(DC_ERR_ALIGN, "%s: strides must be multiples of 16 bytes", name);
  const uint64_t last = (n > 1 ? (n - 1) * tok : 0) + (heads > 1 ? static_cast<uint64_t>(heads - 1) * head : 0);
  return take(p, name, (last + static_cast<uint64_t>(dim)) * es, 16, to);
}

// Whether elements of a strided tensor share memory: dimensions of n[i]
// entries every stride[i] elements around `inner` contiguous ones.
inline bool folds(const uint64_t* n, const uint64_t* stride, int dims, uint64_t inner) {
  int order[4] = {0, 1, 2, 3};
  std::sort(order, order + dims, [&](int a, int b) { return stride[a] < stride[b]; });
  uint64_t extent = inner;
  for (int i = 0; i < dims; ++i) {
    const int d = order[i];
    if (n[d] < 2) continue;
    if (stride[d] < extent) return true;
    extent += (n[d] - 1) * stride[d];
  }
  return false;
}

// A written [n, heads, dim] tensor must not fold onto itself.
inline dc_status_t check_written(const char* name, uint64_t n, int heads, int dim, uint64_t tok, uint64_t head) {
  const uint64_t count[2] = {n, static_cast<uint64_t>(heads)}, stride[2] = {tok, head};
  if (folds(count, stride, 2, static_cast<uint64_t>(dim))) return fail(DC_ERR_OVERLAP, "%s: its rows overlap", name);
  return DC_OK;
}

// A strided tensor as blocks of `inner` bytes: its dimensions of more than one
// place, the longest stride first.
struct Blocks {
  uint64_t base, inner;
  uint64_t n[3], stride[3];
  int dims;
};
inline Blocks blocks(const void* base, uint64_t inner, const uint64_t* n, const uint64_t* stride, int dims) {
  Blocks b{addr(base), inner, {}, {}, 0};
  for (int i = 0; i < dims; ++i) {
    if (n[i] < 2 || stride[i] == 0) continue;
    int at = b.dims++;
    for (; at > 0 && b.stride[at - 1] < stride[i]; --at) {
      b.n[at] = b.n[at - 1];
      b.stride[at] = b.stride[at - 1];
    }
    b.n[at] = n[i];
    b.stride[at] = stride[i];
  }
  return b;
}
// Bytes from the first to the last of the dimensions from `dim` on.
inline uint64_t extent(const Blocks& b, int dim) {
  uint64_t e = b.inner;
  for (int i = dim; i < b.dims; ++i) e += (b.n[i] - 1) * b.stride[i];
  return e;
}
// False if the dimensions of `a` from i on and those of `b` from j on, `off`
// bytes behind, share no byte; true if they do or it cannot be shown that they
// do not.  Where a byte of both is i * S + x = off + j * S + y, x and y inside
// their blocks of at most S bytes, x - y is off modulo S: one of two numbers.
inline bool blocks_meet(const Blocks& a, int i, const Blocks& b, int j, int64_t off) {
  const uint64_t ea = extent(a, i), eb = extent(b, j);
  if (off >= static_cast<int64_t>(ea) || off + static_cast<int64_t>(eb) <= 0) return false;
  const uint64_t sa = i < a.dims ? a.stride[i] : 0, sb = j < b.dims ? b.stride[j] : 0;
  uint64_t s = std::max(sa, sb);
  if (s == 0) return true;
  int ni = i + (sa == s), nj = j + (sb == s);
  if (extent(a, ni) > s || extent(b, nj) > s) {
    if (sa == 0 || sb == 0 || sa == sb) return true;
    s = std::gcd(sa, sb);  // both in rows of what divides both strides
    ni = i + 1;
    nj = j + 1;
    if (extent(a, ni) > s || extent(b, nj) > s) return true;
  }
  const int64_t m = static_cast<int64_t>(s), d = (off % m + m) % m;
  return blocks_meet(a, ni, b, nj, d) || blocks_meet(a, ni, b, nj, d - m);
}
inline bool blocks_meet(const Blocks& a, const Blocks& b) {
  if (!(a.base < b.base + extent(b, 0) && b.base < a.base + extent(a, 0))) return false;
  return blocks_meet(a, 0, b, 0, static_cast<int64_t>(b.base - a.base));
}

// The blocks of a [n, heads, dim] tensor.
inline Blocks token_blocks(const void* p, uint64_t n, int heads, int dim, uint64_t tok, uint64_t head, int es) {
  const uint64_t e = static_cast<uint64_t>(es), count[2] = {n, static_cast<uint64_t>(heads)}, stride[2] = {tok * e, head * e};
  return blocks(p, static_cast<uint64_t>(dim) * e, count, stride, 2);
}

inline Blocks cache_blocks(const dc_paged_cache_t& c, int64_t pages, int page_size, int heads, int dim, int es) {
  const uint64_t e = static_cast<uint64_t>(es);
  const uint64_t n[3] = {static_cast<uint64_t>(pages), static_cast<uint64_t>(page_size), static_cast<uint64_t>(heads)};
  const uint64_t stride[3] = {c.page_stride * e, c.token_stride * e, c.head_stride * e};
  return blocks(c.data, static_cast<uint64_t>(dim) * e, n, stride, 3);
}

inline dc_status_t check_cache(const dc_paged_cache_t& c, const char* name, int64_t pages, int page_size, int heads, int dim,
                        int es, bool written, PagedView* v, Spans& to) {
  if (pages < 1 || pages > 0x7FFFFFFF) return fail(DC_ERR_INVALID, "%lld pages", static_cast<long long>(pages));
  if (page_size < 1) return fail(DC_ERR_INVALID, "page_size = %d is not positive", page_size);
  const uint64_t st[3] = {c.page_stride, c.token_stride, c.head_stride};
  const uint64_t n[3] = {static_cast<uint64_t>(pages), static_cast<uint64_t>(page_size), static_cast<uint64_t>(heads)};
  uint64_t last = 0;
  for (int i = 0; i < 3; ++i) {
    if (st[i] > kTop / 8 / n[i]) return fail(DC_ERR_INVALID, "%s is too large", name);
    if (n[i] > 1 && st[i] * es % 16) return fail(DC_ERR_ALIGN, "%s: strides must be multiples of 16 bytes", name);
    if (n[i] > 1) last += (n[i] - 1) * st[i];
  }
  if (written && folds(n, st, 3, static_cast<uint64_t>(dim))) return fail(DC_ERR_OVERLAP, "%s: its tokens overlap", name);
  DC_TRY(take(c.data, name, (last + static_cast<uint64_t>(dim)) * es, 16, to));
  *v = PagedView{addr(c.data), st[0] * es, st[1] * es, st[2] * es, to[to.n - 1].lo, to[to.n - 1].hi};
  return DC_OK;
}

// The page table: `rows` rows of `width` int32, `stride` apart.
inline dc_status_t check_table(const void* p, int64_t rows, int64_t width, int64_t stride, Spans& to) {
  if (rows < 1 || rows > 0x7FFFFFFF || width < 1 || width > 0x7FFFFFFF)
    return fail(DC_ERR_INVALID, "a page table of %lld x %lld", static_cast<long long>(rows),
                static_cast<long long>(width));
  if (rows > 1 && (stride < width || stride > (1ll << 40)))
    return fail(DC_ERR_INVALID, "page table rows of %lld entries every %lld", static_cast<long long>(width),
                static_cast<long long>(stride));
  return take(p, "page_table", static_cast<uint64_t>((rows - 1) * (rows > 1 ? stride : 0) + width) * 4, 4, to);
}

}  // namespace dc
