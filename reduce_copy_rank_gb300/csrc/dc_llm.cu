// dc_llm.cu -- the C ABI of the language-model operators: argument checks,
// the choice of grid, launch.
#include <algorithm>
#include <cmath>
#include <numeric>

#include "dc.h"
#include "dc_host.h"
#include "dc_llm.h"

namespace {

using namespace dc;

constexpr uint64_t kTop = 1ull << 62;  // sizes and strides above this are refused

uint64_t addr(const void* p) { return reinterpret_cast<uint64_t>(p); }

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

bool meet(const Span& a, const Span& b) { return a.lo < b.hi && b.lo < a.hi; }

// Rejects a written range that meets any other range.
dc_status_t check_apart(const Span& out, const Spans& in, int from = 0) {
  for (int i = from; i < in.n; ++i)
    if (meet(out, in[i])) return fail(DC_ERR_OVERLAP, "%s overlaps %s", out.name, in[i].name);
  return DC_OK;
}
dc_status_t check_disjoint(const Spans& out, const Spans& in) {
  for (int i = 0; i < out.n; ++i) {
    const dc_status_t st = check_apart(out[i], out, i + 1);
    if (st != DC_OK) return st;
    const dc_status_t st_in = check_apart(out[i], in);
    if (st_in != DC_OK) return st_in;
  }
  return DC_OK;
}

// Checks a pointer and its alignment and sets its span of `bytes`.
dc_status_t take(const void* p, const char* name, uint64_t bytes, uint64_t align, Spans& to) {
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

dc_status_t device(int* sms) {
  if (launch_failure_injected())
    return fail(DC_ERR_CUDA, "launch failure injected by the test_fail_launch option");
  int dev = 0;
  DC_TRY(current_device(&dev));
  return sm_count(dev, sms);
}

int elem_bytes(int dtype) { return dtype == kF32 ? 4 : 2; }

// ------------------------------------------------------ log probabilities ---
// Rows of one shard: `width` elements every `stride` elements.
struct Strided {
  uint64_t base, stride, width;  // bytes
  uint64_t hi;                   // end of the last row
};

using Shards = Few<Strided, kMaxRanks>;

// Whether two strided matrices of `rows` rows share a byte.
bool rows_meet(const Strided& a, const Strided& b, uint64_t rows) {
  if (!(a.base < b.hi && b.base < a.hi)) return false;
  if (rows > 1 && a.stride == b.stride) {
    // columns of the same rows: intervals modulo the row length
    const uint64_t d = (b.base >= a.base ? b.base - a.base : a.stride - (a.base - b.base) % a.stride) % a.stride;
    return d < a.width || d + b.width > a.stride;
  }
  return true;
}

dc_status_t check_logits(const void* const* shards, const uint64_t* widths, const uint64_t* strides, int P,
                         int64_t rows, int64_t vocab, int dtype, double temperature, const char* what,
                         Shards& out) {
  if (P < 1 || P > kMaxRanks) return fail(DC_ERR_INVALID, "ranks = %d is outside 1..%d", P, kMaxRanks);
  if (rows < 0) return fail(DC_ERR_INVALID, "rows = %lld is negative", static_cast<long long>(rows));
  if (vocab < 1 || vocab > kMaxVocab)
    return fail(DC_ERR_INVALID, "vocab = %lld is outside 1..%d", static_cast<long long>(vocab), kMaxVocab);
  if (dtype < kBF16 || dtype > kF32) return fail(DC_ERR_INVALID, "dtype %d is not DC_BF16, DC_F16 or DC_F32", dtype);
  // (the kernels' exponents are in units of log2(e) / temperature, in binary32)
  if (!(temperature > 0.0) || !std::isfinite(temperature) ||
      !std::isfinite(static_cast<float>(1.0 / temperature) * 1.44269504f) || static_cast<float>(1.0 / temperature) < 1e-30f)
    return fail(DC_ERR_INVALID, "temperature %g is not a positive number of usable size", temperature);
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

dc_status_t outside_shards(const Spans& out, const Shards& shards, const char* what) {
  for (const Span& o : out)
    for (const Strided& s : shards)
      if (s.width && o.lo < s.hi && s.base < o.hi) return fail(DC_ERR_OVERLAP, "%s overlaps %s", o.name, what);
  return DC_OK;
}

// --------------------------------------------------------- paged tensors ---
dc_status_t check_heads(int q_heads, int kv_heads, int dim, bool need_q) {
  if (kv_heads < 1 || kv_heads > 65535) return fail(DC_ERR_INVALID, "kv_heads = %d is outside 1..65535", kv_heads);
  if (q_heads < (need_q ? 1 : 0) || q_heads > 65535)
    return fail(DC_ERR_INVALID, "q_heads = %d is outside %d..65535", q_heads, need_q ? 1 : 0);
  if (dim < 1) return fail(DC_ERR_INVALID, "head dimension %d is not positive", dim);
  return DC_OK;
}

// A [n, heads, dim] tensor with strides in elements, every head 16-byte aligned.
dc_status_t check_tokens(const void* p, const char* name, uint64_t n, int heads, int dim, uint64_t tok, uint64_t head,
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
bool folds(const uint64_t* n, const uint64_t* stride, int dims, uint64_t inner) {
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
dc_status_t check_written(const char* name, uint64_t n, int heads, int dim, uint64_t tok, uint64_t head) {
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
Blocks blocks(const void* base, uint64_t inner, const uint64_t* n, const uint64_t* stride, int dims) {
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
uint64_t extent(const Blocks& b, int dim) {
  uint64_t e = b.inner;
  for (int i = dim; i < b.dims; ++i) e += (b.n[i] - 1) * b.stride[i];
  return e;
}
// False if the dimensions of `a` from i on and those of `b` from j on, `off`
// bytes behind, share no byte; true if they do or it cannot be shown that they
// do not.  Where a byte of both is i * S + x = off + j * S + y, x and y inside
// their blocks of at most S bytes, x - y is off modulo S: one of two numbers.
bool blocks_meet(const Blocks& a, int i, const Blocks& b, int j, int64_t off) {
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
bool blocks_meet(const Blocks& a, const Blocks& b) {
  if (!(a.base < b.base + extent(b, 0) && b.base < a.base + extent(a, 0))) return false;
  return blocks_meet(a, 0, b, 0, static_cast<int64_t>(b.base - a.base));
}

// The blocks of a [n, heads, dim] tensor.
Blocks token_blocks(const void* p, uint64_t n, int heads, int dim, uint64_t tok, uint64_t head, int es) {
  const uint64_t e = static_cast<uint64_t>(es), count[2] = {n, static_cast<uint64_t>(heads)}, stride[2] = {tok * e, head * e};
  return blocks(p, static_cast<uint64_t>(dim) * e, count, stride, 2);
}

Blocks cache_blocks(const dc_paged_cache_t& c, int64_t pages, int page_size, int heads, int dim, int es) {
  const uint64_t e = static_cast<uint64_t>(es);
  const uint64_t n[3] = {static_cast<uint64_t>(pages), static_cast<uint64_t>(page_size), static_cast<uint64_t>(heads)};
  const uint64_t stride[3] = {c.page_stride * e, c.token_stride * e, c.head_stride * e};
  return blocks(c.data, static_cast<uint64_t>(dim) * e, n, stride, 3);
}

dc_status_t check_cache(const dc_paged_cache_t& c, const char* name, int64_t pages, int page_size, int heads, int dim,
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
dc_status_t check_table(const void* p, int64_t rows, int64_t width, int64_t stride, Spans& to) {
  if (rows < 1 || rows > 0x7FFFFFFF || width < 1 || width > 0x7FFFFFFF)
    return fail(DC_ERR_INVALID, "a page table of %lld x %lld", static_cast<long long>(rows),
                static_cast<long long>(width));
  if (rows > 1 && (stride < width || stride > (1ll << 40)))
    return fail(DC_ERR_INVALID, "page table rows of %lld entries every %lld", static_cast<long long>(width),
                static_cast<long long>(stride));
  return take(p, "page_table", static_cast<uint64_t>((rows - 1) * (rows > 1 ? stride : 0) + width) * 4, 4, to);
}

struct AttendPlan {
  int head_blocks, hb;
  uint32_t pieces;         // most pieces that one sequence is cut into
  uint64_t units, partial_bytes;
};

dc_status_t plan_attend(int64_t seqs, int q_heads, int kv_heads, int dim, uint64_t max_tokens, AttendPlan* a) {
  DC_TRY(check_heads(q_heads, kv_heads, dim, true));
  if (q_heads % kv_heads)
    return fail(DC_ERR_INVALID, "q_heads = %d is not a multiple of kv_heads = %d", q_heads, kv_heads);
  if (dim != 64 && dim != 96 && dim != 128 && dim != 192 && dim != 256)
    return fail(DC_ERR_INVALID, "head dimension %d is not 64, 96, 128, 192 or 256", dim);
  if (seqs < 0 || seqs > 0x7FFFFFFF) return fail(DC_ERR_INVALID, "%lld sequences", static_cast<long long>(seqs));
  if (max_tokens > 0x7FFFFFFFull)
    return fail(DC_ERR_INVALID, "sequences of up to %llu tokens", static_cast<unsigned long long>(max_tokens));
  const int group = q_heads / kv_heads;
  // no sequence of up to n tokens has more than `most` pieces at level 0; one
  // with fewer may be cut finer
  const uint32_t n = static_cast<uint32_t>(max_tokens);
  const uint32_t most = n > 512 * 128 ? kAttendMaxPieces
                                      : std::max({attend_pieces(n, 0), attend_pieces(std::min(n, kAttendShort), 0),
                                                  attend_pieces(std::min(n, kAttendTiny), 0)});
  const uint64_t kv_units = static_cast<uint64_t>(seqs) * static_cast<uint64_t>(kv_heads);
  a->hb = attend_head_block(group, kv_units, most, dim);
  a->head_blocks = (group + a->hb - 1) / a->hb;
  a->units = kv_units * static_cast<uint64_t>(a->head_blocks);
  if (a->units * kAttendMaxPieces > 0x7FFFFFFFull)
    return fail(DC_ERR_INVALID, "%llu units of work exceed a grid", static_cast<unsigned long long>(a->units));
  const uint32_t units = static_cast<uint32_t>(a->units);
  const int levels = attend_levels(dim, a->hb);
  a->pieces = 1;
  for (uint32_t s = 1; s <= most; ++s) {
    const uint32_t k = attend_level(s, units, levels);
    a->pieces = std::max(a->pieces, (s + (1u << k) - 1) >> k);
  }
  // room for this call and for any of fewer units (which may be cut finer)
  const uint64_t slots = std::max<uint64_t>(
      a->units * a->pieces, std::min<uint64_t>(a->units * most, static_cast<uint64_t>(kAttendCtas)));
  a->partial_bytes = most > 1 ? (slots * (static_cast<uint64_t>(dim) + 2) + a->units * 2 * kAttendGroups) *
                                    static_cast<uint64_t>(a->hb) * 4
                              : 0;
  return DC_OK;
}

}  // namespace

extern "C" {

dc_status_t dc_token_logprobs(const dc_token_logprobs_t* a, dc_stream_t stream) {
  read_options();
  if (!a) return fail(DC_ERR_INVALID, "the argument block is NULL");
  Shards shards;
  DC_TRY(check_logits(a->shards, a->widths, a->row_strides, a->ranks, a->rows, a->vocab, a->dtype, a->temperature,
                      "shards", shards));
  if (a->top < 0 || a->top > kMaxTop || a->top > a->vocab)
    return fail(DC_ERR_INVALID, "top = %d is outside 0..min(%d, vocab)", a->top, kMaxTop);
  if (a->top > 0 && !a->top_logprobs && !a->top_tokens)
    return fail(DC_ERR_INVALID, "top = %d but neither top_logprobs nor top_tokens is given", a->top);
  if (a->rows == 0) return ok();
  const uint64_t n = static_cast<uint64_t>(a->rows);
  Spans in, out;
  DC_TRY(take(a->tokens, "tokens", n * (a->tokens_64 ? 8 : 4), a->tokens_64 ? 8 : 4, in));
  DC_TRY(take(a->logprobs, "logprobs", n * 4, 4, out));
  if (a->entropy) DC_TRY(take(a->entropy, "entropy", n * 4, 4, out));
  if (a->lse) DC_TRY(take(a->lse, "lse", n * 4, 4, out));
  const uint64_t nt = n * static_cast<uint64_t>(a->top);
  if (a->top && a->top_logprobs) DC_TRY(take(a->top_logprobs, "top_logprobs", nt * 4, 4, out));
  if (a->top && a->top_tokens)
    DC_TRY(take(a->top_tokens, "top_tokens", nt * (a->top_tokens_64 ? 8 : 4), a->top_tokens_64 ? 8 : 4, out));
  DC_TRY(check_disjoint(out, in));
  DC_TRY(outside_shards(out, shards, "a shard of the logits"));
  int sms = 0;
  DC_TRY(device(&sms));

  ScoreParams p{};
  p.tokens = addr(a->tokens);
  p.logprobs = addr(a->logprobs);
  p.entropy = addr(a->entropy);
  p.lse = addr(a->lse);
  p.top_logprobs = a->top ? addr(a->top_logprobs) : 0;
  p.top_tokens = a->top ? addr(a->top_tokens) : 0;
  p.rows = n;
  p.inv_t = static_cast<float>(1.0 / a->temperature);
  p.vocab = static_cast<uint32_t>(a->vocab);
  const int seg = vocab_seg(a->dtype);
  p.nseg = static_cast<int32_t>((a->vocab + seg - 1) / seg);
  p.top = a->top;
  p.tokens64 = a->tokens_64 != 0;
  p.top64 = a->top_tokens_64 != 0;
  uint64_t first = 0;
  for (int r = 0; r < a->ranks && first < p.vocab; ++r) {
    if (a->widths[r] == 0) continue;
    const uint64_t end = std::min<uint64_t>(first + a->widths[r], p.vocab);  // padding is not read
    p.shard[p.P++] = LogitShard{shards[r].base, shards[r].stride, static_cast<uint32_t>(first),
                                static_cast<uint32_t>(end)};
    first = end;
  }
  // few rows: up to 8 CTAs share a row, as long as the GPU has SMs to spare
  p.cluster = 1;
  while (p.cluster < kScoreMaxCluster && p.cluster * kScoreWarps < p.nseg &&
         n * static_cast<uint64_t>(p.cluster) < 2 * static_cast<uint64_t>(sms))
    p.cluster *= 2;
  // a row of few segments: a CTA of as many warps; of a few more than 8 leave
  // idle in their last round (9 segments take 16 warps' time): 4, where there
  // are rows enough to fill the GPU so (alternatives cost a CTA more than that saves)
  p.warps = kScoreWarps;
  while (p.warps > 1 && p.warps / 2 >= p.nseg) p.warps /= 2;
  const auto slots = [&](int w) { return (p.nseg + w - 1) / w * w; };
  if (p.top == 0 && p.cluster == 1 && p.warps == kScoreWarps && n >= 6 * static_cast<uint64_t>(sms) && 8 * slots(8) >= 9 * slots(4))
    p.warps = kScoreWarps / 2;
  if (n * static_cast<uint64_t>(p.cluster) > 0x7FFFFFFFull)
    return fail(DC_ERR_INVALID, "%lld rows exceed a grid", static_cast<long long>(a->rows));
  int grid = 0;
  const cudaError_t e = launch_score(p, a->dtype, pdl_option(), static_cast<cudaStream_t>(stream), &grid);
  return check_launch(e, "token log probabilities", grid);
}

dc_status_t dc_token_logprobs_backward(const dc_token_logprobs_backward_t* a, dc_stream_t stream) {
  read_options();
  if (!a) return fail(DC_ERR_INVALID, "the argument block is NULL");
  Shards shards, grads;
  DC_TRY(check_logits(a->shards, a->widths, a->row_strides, a->ranks, a->rows, a->vocab, a->dtype, a->temperature,
                      "shards", shards));
  DC_TRY(check_logits(a->grads, a->widths, a->grad_row_strides, a->ranks, a->rows, a->vocab, a->dtype, a->temperature,
                      "grads", grads));
  if (!a->grad_logprobs && !a->grad_entropy)
    return fail(DC_ERR_INVALID, "neither grad_logprobs nor grad_entropy is given");
  if (a->rows == 0) return ok();
  const uint64_t n = static_cast<uint64_t>(a->rows);
  Spans in;
  DC_TRY(take(a->tokens, "tokens", n * (a->tokens_64 ? 8 : 4), a->tokens_64 ? 8 : 4, in));
  DC_TRY(take(a->lse, "lse", n * 4, 4, in));
  if (a->grad_logprobs) DC_TRY(take(a->grad_logprobs, "grad_logprobs", n * 4, 4, in));
  if (a->grad_entropy) {
    DC_TRY(take(a->grad_entropy, "grad_entropy", n * 4, 4, in));
    DC_TRY(take(a->entropy, "entropy", n * 4, 4, in));
  }
  for (int r = 0; r < grads.n; ++r) {
    if (grads[r].width == 0) continue;
    for (int q = 0; q < shards.n; ++q) {
      if (q > r && grads[q].width && rows_meet(grads[r], grads[q], n))
        return fail(DC_ERR_OVERLAP, "grads[%d] overlaps grads[%d]", r, q);
      if (shards[q].width == 0) continue;
      const bool same = q == r && grads[r].base == shards[q].base && grads[r].stride == shards[q].stride;
      if (!same && rows_meet(grads[r], shards[q], n))
        return fail(DC_ERR_OVERLAP, "grads[%d] overlaps shards[%d] and is not the same tensor", r, q);
    }
  }
  DC_TRY(outside_shards(in, grads, "a shard of the gradient"));
  int sms = 0;
  DC_TRY(device(&sms));

  GradParams p{};
  p.tokens = addr(a->tokens);
  p.lse = addr(a->lse);
  p.entropy = addr(a->entropy);
  p.grad_logprobs = addr(a->grad_logprobs);
  p.grad_entropy = addr(a->grad_entropy);
  p.rows = n;
  p.inv_t = static_cast<float>(1.0 / a->temperature);
  p.vocab = static_cast<uint32_t>(a->vocab);
  p.tokens64 = a->tokens_64 != 0;
  const uint64_t per = 16 / static_cast<uint64_t>(elem_bytes(a->dtype));
  uint64_t first = 0, chunks = 0;
  for (int r = 0; r < a->ranks; ++r) {
    if (a->widths[r] == 0) continue;
    p.shard[p.P++] = GradShard{shards[r].base, shards[r].stride, grads[r].base, grads[r].stride,
                               static_cast<uint32_t>(first), static_cast<uint32_t>(a->widths[r]),
                               static_cast<uint32_t>(chunks), 0u};
    first += a->widths[r];
    chunks += std::max<uint64_t>(1, (a->widths[r] / per + kGradChunk - 1) / kGradChunk);
  }
  p.chunks = static_cast<uint32_t>(chunks);
  int grid = 0;
  const cudaError_t e = launch_score_grad(p, a->dtype, pdl_option(), static_cast<cudaStream_t>(stream), &grid);
  return check_launch(e, "token log probabilities' gradient", grid);
}

dc_status_t dc_kv_append(const dc_kv_append_t* a, dc_stream_t stream) {
  read_options();
  if (!a) return fail(DC_ERR_INVALID, "the argument block is NULL");
  if (a->dtype < kBF16 || a->dtype > kF32)
    return fail(DC_ERR_INVALID, "dtype %d is not DC_BF16, DC_F16 or DC_F32", a->dtype);
  const int es = elem_bytes(a->dtype), per = 16 / es;
  DC_TRY(check_heads(a->q_heads, a->kv_heads, a->dim, false));
  if (a->dim % per || a->dim > 1024)
    return fail(DC_ERR_INVALID, "head dimension %d is not a multiple of %d up to 1024", a->dim, per);
  if (a->rotary_dim < 0 || a->rotary_dim > a->dim || a->rotary_dim % (a->interleaved ? per : 2 * per))
    return fail(DC_ERR_INVALID, "rotary_dim = %d is not a multiple of %d up to the head dimension", a->rotary_dim,
                a->interleaved ? per : 2 * per);
  if (a->tokens < 0 || a->tokens > 0x7FFFFFFF / 512)
    return fail(DC_ERR_INVALID, "%lld tokens", static_cast<long long>(a->tokens));
  if (a->tokens == 0) return ok();
  const uint64_t n = static_cast<uint64_t>(a->tokens);
  AppendParams p{};
  Spans in, cache, out;
  DC_TRY(check_tokens(a->k, "k", n, a->kv_heads, a->dim, a->k_token_stride, a->k_head_stride, es, in));
  DC_TRY(check_tokens(a->v, "v", n, a->kv_heads, a->dim, a->v_token_stride, a->v_head_stride, es, in));
  DC_TRY(take(a->positions, "positions", n * 4, 4, in));
  DC_TRY(take(a->seqs, "seqs", n * 4, 4, in));
  DC_TRY(check_table(a->page_table, a->table_rows, a->table_width, a->table_stride, in));
  if (a->rotary_dim) {
    if (a->cos_sin_rows < 1 || a->cos_sin_rows > (1ll << 40))
      return fail(DC_ERR_INVALID, "cos_sin has %lld rows", static_cast<long long>(a->cos_sin_rows));
    DC_TRY(take(a->cos_sin, "cos_sin", static_cast<uint64_t>(a->cos_sin_rows) * a->rotary_dim * 4, 4, in));
  }
  DC_TRY(check_cache(a->k_cache, "k_cache", a->num_pages, a->page_size, a->kv_heads, a->dim, es, true, &p.kc, cache));
  DC_TRY(check_cache(a->v_cache, "v_cache", a->num_pages, a->page_size, a->kv_heads, a->dim, es, true, &p.vc, cache));
  // (the caches may be interleaved in one tensor: their spans may meet, their tokens' heads not)
  if (blocks_meet(cache_blocks(a->k_cache, a->num_pages, a->page_size, a->kv_heads, a->dim, es),
                  cache_blocks(a->v_cache, a->num_pages, a->page_size, a->kv_heads, a->dim, es)))
    return fail(DC_ERR_OVERLAP, "k_cache overlaps v_cache");
  for (const Span& c : cache) DC_TRY(check_apart(c, in));
  if (a->q_heads) {
    Spans q;
    DC_TRY(check_tokens(a->q, "q", n, a->q_heads, a->dim, a->q_token_stride, a->q_head_stride, es, q));
    DC_TRY(check_tokens(a->q_out, "q_out", n, a->q_heads, a->dim, a->q_out_token_stride, a->q_out_head_stride, es, out));
    DC_TRY(check_written("q_out", n, a->q_heads, a->dim, a->q_out_token_stride, a->q_out_head_stride));
    const bool same = a->q == a->q_out && a->q_token_stride == a->q_out_token_stride &&
                      a->q_head_stride == a->q_out_head_stride;
    if (!same) {
      DC_TRY(check_disjoint(out, q));
      DC_TRY(check_disjoint(out, in));
    } else {
      // in place: heads of queries beside those of keys and values in one tensor are fine
      const Blocks qb = token_blocks(a->q_out, n, a->q_heads, a->dim, a->q_out_token_stride, a->q_out_head_stride, es);
      if (blocks_meet(qb, token_blocks(a->k, n, a->kv_heads, a->dim, a->k_token_stride, a->k_head_stride, es)))
        return fail(DC_ERR_OVERLAP, "q_out overlaps k");
      if (blocks_meet(qb, token_blocks(a->v, n, a->kv_heads, a->dim, a->v_token_stride, a->v_head_stride, es)))
        return fail(DC_ERR_OVERLAP, "q_out overlaps v");
      DC_TRY(check_apart(out[0], in, 2));  // (k and v are the first two)
    }
    DC_TRY(check_disjoint(out, cache));
    for (const Span& c : cache) DC_TRY(check_apart(c, q));
  }
  int sms = 0;
  DC_TRY(device(&sms));
  const uint64_t e8 = static_cast<uint64_t>(es);
  p.q = addr(a->q);
  p.q_token = a->q_token_stride * e8;
  p.q_head = a->q_head_stride * e8;
  p.qo = addr(a->q_out);
  p.qo_token = a->q_out_token_stride * e8;
  p.qo_head = a->q_out_head_stride * e8;
  p.k = addr(a->k);
  p.k_token = a->k_token_stride * e8;
  p.k_head = a->k_head_stride * e8;
  p.v = addr(a->v);
  p.v_token = a->v_token_stride * e8;
  p.v_head = a->v_head_stride * e8;
  p.positions = addr(a->positions);
  p.seqs = addr(a->seqs);
  p.table = addr(a->page_table);
  p.cos_sin = addr(a->cos_sin);
  p.tokens = n;
  p.table_stride = a->table_rows > 1 ? a->table_stride : 0;
  p.cos_rows = a->cos_sin_rows;
  p.num_pages = a->num_pages;
  p.page_size = static_cast<uint32_t>(a->page_size);
  p.table_width = static_cast<uint32_t>(a->table_width);
  p.num_seqs = static_cast<uint32_t>(a->table_rows);
  p.q_heads = a->q_heads;
  p.kv_heads = a->kv_heads;
  p.dim = a->dim;
  p.rot = a->rotary_dim;
  p.interleaved = a->interleaved != 0;
  int grid = 0;
  const cudaError_t e = launch_append(p, a->dtype, sms, pdl_option(), static_cast<cudaStream_t>(stream), &grid);
  return check_launch(e, "cache append", grid);
}

size_t dc_attention_workspace_bytes(int64_t seqs, int q_heads, int kv_heads, int dim, int64_t max_tokens) {
  AttendPlan plan{};
  if (max_tokens < 0 || plan_attend(seqs, q_heads, kv_heads, dim, static_cast<uint64_t>(max_tokens), &plan) != DC_OK)
    return 0;
  // (1024: a workspace of a call that needs none is not empty; 0 says that there is no such call)
  return static_cast<size_t>(plan.partial_bytes ? (kAttendCounterBytes + plan.partial_bytes + 255) / 256 * 256 : 1024);
}

dc_status_t dc_paged_attention(const dc_paged_attention_t* a, dc_stream_t stream) {
  read_options();
  if (!a) return fail(DC_ERR_INVALID, "the argument block is NULL");
  if (a->dtype != kBF16 && a->dtype != kF16) return fail(DC_ERR_INVALID, "dtype %d is not DC_BF16 or DC_F16", a->dtype);
  if (a->page_size < 1) return fail(DC_ERR_INVALID, "page_size = %d is not positive", a->page_size);
  if (a->window < 0) return fail(DC_ERR_INVALID, "window = %d is negative", a->window);
  if (!std::isfinite(a->scale)) return fail(DC_ERR_INVALID, "scale is not finite");
  Spans in, out;
  if (a->seqs == 0) return ok();
  DC_TRY(check_table(a->page_table, a->seqs, a->table_width, a->table_stride, in));
  uint64_t most = static_cast<uint64_t>(a->table_width) * static_cast<uint64_t>(a->page_size);
  if (a->window > 0) most = std::min<uint64_t>(most, static_cast<uint64_t>(a->window));
  AttendPlan plan{};
  DC_TRY(plan_attend(a->seqs, a->q_heads, a->kv_heads, a->dim, most, &plan));
  const uint64_t n = static_cast<uint64_t>(a->seqs);
  AttendParams p{};
  DC_TRY(check_tokens(a->q, "q", n, a->q_heads, a->dim, a->q_seq_stride, a->q_head_stride, 2, in));
  DC_TRY(take(a->lengths, "lengths", n * 4, 4, in));
  DC_TRY(check_cache(a->k_cache, "k_cache", a->num_pages, a->page_size, a->kv_heads, a->dim, 2, false, &p.kc, in));
  DC_TRY(check_cache(a->v_cache, "v_cache", a->num_pages, a->page_size, a->kv_heads, a->dim, 2, false, &p.vc, in));
  DC_TRY(check_tokens(a->out, "out", n, a->q_heads, a->dim, a->out_seq_stride, a->out_head_stride, 2, out));
  DC_TRY(check_written("out", n, a->q_heads, a->dim, a->out_seq_stride, a->out_head_stride));
  if (a->lse) DC_TRY(take(a->lse, "lse", n * static_cast<uint64_t>(a->q_heads) * 4, 4, out));
  if (plan.partial_bytes) {  // the counters, then the pieces' partial results
    if (kAttendCounterBytes + plan.partial_bytes > a->workspace_bytes)
      return fail(DC_ERR_INVALID, "the workspace holds %llu bytes; dc_attention_workspace_bytes says %llu",
                  static_cast<unsigned long long>(a->workspace_bytes),
                  static_cast<unsigned long long>(dc_attention_workspace_bytes(
                      a->seqs, a->q_heads, a->kv_heads, a->dim, static_cast<int64_t>(most))));
    DC_TRY(take(a->workspace, "workspace", a->workspace_bytes, 16, out));
  }
  DC_TRY(check_disjoint(out, in));
  int sms = 0;
  DC_TRY(device(&sms));
  p.q = addr(a->q);
  p.q_seq = a->q_seq_stride * 2;
  p.q_head = a->q_head_stride * 2;
  p.out = addr(a->out);
  p.out_seq = a->out_seq_stride * 2;
  p.out_head = a->out_head_stride * 2;
  p.lse = addr(a->lse);
  p.table = addr(a->page_table);
  p.lengths = addr(a->lengths);
  p.counters = addr(a->workspace);
  p.partial = addr(a->workspace) + kAttendCounterBytes;
  p.table_stride = a->seqs > 1 ? a->table_stride : 0;
  p.num_pages = a->num_pages;
  p.page_size = static_cast<uint32_t>(a->page_size);
  p.table_width = static_cast<uint32_t>(a->table_width);
  p.seqs = static_cast<int32_t>(a->seqs);
  p.q_heads = a->q_heads;
  p.kv_heads = a->kv_heads;
  p.group = a->q_heads / a->kv_heads;
  p.head_blocks = plan.head_blocks;
  p.hb = plan.hb;
  p.window = a->window;
  p.units = static_cast<int32_t>(plan.units);
  p.pieces = static_cast<int32_t>(plan.pieces);
  // Few CTAs, all resident at once, and few enough pieces: a unit's CTAs are a
  // cluster and join them in shared memory.  Measured, us, workspace / cluster:
  // one sequence of 1025 tokens, 8/1 heads of 128 (5 pieces): 8.2 / 6.9; of 4096
  // (16 pieces, two clusters and the workspace): 8.1 / 10.
  const uint32_t resident = static_cast<uint32_t>(sms) * (a->dim <= 128 ? 2u : 1u);
  const uint32_t c = plan.pieces > 4 ? 8u : plan.pieces > 2 ? 4u : 2u;
  const bool cluster = plan.pieces > 1 && plan.pieces <= c && plan.units * c <= resident;
  p.cluster = cluster ? static_cast<int32_t>(c) : 1;
  p.places = cluster ? static_cast<int32_t>(c) : p.pieces;
  // A table with room for much longer sequences than most are must not flood
  // the GPU with CTAs that find nothing to do (about 0.5 us each, two at a time
  // on an SM): beyond four times the CTAs that fill it, a unit's take turns.
  if (!cluster && plan.pieces > 8 && plan.units * plan.pieces > 4 * kAttendCtas)
    p.places = static_cast<int32_t>(std::max<uint64_t>(8, std::min<uint64_t>(plan.pieces, 4 * kAttendCtas / plan.units)));
  // more units than the counters have room for (29127 at least): a CTA each
  if (!cluster && plan.pieces > 1 && plan.units * attend_counters(plan.pieces) * 4 > kAttendCounterBytes) p.places = 1;
  p.page_shift = (p.page_size & (p.page_size - 1)) == 0 ? __builtin_ctz(p.page_size) : -1;
  p.scale = a->scale;
  int grid = 0;
  const cudaError_t e = launch_attend(p, a->dtype, a->dim, pdl_option(), static_cast<cudaStream_t>(stream), &grid);
  return check_launch(e, "paged attention", grid);
}

}  // extern "C"
