// dc_llm_more.cu -- the C ABI of the operators around a rollout and a training
// step on it: log probabilities from hidden rows, normed and rotated queries and
// keys.  Argument checks, the cut of the work, launches.
#include "dc_checks.h"

namespace {

using namespace dc;

constexpr int64_t kMaxLinearRows = 1 << 24;
constexpr int64_t kMaxHidden = 1 << 20;

uint64_t round_up(uint64_t n, uint64_t to) { return (n + to - 1) / to * to; }

// A [rows, columns] matrix of 16-bit elements whose rows TMA can copy: 16-byte
// aligned, `columns` a multiple of 8.
dc_status_t check_matrix(const void* p, uint64_t rows, uint64_t columns, uint64_t stride, const char* name, int r, Strided* out) {
  char what[48];
  if (r < 0) std::snprintf(what, sizeof what, "%s", name);
  else std::snprintf(what, sizeof what, "%s[%d]", name, r);
  *out = Strided{0, 1, 0, 0};
  if (rows == 0) return DC_OK;
  if (!p) return fail(DC_ERR_INVALID, "%s is NULL", what);
  if (rows < 2) stride = columns;
  if (stride < columns)
    return fail(DC_ERR_INVALID, "%s: rows of %llu elements every %llu overlap", what,
                static_cast<unsigned long long>(columns), static_cast<unsigned long long>(stride));
  if (stride > (1ull << 38)) return fail(DC_ERR_INVALID, "%s is too large", what);
  if (addr(p) % 16 || stride % 8) return fail(DC_ERR_ALIGN, "%s: rows must be 16-byte aligned", what);
  const uint64_t lo = addr(p), hi = lo + ((rows - 1) * stride + columns) * 2;
  if (hi < lo) return fail(DC_ERR_INVALID, "%s wraps around", what);
  *out = Strided{lo, stride * 2, columns * 2, hi};
  return DC_OK;
}

// What both directions take: hidden rows, the head's shards, tokens.
struct Head {
  Strided hidden;
  Shards weights;
  Spans in;
};

dc_status_t check_head(const void* hidden, uint64_t hidden_stride, const void* const* weights, const uint64_t* widths,
                       const uint64_t* strides, const void* tokens, int64_t rows, int64_t size, int64_t vocab,
                       double temperature, int ranks, int dtype, int tokens_64, Head* h) {
  if (ranks < 1 || ranks > kMaxRanks) return fail(DC_ERR_INVALID, "ranks = %d is outside 1..%d", ranks, kMaxRanks);
  if (rows < 0 || rows > kMaxLinearRows)
    return fail(DC_ERR_INVALID, "rows = %lld is outside 0..%lld", static_cast<long long>(rows), static_cast<long long>(kMaxLinearRows));
  if (size < 8 || size > kMaxHidden || size % 8)
    return fail(DC_ERR_INVALID, "a hidden size of %lld is not a multiple of 8 up to %lld", static_cast<long long>(size),
                static_cast<long long>(kMaxHidden));
  if (vocab < 1 || vocab > kMaxVocab)
    return fail(DC_ERR_INVALID, "vocab = %lld is outside 1..%d", static_cast<long long>(vocab), kMaxVocab);
  if (dtype != kBF16 && dtype != kF16) return fail(DC_ERR_INVALID, "dtype %d is not DC_BF16 or DC_F16", dtype);
  DC_TRY(check_temperature(temperature));
  if (!weights || !widths || !strides) return fail(DC_ERR_INVALID, "weights, widths and strides must not be NULL");
  uint64_t sum = 0;
  for (int r = 0; r < ranks; ++r) {
    if (widths[r] > static_cast<uint64_t>(kMaxVocab))
      return fail(DC_ERR_INVALID, "weights[%d] has %llu rows, more than %d", r, static_cast<unsigned long long>(widths[r]), kMaxVocab);
    sum += widths[r];
    Strided m;
    DC_TRY(check_matrix(weights[r], widths[r], static_cast<uint64_t>(size), strides[r], "weights", r, &m));
    h->weights.add(m);
  }
  if (sum < static_cast<uint64_t>(vocab) || sum > static_cast<uint64_t>(kMaxVocab))
    return fail(DC_ERR_INVALID, "the shards hold %llu columns; vocab = %lld, and at most %d", static_cast<unsigned long long>(sum),
                static_cast<long long>(vocab), kMaxVocab);
  DC_TRY(check_matrix(hidden, static_cast<uint64_t>(rows), static_cast<uint64_t>(size), hidden_stride, "hidden", -1, &h->hidden));
  if (rows) DC_TRY(take(tokens, "tokens", static_cast<uint64_t>(rows) * (tokens_64 ? 8 : 4), tokens_64 ? 8 : 4, h->in));
  return DC_OK;
}

// The forward's workspace: every tile's parts, then the tokens' logits.
uint64_t stats_bytes(uint64_t rows, uint64_t tiles) { return rows * (tiles * (kLinearN / kLinearPart) * 16 + 4); }
// The gradient's: its power of two, then what d loses at the rows' tokens, where those
// are, and how dW's rows find it; d of one chunk of the vocabulary, and the sums of d W,
// a slice each.
uint64_t lost_bytes(uint64_t rows) { return round_up(rows * 4, 256); }
uint64_t marks_bytes(uint64_t rows, uint64_t stride) { return round_up(linear_marks(rows, stride), 256); }
uint64_t chunk_stride(uint64_t columns) { return round_up(std::min<uint64_t>(columns, kLinearChunk), kLinearN) * 2; }
uint64_t d_bytes(uint64_t rows, uint64_t stride) { return round_up(rows * stride, 256); }

// dW's sums of one tile a pair of CTAs, where a sum takes more than one run.
uint64_t tile_bytes(uint64_t rows) { return rows > kLinearChunk ? kLinearPairs * static_cast<uint64_t>(kLinearM) * kLinearN * 4 : 0; }
uint64_t table_bytes(uint64_t rows, uint64_t stride) { return rows > kLostFew ? round_up(stride * 2, 256) : 0; }
uint64_t next_bytes(uint64_t rows) { return rows > kLostFew ? round_up(rows * 4, 256) : 0; }
uint64_t sums_bytes(uint64_t rows, uint64_t stride, uint64_t size) { return round_up(linear_lost_places(rows, stride) * size * 4, 256); }
// All of it but the sums of d W.
uint64_t fixed_bytes(uint64_t rows, uint64_t stride, uint64_t size) {
  return 256 + lost_bytes(rows) + marks_bytes(rows, stride) + table_bytes(rows, stride) + next_bytes(rows) + sums_bytes(rows, stride, size) +
         d_bytes(rows, stride) + tile_bytes(rows);
}

dc_status_t check_workspace(void* p, uint64_t have, uint64_t need, Spans& out) {
  if (have < need)
    return fail(DC_ERR_INVALID, "the workspace holds %llu bytes, this call needs %llu (dc_linear_logprobs_workspace_bytes)",
                static_cast<unsigned long long>(have), static_cast<unsigned long long>(need));
  return take(p, "workspace", have, 256, out);
}

// Written spans meet neither one another, what is read, nor the matrices.
dc_status_t check_head_outputs(const Spans& out, const Head& h) {
  DC_TRY(check_disjoint(out, h.in));
  DC_TRY(outside_shards(out, h.weights, "a shard of the weights"));
  Shards hidden;
  hidden.add(h.hidden);
  return outside_shards(out, hidden, "hidden");
}

// ------------------------------------------------- normed queries and keys ---
struct NormShape {
  int64_t tokens;
  int q_heads, kv_heads, dim, rotary, dtype;
  bool interleaved;
};

dc_status_t check_norm_shape(const NormShape& s, float eps) {
  if (s.dtype < kBF16 || s.dtype > kF32) return fail(DC_ERR_INVALID, "dtype %d is not DC_BF16, DC_F16 or DC_F32", s.dtype);
  const int per = 16 / elem_bytes(s.dtype);
  DC_TRY(check_heads(s.q_heads, s.kv_heads, s.dim, true));
  if (s.dim % per) return fail(DC_ERR_INVALID, "head dimension %d is not a multiple of %d", s.dim, per);
  DC_TRY(check_norm(s.dim, eps));
  if (s.rotary < 0 || s.rotary > s.dim || s.rotary % (s.interleaved ? per : 2 * per))
    return fail(DC_ERR_INVALID, "rotary_dim = %d is not a multiple of %d up to the head dimension", s.rotary,
                s.interleaved ? per : 2 * per);
  if (s.tokens < 0 || s.tokens > 0x7FFFFFFF) return fail(DC_ERR_INVALID, "%lld tokens", static_cast<long long>(s.tokens));
  return DC_OK;
}

// The positions, angles and weights of both directions.
dc_status_t take_norm_inputs(const NormShape& s, const void* positions, const void* cos_sin, int64_t rows, const void* q_norm,
                             const void* k_norm, bool norm_32, NormParams& p, Spans& in) {
  DC_TRY(take(positions, "positions", static_cast<uint64_t>(s.tokens) * 4, 4, in));
  if (s.rotary) {
    if (rows < 1 || rows > (1ll << 40)) return fail(DC_ERR_INVALID, "cos_sin has %lld rows", static_cast<long long>(rows));
    DC_TRY(take(cos_sin, "cos_sin", static_cast<uint64_t>(rows) * s.rotary * 4, 4, in));
  }
  const int es = norm_32 ? 4 : elem_bytes(s.dtype);
  DC_TRY(take(q_norm, "q_norm", static_cast<uint64_t>(s.dim) * es, es, in));
  DC_TRY(take(k_norm, "k_norm", static_cast<uint64_t>(s.dim) * es, es, in));
  p.positions = addr(positions);
  p.cos_sin = s.rotary ? addr(cos_sin) : 0;
  p.tokens = static_cast<uint64_t>(s.tokens);
  p.cos_rows = rows;
  p.jobs = 2;
  p.dim = s.dim;
  p.rot = s.rotary;
  p.w32 = norm_32;
  p.job[0].w = addr(q_norm);
  p.job[1].w = addr(k_norm);
  p.job[0].heads = s.q_heads;
  p.job[1].heads = s.kv_heads;
  return DC_OK;
}

struct Heads {
  const dc_heads_t* t;
  const char* name;
  int heads;
};

dc_status_t take_heads(const NormShape& s, const Heads& h, HeadsView* v, Spans& to) {
  const uint64_t es = static_cast<uint64_t>(elem_bytes(s.dtype));
  DC_TRY(check_tokens(h.t->data, h.name, static_cast<uint64_t>(s.tokens), h.heads, s.dim, h.t->token_stride, h.t->head_stride,
                      static_cast<int>(es), to));
  *v = HeadsView{addr(h.t->data), h.t->token_stride * es, h.t->head_stride * es};
  return DC_OK;
}

Blocks heads_blocks(const NormShape& s, const Heads& h) {
  return token_blocks(h.t->data, static_cast<uint64_t>(s.tokens), h.heads, s.dim, h.t->token_stride, h.t->head_stride,
                      elem_bytes(s.dtype));
}

bool same_place(const Heads& a, const Heads& b) {
  return a.t->data == b.t->data && a.t->token_stride == b.t->token_stride && a.t->head_stride == b.t->head_stride && a.heads == b.heads;
}

// The written heads fold onto neither themselves nor one another, and meet what
// is read only where they are exactly it (out[i] and in_place[i]).
dc_status_t check_heads_apart(const NormShape& s, const Heads* out, const Heads* in_place, int n_out, const Heads* in, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    DC_TRY(check_written(out[i].name, static_cast<uint64_t>(s.tokens), out[i].heads, s.dim, out[i].t->token_stride,
                         out[i].t->head_stride));
    const Blocks b = heads_blocks(s, out[i]);
    for (int k = i + 1; k < n_out; ++k)
      if (blocks_meet(b, heads_blocks(s, out[k]))) return fail(DC_ERR_OVERLAP, "%s overlaps %s", out[i].name, out[k].name);
    for (int k = 0; k < n_in; ++k) {
      if (in[k].t == in_place[i].t && same_place(out[i], in[k])) continue;
      if (blocks_meet(b, heads_blocks(s, in[k]))) return fail(DC_ERR_OVERLAP, "%s overlaps %s", out[i].name, in[k].name);
    }
  }
  return DC_OK;
}

uint64_t norm_workspace(int dim) { return 2ull * kNormGradCtas * static_cast<uint64_t>(dim) * 4; }

}  // namespace

extern "C" {

size_t dc_linear_logprobs_workspace_bytes(int64_t rows, int64_t hidden_size, int64_t columns, int backward) {
  if (rows < 0 || rows > kMaxLinearRows || hidden_size < 8 || hidden_size > kMaxHidden || hidden_size % 8 || columns < 1 ||
      columns > kMaxVocab) {
    fail(DC_ERR_INVALID, "no such head: %lld rows of %lld, %lld columns", static_cast<long long>(rows),
         static_cast<long long>(hidden_size), static_cast<long long>(columns));
    return 0;
  }
  const uint64_t n = static_cast<uint64_t>(std::max<int64_t>(rows, 1)), v = static_cast<uint64_t>(columns);
  // (a shard's last tile may be narrower: at most one more tile a rank)
  if (!backward) return round_up(stats_bytes(n, (v + kLinearN - 1) / kLinearN + kMaxRanks), 256);
  return fixed_bytes(n, chunk_stride(v), static_cast<uint64_t>(hidden_size)) +
         round_up(n * static_cast<uint64_t>(hidden_size) * 4 * linear_slices(static_cast<uint32_t>(hidden_size)), 256);
}

dc_status_t dc_linear_logprobs(const dc_linear_logprobs_t* a, dc_stream_t stream) {
  read_options();
  if (!a) return fail(DC_ERR_INVALID, "the argument block is NULL");
  Head h;
  DC_TRY(check_head(a->hidden, a->hidden_row_stride, a->weights, a->widths, a->weight_row_strides, a->tokens, a->rows,
                    a->hidden_size, a->vocab, a->temperature, a->ranks, a->dtype, a->tokens_64, &h));
  if (a->rows == 0) return ok();
  const uint64_t n = static_cast<uint64_t>(a->rows), size = static_cast<uint64_t>(a->hidden_size);
  Spans out;
  DC_TRY(take(a->logprobs, "logprobs", n * 4, 4, out));
  if (a->entropy) DC_TRY(take(a->entropy, "entropy", n * 4, 4, out));
  if (a->lse) DC_TRY(take(a->lse, "lse", n * 4, 4, out));
  LinearOperand b[kMaxRanks];
  LinearShard shard[kMaxRanks];
  LinearParams p{};
  uint64_t first = 0, tiles = 0;
  for (int r = 0; r < a->ranks && first < static_cast<uint64_t>(a->vocab); ++r) {
    if (a->widths[r] == 0) continue;
    const uint64_t end = std::min<uint64_t>(first + a->widths[r], static_cast<uint64_t>(a->vocab));
    b[p.shards] = LinearOperand{h.weights[r].base, end - first, size, h.weights[r].stride};  // (padding is not read)
    shard[p.shards++] = LinearShard{static_cast<uint32_t>(tiles), static_cast<uint32_t>(first), static_cast<uint32_t>(end), 0};
    tiles += (end - first + kLinearN - 1) / kLinearN;
    first = end;
  }
  DC_TRY(check_workspace(a->workspace, a->workspace_bytes, stats_bytes(n, tiles), out));
  DC_TRY(check_head_outputs(out, h));
  p.m = static_cast<uint32_t>(n);
  p.m_tiles = static_cast<uint32_t>((n + kLinearM - 1) / kLinearM);
  p.n_tiles = static_cast<uint32_t>(tiles);
  if (static_cast<uint64_t>(p.m_tiles) * tiles > 0x7FFFFFFFull)
    return fail(DC_ERR_INVALID, "%lld rows of %llu tiles are too many", static_cast<long long>(a->rows), static_cast<unsigned long long>(tiles));
  int sms = 0;
  DC_TRY(device(&sms));
  p.k_blocks = static_cast<uint32_t>((size + kLinearK - 1) / kLinearK);
  p.vocab = static_cast<uint32_t>(a->vocab);
  p.inv_t = static_cast<float>(1.0 / a->temperature);
  p.tokens64 = a->tokens_64 != 0;
  p.rows = n;
  p.tokens = addr(a->tokens);
  p.part = addr(a->workspace);
  p.target = p.part + tiles * (kLinearN / kLinearPart) * n * 16;
  p.wait_ns = wait_limit_option();
  p.late = tensor_late_option();
  const LinearOperand x{h.hidden.base, n, size, h.hidden.stride};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  int grid = 0;
  cudaError_t e = launch_linear(kLinearStats, a->dtype, p, x, b, shard, sms, pdl_option(), s, &grid);
  DC_TRY(check_launch(e, "log probabilities of a linear head", grid));
  LinearFinishParams f{};
  f.part = p.part;
  f.target = p.target;
  f.tokens = p.tokens;
  f.logprobs = addr(a->logprobs);
  f.entropy = addr(a->entropy);
  f.lse = addr(a->lse);
  f.rows = n;
  f.parts = p.n_tiles * (kLinearN / kLinearPart);
  f.vocab = p.vocab;
  f.tokens64 = p.tokens64;
  f.inv_t = p.inv_t;
  e = launch_linear_finish(f, pdl_option(), s, &grid);
  return check_launch(e, "log probabilities of a linear head", grid);
}

dc_status_t dc_linear_logprobs_backward(const dc_linear_logprobs_backward_t* a, dc_stream_t stream) {
  read_options();
  if (!a) return fail(DC_ERR_INVALID, "the argument block is NULL");
  Head h;
  DC_TRY(check_head(a->hidden, a->hidden_row_stride, a->weights, a->widths, a->weight_row_strides, a->tokens, a->rows,
                    a->hidden_size, a->vocab, a->temperature, a->ranks, a->dtype, a->tokens_64, &h));
  const uint64_t n = static_cast<uint64_t>(a->rows), size = static_cast<uint64_t>(a->hidden_size);
  const uint64_t vocab = static_cast<uint64_t>(a->vocab);
  // (without rows the vectors of rows may be NULL: only the weights' gradient, zeros, is written)
  if (n && !a->grad_logprobs && !a->grad_entropy)
    return fail(DC_ERR_INVALID, "neither grad_logprobs nor grad_entropy is given");
  const bool want_h = a->grad_hidden != nullptr, want_w = a->grad_weights != nullptr;
  if (n && !want_h && !want_w) return fail(DC_ERR_INVALID, "neither grad_hidden nor grad_weights is given");
  if (want_w && !a->grad_weight_row_strides) return fail(DC_ERR_INVALID, "grad_weights need their strides");
  // what is written: grad_hidden, then the shards' gradients
  Strided gh{0, 1, 0, 0};
  Shards gw;
  if (want_h) DC_TRY(check_matrix(a->grad_hidden, n, size, a->grad_hidden_row_stride, "grad_hidden", -1, &gh));
  uint64_t widest = 0, chunks = 0, first = 0;
  for (int r = 0; r < a->ranks; ++r) {
    Strided m{0, 1, 0, 0};
    if (want_w)
      DC_TRY(check_matrix(a->grad_weights[r], a->widths[r], size, a->grad_weight_row_strides[r], "grad_weights", r, &m));
    gw.add(m);
    const uint64_t held = first < vocab ? std::min<uint64_t>(a->widths[r], vocab - first) : 0;
    widest = std::max<uint64_t>(widest, linear_chunk(static_cast<uint32_t>(held)));
    if (held) chunks += (held + linear_chunk(static_cast<uint32_t>(held)) - 1) / linear_chunk(static_cast<uint32_t>(held));
    first += a->widths[r];
  }
  auto apart = [&](const Strided& x, const char* name, int r) -> dc_status_t {
    if (x.width == 0) return DC_OK;
    const char* with = nullptr;
    if (h.hidden.width && rows_meet(x, h.hidden, 2)) with = "hidden";
    for (int q = 0; q < h.weights.n; ++q)
      if (h.weights[q].width && rows_meet(x, h.weights[q], 2)) with = "a shard of the weights";
    for (int q = r + 1; q < gw.n; ++q)
      if (gw[q].width && rows_meet(x, gw[q], 2)) with = "a shard of grad_weights";
    return with ? fail(DC_ERR_OVERLAP, "%s overlaps %s", name, with) : DC_OK;
  };
  DC_TRY(apart(gh, "grad_hidden", -1));
  for (int r = 0; r < gw.n; ++r) DC_TRY(apart(gw[r], "grad_weights", r));
  Spans out;
  const uint64_t stride = chunk_stride(widest);
  const uint32_t slices = linear_slices(static_cast<uint32_t>(size));
  const bool sum = want_h && (chunks > 1 || slices > 1);
  if (n) {
    DC_TRY(take(a->lse, "lse", n * 4, 4, h.in));
    if (a->grad_logprobs) DC_TRY(take(a->grad_logprobs, "grad_logprobs", n * 4, 4, h.in));
    if (a->grad_entropy) {
      DC_TRY(take(a->grad_entropy, "grad_entropy", n * 4, 4, h.in));
      DC_TRY(take(a->entropy, "entropy", n * 4, 4, h.in));
    }
    DC_TRY(check_workspace(a->workspace, a->workspace_bytes, fixed_bytes(n, stride, size) + (sum ? n * size * 4 * slices : 0), out));
    DC_TRY(check_head_outputs(out, h));
    Shards written = gw;
    DC_TRY(outside_shards(out, written, "a shard of grad_weights"));
    DC_TRY(outside_shards(h.in, written, "a shard of grad_weights"));
    Shards hidden;
    hidden.add(gh);
    DC_TRY(outside_shards(out, hidden, "grad_hidden"));
    DC_TRY(outside_shards(h.in, hidden, "grad_hidden"));
  }
  if (n == 0 && !want_w) return ok();
  int sms = 0;
  DC_TRY(device(&sms));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool pdl = pdl_option();
  int grid = 0;
  LinearParams p{};
  p.tokens64 = a->tokens_64 != 0;
  p.vocab = static_cast<uint32_t>(vocab);
  p.inv_t = static_cast<float>(1.0 / a->temperature);
  p.rows = n;
  p.tokens = addr(a->tokens);
  p.lse = addr(a->lse);
  p.entropy = addr(a->entropy);
  p.grad_logprobs = addr(a->grad_logprobs);
  p.grad_entropy = addr(a->grad_entropy);
  p.lost = addr(a->workspace) + 256;
  p.marks = p.lost + lost_bytes(n);
  const uint64_t table = p.marks + marks_bytes(n, stride), next = table + table_bytes(n, stride), lost_sums = next + next_bytes(n);
  p.d = lost_sums + sums_bytes(n, stride, size);
  const uint64_t tile = tile_bytes(n) ? p.d + d_bytes(n, stride) : 0;
  p.d_stride = stride;
  const uint64_t acc = sum ? addr(a->workspace) + fixed_bytes(n, stride, size) : 0;
  p.wait_ns = wait_limit_option();
  p.late = tensor_late_option();
  if (n && a->dtype == kF16) {
    p.scale = addr(a->workspace);
    const cudaError_t e = launch_linear_scale(p.grad_logprobs, p.grad_entropy, p.tokens, p.tokens64 != 0, n, p.inv_t, p.scale, pdl, s);
    DC_TRY(check_launch(e, "a linear head's gradient", 1));
  }
  const LinearOperand x{h.hidden.base, n, size, h.hidden.stride};
  const uint32_t m_rows = static_cast<uint32_t>((n + kLinearM - 1) / kLinearM);
  const uint32_t size_tiles = static_cast<uint32_t>((size + kLinearN - 1) / kLinearN);
  uint64_t at = 0, chunk = 0;
  for (int r = 0; r < a->ranks; at += a->widths[r], ++r) {
    const uint64_t held = n && at < vocab ? std::min<uint64_t>(a->widths[r], vocab - at) : 0;  // padding has no gradient
    if (want_w && held < a->widths[r]) {
      const cudaError_t e = cudaMemset2DAsync(reinterpret_cast<void*>(gw[r].base + held * gw[r].stride), gw[r].stride, 0,
                                              gw[r].width, a->widths[r] - held, s);
      if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(DC_ERR_CUDA, "clearing the padding's gradient failed: %s", cudaGetErrorString(e));
      }
    }
    const uint64_t step = linear_chunk(static_cast<uint32_t>(held));
    for (uint64_t c = 0; c < held; c += step, ++chunk) {
      const uint32_t columns = static_cast<uint32_t>(std::min<uint64_t>(step, held - c));
      const LinearOperand w{h.weights[r].base, c + columns, size, h.weights[r].stride};
      const LinearOperand d{p.d, n, columns, stride};
      LinearParams l = p;
      l.m = static_cast<uint32_t>(n);
      l.n = columns;
      l.m_tiles = m_rows;
      l.n_tiles = (columns + kLinearN - 1) / kLinearN;
      l.k_blocks = static_cast<uint32_t>((size + kLinearK - 1) / kLinearK);
      l.b_row0 = static_cast<uint32_t>(c);
      l.first = static_cast<uint32_t>(at + c);
      cudaError_t e = launch_linear(kLinearDLogits, a->dtype, l, x, &w, nullptr, sms, pdl, s, &grid);
      DC_TRY(check_launch(e, "a linear head's gradient", grid));
      if (want_w && n > kLostFew) {
        LinearLostParams t{};
        t.tokens = p.tokens;
        t.lost = p.lost;
        t.marks = p.marks;
        t.table = table;
        t.next = next;
        t.sums = lost_sums;
        t.places = linear_lost_places(n, stride);
        t.x = x.base;
        t.x_stride = x.stride;
        t.rows = n;
        t.d_stride = stride;
        t.first = l.first;
        t.columns = columns;
        t.size = static_cast<uint32_t>(size);
        t.tokens64 = p.tokens64;
        t.by_row = n - kLostAlone < stride / 2;
        e = launch_linear_lost(t, a->dtype, pdl, s, &grid);
        DC_TRY(check_launch(e, "a linear head's gradient", grid));
      }
      LinearParams q = p;
      q.m = static_cast<uint32_t>(n);
      q.n = static_cast<uint32_t>(size);
      q.b_row0 = static_cast<uint32_t>(c);
      q.first = l.first;
      LinearGrads& g = q.g;
      g.x = x.base;
      g.x_stride = x.stride;
      g.table = table;
      g.next = next;
      g.sums = lost_sums;
      g.w = w.base + c * w.stride;
      g.w_stride = w.stride;
      g.columns = columns;
      g.h_blocks = (columns + kLinearK - 1) / kLinearK;
      g.slice_blocks = (g.h_blocks + slices - 1) / slices;
      g.h_m = m_rows;
      g.h_n = size_tiles;
      g.h_tiles = want_h ? m_rows * size_tiles * slices : 0;
      g.w_m = (columns + kLinearM - 1) / kLinearM;
      g.w_blocks = static_cast<uint32_t>((n + kLinearK - 1) / kLinearK);
      g.w_tiles = want_w ? g.w_m * size_tiles : 0;
      g.add = chunk > 0;
      g.last = slices == 1 && chunk + 1 == chunks;
      g.acc = acc;
      g.tile = tile;
      g.out_h = gh.base;
      g.out_h_stride = gh.stride;
      g.out_w = gw[r].base + c * gw[r].stride;
      g.out_w_stride = gw[r].stride;
      const LinearOperand b[2] = {w, x};
      e = launch_linear(kLinearGrads, a->dtype, q, d, b, nullptr, sms, pdl, s, &grid);
      DC_TRY(check_launch(e, "a linear head's gradient", grid));
    }
  }
  if (want_h && n && slices > 1) {
    const LinearSumParams f{acc, gh.base, gh.stride, p.scale, n, static_cast<uint32_t>(size), slices};
    const cudaError_t e = launch_linear_sum(f, a->dtype, pdl, s, &grid);
    return check_launch(e, "a linear head's gradient", grid);
  }
  return ok();
}

dc_status_t dc_qk_norm_rotate(const dc_qk_norm_rotate_t* a, dc_stream_t stream) {
  read_options();
  if (!a) return fail(DC_ERR_INVALID, "the argument block is NULL");
  const NormShape s{a->tokens, a->q_heads, a->kv_heads, a->dim, a->rotary_dim, a->dtype, a->interleaved != 0};
  DC_TRY(check_norm_shape(s, a->eps));
  if (a->tokens == 0) return ok();
  NormParams p{};
  Spans in, heads, out;
  DC_TRY(take_norm_inputs(s, a->positions, a->cos_sin, a->cos_sin_rows, a->q_norm, a->k_norm, a->norm_32 != 0, p, in));
  const Heads x[2] = {{&a->q, "q", a->q_heads}, {&a->k, "k", a->kv_heads}};
  const Heads y[2] = {{&a->q_out, "q_out", a->q_heads}, {&a->k_out, "k_out", a->kv_heads}};
  for (int j = 0; j < 2; ++j) {
    DC_TRY(take_heads(s, x[j], &p.job[j].x, heads));
    DC_TRY(take_heads(s, y[j], &p.job[j].y, out));
  }
  DC_TRY(check_heads_apart(s, y, x, 2, x, 2));
  for (const Span& o : out) DC_TRY(check_apart(o, in));
  int sms = 0, grid = 0;
  DC_TRY(device(&sms));
  p.eps = a->eps;
  plan_norm(&p, a->dtype, s.interleaved, false);
  const cudaError_t e = launch_norm(p, a->dtype, s.interleaved, false, pdl_option(), static_cast<cudaStream_t>(stream), &grid);
  return check_launch(e, "normed queries and keys", grid);
}

size_t dc_qk_norm_workspace_bytes(int64_t tokens, int q_heads, int kv_heads, int dim) {
  const NormShape s{tokens, q_heads, kv_heads, dim, 0, kF32, false};
  if (check_norm_shape(s, 0.0f) != DC_OK) return 0;
  return static_cast<size_t>(norm_workspace(dim));
}

dc_status_t dc_qk_norm_rotate_backward(const dc_qk_norm_rotate_backward_t* a, dc_stream_t stream) {
  read_options();
  if (!a) return fail(DC_ERR_INVALID, "the argument block is NULL");
  const NormShape s{a->tokens, a->q_heads, a->kv_heads, a->dim, a->rotary_dim, a->dtype, a->interleaved != 0};
  DC_TRY(check_norm_shape(s, a->eps));
  const int es = a->norm_32 ? 4 : elem_bytes(a->dtype);
  const uint64_t bytes = static_cast<uint64_t>(a->dim) * static_cast<uint64_t>(es);
  const bool sums = a->grad_q_norm || a->grad_k_norm;
  NormParams p{};
  Spans in, heads, out, sums_out;
  if (a->grad_q_norm) DC_TRY(take(a->grad_q_norm, "grad_q_norm", bytes, es, sums_out));
  if (a->grad_k_norm) DC_TRY(take(a->grad_k_norm, "grad_k_norm", bytes, es, sums_out));
  const cudaStream_t stream_ = static_cast<cudaStream_t>(stream);
  if (a->tokens == 0) {  // a sum over no tokens
    DC_TRY(check_disjoint(sums_out, in));
    if (!sums) return ok();
    int sms = 0;
    DC_TRY(device(&sms));
    for (const Span& o : sums_out) {
      const cudaError_t e = cudaMemsetAsync(reinterpret_cast<void*>(o.lo), 0, o.hi - o.lo, stream_);
      if (e != cudaSuccess) {
        cudaGetLastError();
        return fail(DC_ERR_CUDA, "clearing %s failed: %s", o.name, cudaGetErrorString(e));
      }
    }
    return ok();
  }
  DC_TRY(take_norm_inputs(s, a->positions, a->cos_sin, a->cos_sin_rows, a->q_norm, a->k_norm, a->norm_32 != 0, p, in));
  const Heads x[4] = {{&a->grad_q_out, "grad_q_out", a->q_heads}, {&a->grad_k_out, "grad_k_out", a->kv_heads},
                      {&a->q, "q", a->q_heads}, {&a->k, "k", a->kv_heads}};
  const Heads y[2] = {{&a->grad_q, "grad_q", a->q_heads}, {&a->grad_k, "grad_k", a->kv_heads}};
  for (int j = 0; j < 2; ++j) {
    DC_TRY(take_heads(s, x[j], &p.job[j].dy, heads));
    DC_TRY(take_heads(s, x[j + 2], &p.job[j].x, heads));
    DC_TRY(take_heads(s, y[j], &p.job[j].y, out));
  }
  DC_TRY(check_heads_apart(s, y, x, 2, x, 4));
  for (const Span& o : out) DC_TRY(check_apart(o, in));
  if (sums) {
    if (a->workspace_bytes < norm_workspace(a->dim))
      return fail(DC_ERR_INVALID, "the workspace holds %llu bytes; dc_qk_norm_workspace_bytes says %llu",
                  static_cast<unsigned long long>(a->workspace_bytes), static_cast<unsigned long long>(norm_workspace(a->dim)));
    DC_TRY(take(a->workspace, "workspace", a->workspace_bytes, 16, sums_out));
    p.job[0].partial = a->grad_q_norm ? addr(a->workspace) : 0;
    p.job[1].partial = a->grad_k_norm ? addr(a->workspace) + norm_workspace(a->dim) / 2 : 0;
  }
  DC_TRY(check_disjoint(sums_out, in));
  DC_TRY(check_disjoint(sums_out, heads));
  DC_TRY(check_disjoint(sums_out, out));
  int sms = 0, grid = 0;
  DC_TRY(device(&sms));
  p.eps = a->eps;
  plan_norm(&p, a->dtype, s.interleaved, true);
  cudaError_t e = launch_norm(p, a->dtype, s.interleaved, true, pdl_option(), stream_, &grid);
  DC_TRY(check_launch(e, "normed queries' and keys' gradient", grid));
  if (!sums) return ok();
  NormFinishParams f{};
  f.dim = a->dim;
  f.out32 = a->norm_32 != 0;
  for (int j = 0; j < 2; ++j) {
    f.partial[j] = p.job[j].partial;
    f.ctas[j] = p.job[j].ctas;
    f.out[j] = addr(j ? a->grad_k_norm : a->grad_q_norm);
  }
  e = launch_norm_finish(f, a->dtype, pdl_option(), stream_, &grid);
  return check_launch(e, "normed queries' and keys' gradient", grid);
}

}  // extern "C"
