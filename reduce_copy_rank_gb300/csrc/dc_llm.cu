// dc_llm.cu -- the C ABI of the language-model operators: argument checks,
// the choice of grid, launch.
#include "dc_checks.h"

namespace {

using namespace dc;

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

// Checks an append's arguments (of at least one token) and fills its parameters;
// `written`: the spans that it writes.
dc_status_t take_append(const dc_kv_append_t* a, AppendParams& p, Spans& written) {
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
  if (a->tokens == 0) return DC_OK;
  const uint64_t n = static_cast<uint64_t>(a->tokens);
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
  for (const Span& c : cache) written.add(c);
  for (const Span& o : out) written.add(o);
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
  return DC_OK;
}

// Checks the arguments of an attention (of at least one sequence); `in` and
// `out` get what it reads and writes.
dc_status_t take_attend(const dc_paged_attention_t* a, AttendParams& p, AttendPlan& plan, Spans& in, Spans& out) {
  if (a->dtype != kBF16 && a->dtype != kF16) return fail(DC_ERR_INVALID, "dtype %d is not DC_BF16 or DC_F16", a->dtype);
  if (a->page_size < 1) return fail(DC_ERR_INVALID, "page_size = %d is not positive", a->page_size);
  if (a->window < 0) return fail(DC_ERR_INVALID, "window = %d is negative", a->window);
  if (!std::isfinite(a->scale)) return fail(DC_ERR_INVALID, "scale is not finite");
  if (a->seqs == 0) return DC_OK;
  DC_TRY(check_table(a->page_table, a->seqs, a->table_width, a->table_stride, in));
  uint64_t most = static_cast<uint64_t>(a->table_width) * static_cast<uint64_t>(a->page_size);
  if (a->window > 0) most = std::min<uint64_t>(most, static_cast<uint64_t>(a->window));
  DC_TRY(plan_attend(a->seqs, a->q_heads, a->kv_heads, a->dim, most, &plan));
  const uint64_t n = static_cast<uint64_t>(a->seqs);
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
  p.page_shift = (p.page_size & (p.page_size - 1)) == 0 ? __builtin_ctz(p.page_size) : -1;
  p.scale = a->scale;
  return DC_OK;
}

// The last choices, which need the GPU's size, and the launch.
dc_status_t run_attend(AttendParams& p, const AttendPlan& plan, int dtype, int dim, int sms, dc_stream_t stream) {
  // Few CTAs, all resident at once, and few enough pieces: a unit's CTAs are a
  // cluster and join them in shared memory.  Measured, us, workspace / cluster:
  // one sequence of 1025 tokens, 8/1 heads of 128 (5 pieces): 8.2 / 6.9; of 4096
  // (16 pieces, two clusters and the workspace): 8.1 / 10.
  const uint32_t resident = static_cast<uint32_t>(sms) * (dim <= 128 ? 2u : 1u);
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
  if (!cluster && plan.pieces > 1 && plan.units * attend_counters(plan.pieces) > kAttendCounters) p.places = 1;
  int grid = 0;
  const cudaError_t e = (p.raw ? launch_attend_parts : launch_attend)(p, dtype, dim, pdl_option(), static_cast<cudaStream_t>(stream), &grid);
  return check_launch(e, "paged attention", grid);
}

// Neighbouring tokens that a TMA copy can move: as many as divide a page and a
// tile, 8 at least (the swizzled rows of 128 bytes come in eights), and the
// caches' strides have to fit a tensor map.  0: none.
int prefix_slots(const AttendParams& p, const dc_paged_attention_t& a) {
  int slots = 1;
  while (slots < kPrefixTile && p.page_size % (2u * static_cast<uint32_t>(slots)) == 0) slots *= 2;
  const PagedView* const views[2] = {&p.kc, &p.vc};
  for (const PagedView* v : views)
    for (const uint64_t stride : {a.kv_heads > 1 ? v->head : 16, a.page_size > 1 ? v->token : 16, a.num_pages > 1 ? v->page : 16})
      if (stride == 0 || stride % 16 || stride >= 1ull << 40) return 0;
  return slots >= 8 ? slots : 0;
}

// Where the parts of an attention to shared prefixes lie in its workspace,
// behind the one of paged attention.
struct PrefixSizes {
  uint64_t raw, raw_rl, partial, partial_rl, end;
  uint32_t chunks;
};

dc_status_t plan_prefix(int64_t seqs, int64_t prefixes, int q_heads, int kv_heads, int dim, uint64_t max_tokens,
                        const AttendPlan& own, PrefixSizes* z) {
  if (prefixes < 1 || prefixes > 0x7FFFFFFF || seqs % prefixes)
    return fail(DC_ERR_INVALID, "%lld sequences are not shared out among %lld prefixes", static_cast<long long>(seqs),
                static_cast<long long>(prefixes));
  if (max_tokens > 0x7FFFFFFFull)
    return fail(DC_ERR_INVALID, "prefixes of up to %llu tokens", static_cast<unsigned long long>(max_tokens));
  const uint64_t tiles = (max_tokens + kPrefixTile - 1) / kPrefixTile;
  const uint64_t most = std::max<uint64_t>(prefix_most_chunks(kv_heads), (max_tokens + kPrefixChunk - 1) / kPrefixChunk);
  z->chunks = static_cast<uint32_t>(std::max<uint64_t>(1, std::min<uint64_t>(tiles, most)));
  const uint64_t rows = static_cast<uint64_t>(seqs / prefixes) * static_cast<uint64_t>(q_heads / kv_heads);
  const uint64_t units = static_cast<uint64_t>(prefixes) * static_cast<uint64_t>(kv_heads) * z->chunks;
  if (rows > 0x7FFFFFFFull - kPrefixRows || units > 0x7FFFFFFFull || units * ((rows + kPrefixRows - 1) / kPrefixRows) > 0x7FFFFFFFull ||
      static_cast<uint64_t>(seqs) * q_heads > 0x7FFFFFF0ull)
    return fail(DC_ERR_INVALID, "%lld sequences of %d heads exceed a grid", static_cast<long long>(seqs), q_heads);
  const uint64_t all = static_cast<uint64_t>(seqs) * static_cast<uint64_t>(q_heads), d = static_cast<uint64_t>(dim);
  const auto up = [](uint64_t n) { return (n + 255) / 256 * 256; };
  z->raw = up(kAttendCounterBytes + own.partial_bytes);
  z->raw_rl = z->raw + up(all * d * 4);
  z->partial = z->raw_rl + up(all * 8);
  z->partial_rl = z->partial + up(units * rows * d * 4);
  z->end = z->partial_rl + up(units * rows * 8);
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
  AppendParams p{};
  Spans written;
  DC_TRY(take_append(a, p, written));
  if (a->tokens == 0) return ok();
  int sms = 0;
  DC_TRY(device(&sms));
  int grid = 0;
  const cudaError_t e = launch_append(p, a->dtype, sms, pdl_option(), static_cast<cudaStream_t>(stream), &grid);
  return check_launch(e, "cache append", grid);
}

dc_status_t dc_kv_append_norm(const dc_kv_append_norm_t* a, dc_stream_t stream) {
  read_options();
  if (!a) return fail(DC_ERR_INVALID, "the argument block is NULL");
  AppendParams x{};
  Spans written, in;
  DC_TRY(check_norm(a->append.dim, a->eps));
  DC_TRY(take_append(&a->append, x, written));
  const int es = a->norm_32 ? 4 : elem_bytes(a->append.dtype);
  const uint64_t bytes = static_cast<uint64_t>(a->append.dim) * static_cast<uint64_t>(es);
  if (a->append.q_heads) DC_TRY(take(a->q_norm, "q_norm", bytes, es, in));
  DC_TRY(take(a->k_norm, "k_norm", bytes, es, in));
  if (a->append.tokens == 0) return ok();
  for (const Span& w : written) DC_TRY(check_apart(w, in));
  int sms = 0;
  DC_TRY(device(&sms));
  NormParams p{};
  p.job[0] = NormJob{{x.q, x.q_token, x.q_head}, {x.qo, x.qo_token, x.qo_head}, {}, addr(a->q_norm), 0, x.q_heads, 1, 0, 0};
  p.job[1] = NormJob{{x.k, x.k_token, x.k_head}, {x.kc.base, 0, x.kc.head}, {}, addr(a->k_norm), 0, x.kv_heads, 1, 0, 0};
  p.job[2] = NormJob{{x.v, x.v_token, x.v_head}, {x.vc.base, 0, x.vc.head}, {}, 0, 0, x.kv_heads, 1, 0, 0};
  p.jobs = 3;
  p.cached = 1;
  p.positions = x.positions;
  p.cos_sin = x.cos_sin;
  p.tokens = x.tokens;
  p.cos_rows = x.cos_rows;
  p.seqs = x.seqs;
  p.table = x.table;
  p.table_stride = x.table_stride;
  p.num_pages = x.num_pages;
  p.page_size = x.page_size;
  p.table_width = x.table_width;
  p.num_seqs = x.num_seqs;
  p.kc = x.kc;
  p.vc = x.vc;
  p.dim = x.dim;
  p.rot = x.rot;
  p.w32 = a->norm_32 != 0;
  p.eps = a->eps;
  plan_norm(&p, a->append.dtype, x.interleaved != 0, false);
  int grid = 0;
  const cudaError_t e = launch_norm(p, a->append.dtype, x.interleaved != 0, false, pdl_option(), static_cast<cudaStream_t>(stream), &grid);
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
  AttendParams p{};
  AttendPlan plan{};
  Spans in, out;
  DC_TRY(take_attend(a, p, plan, in, out));
  if (a->seqs == 0) return ok();
  int sms = 0;
  DC_TRY(device(&sms));
  return run_attend(p, plan, a->dtype, a->dim, sms, stream);
}

size_t dc_prefix_attention_workspace_bytes(int64_t seqs, int64_t prefixes, int q_heads, int kv_heads, int dim,
                                           int64_t max_prefix_tokens, int64_t max_tokens) {
  AttendPlan plan{};
  PrefixSizes sizes{};
  if (max_tokens < 0 || max_prefix_tokens < 0 ||
      plan_attend(seqs, q_heads, kv_heads, dim, static_cast<uint64_t>(max_tokens), &plan) != DC_OK ||
      plan_prefix(seqs, prefixes, q_heads, kv_heads, dim, static_cast<uint64_t>(max_prefix_tokens), plan, &sizes) != DC_OK)
    return 0;
  return static_cast<size_t>(sizes.end);
}

dc_status_t dc_prefix_attention(const dc_prefix_attention_t* a, dc_stream_t stream) {
  read_options();
  if (!a) return fail(DC_ERR_INVALID, "the argument block is NULL");
  const dc_paged_attention_t& own = a->own;
  if (own.window != 0) return fail(DC_ERR_INVALID, "attention to shared prefixes has no window (got %d)", own.window);
  AttendParams p{};
  AttendPlan plan{};
  Spans in, out;
  DC_TRY(take_attend(&own, p, plan, in, out));
  if (own.seqs == 0) return ok();
  PrefixSizes sizes{};
  const uint64_t most = static_cast<uint64_t>(a->prefix_table_width < 0 ? 0 : a->prefix_table_width) * static_cast<uint64_t>(own.page_size);
  DC_TRY(plan_prefix(own.seqs, a->prefixes, own.q_heads, own.kv_heads, own.dim, most, plan, &sizes));
  Spans more;
  DC_TRY(check_table(a->prefix_table, a->prefixes, a->prefix_table_width, a->prefix_table_stride, more));
  DC_TRY(take(a->prefix_lengths, "prefix_lengths", static_cast<uint64_t>(a->prefixes) * 4, 4, more));
  if (own.workspace_bytes < sizes.end)
    return fail(DC_ERR_INVALID, "the workspace holds %llu bytes; dc_prefix_attention_workspace_bytes says %llu",
                static_cast<unsigned long long>(own.workspace_bytes), static_cast<unsigned long long>(sizes.end));
  if (!plan.partial_bytes) {  // (else it is among what is written already)
    Spans ws;
    DC_TRY(take(own.workspace, "workspace", own.workspace_bytes, 16, ws));
    DC_TRY(check_disjoint(ws, in));
    DC_TRY(check_disjoint(ws, out));
    DC_TRY(check_disjoint(ws, more));
  }
  for (const Span& o : out) DC_TRY(check_apart(o, more));
  int sms = 0, grid = 0;
  DC_TRY(device(&sms));
  const uint64_t ws = addr(own.workspace);
  PrefixParams x{};
  x.q = p.q;
  x.q_seq = p.q_seq;
  x.q_head = p.q_head;
  x.out = p.out;
  x.out_seq = p.out_seq;
  x.out_head = p.out_head;
  x.lse = p.lse;
  x.table = addr(a->prefix_table);
  x.lengths = addr(a->prefix_lengths);
  x.raw = ws + sizes.raw;
  x.raw_rl = ws + sizes.raw_rl;
  x.partial = ws + sizes.partial;
  x.partial_rl = ws + sizes.partial_rl;
  x.table_stride = a->prefixes > 1 ? a->prefix_table_stride : 0;
  x.num_pages = p.num_pages;
  x.page_size = p.page_size;
  x.table_width = static_cast<uint32_t>(a->prefix_table_width);
  x.page_shift = p.page_shift;
  x.seqs = p.seqs;
  x.prefixes = static_cast<int32_t>(a->prefixes);
  x.each = static_cast<int32_t>(own.seqs / a->prefixes);
  x.q_heads = p.q_heads;
  x.kv_heads = p.kv_heads;
  x.group = p.group;
  x.rows = x.each * x.group;
  x.row_tiles = (x.rows + kPrefixRows - 1) / kPrefixRows;
  x.chunks = static_cast<int32_t>(sizes.chunks);
  x.slots = prefix_slots(p, own);
  x.scale = own.scale;
  x.wait_ns = wait_limit_option();
  x.late = tensor_late_option();
  x.kc = p.kc;
  x.vc = p.vc;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  p.raw = x.raw;
  p.raw_rl = x.raw_rl;
  x.ready = p.ready = ws + kAttendCounters * 4;
  // (the prefix's kernel may start before the own tokens' has ended: that one waits for
  // what came before the call, and only then lets this one start)
  DC_TRY(run_attend(p, plan, own.dtype, own.dim, sms, stream));
  cudaError_t e = launch_prefix(x, own.dtype, own.dim, pdl_option(), s, &grid);
  DC_TRY(check_launch(e, "attention to shared prefixes", grid));
  e = launch_prefix_join(x, own.dtype, own.dim, pdl_option(), s, &grid);
  return check_launch(e, "attention to shared prefixes", grid);
}

}  // extern "C"
