// dc_llm.h -- parameter blocks of the language-model operators, shared by
// their host checks (dc_llm.cu) and their kernels (dc_logprobs.cu,
// dc_kv_append.cu, dc_attention.cu).  As for the collectives, everything a
// kernel needs travels by value.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "dc_internal.h"

namespace dc {

// --------------------------------------------------------- log probabilities
// The vocabulary is cut into segments of 4 KB of logits, counted over the
// concatenated shards; one warp reduces one segment, and a row's segments are
// folded in one fixed order.  The tree of additions therefore depends on the
// vocabulary and its type alone: not on the rows of the call, the shards or
// the grid.
__host__ __device__ constexpr int vocab_seg(int dtype) { return dtype == kF32 ? 1024 : 2048; }
constexpr int kScoreWarps = 8;      // most warps per CTA
constexpr int kScoreMaxCluster = 8; // CTAs that may share a row
constexpr int kMaxVocab = 1 << 22;  // at most 4096 segments: 64 KB of partials
constexpr int kMaxTop = 32;         // alternatives: one lane each

// One rank's columns [first, end) of the vocabulary; row i starts at base + i * stride bytes.
struct LogitShard {
  uint64_t base;
  uint64_t stride;
  uint32_t first;
  uint32_t end;
};

struct ScoreParams {
  uint64_t tokens;         // int32 or int64 [rows]
  uint64_t logprobs;       // f32 [rows]
  uint64_t entropy;        // f32 [rows] or 0
  uint64_t lse;            // f32 [rows] or 0
  uint64_t top_logprobs;   // f32 [rows, top] or 0
  uint64_t top_tokens;     // int32 or int64 [rows, top] or 0
  uint64_t rows;
  float inv_t;
  uint32_t vocab;
  int32_t P;
  int32_t nseg;
  int32_t cluster;         // CTAs per row
  int32_t warps;           // per CTA: a power of two; all of them in a cluster
  int32_t top;
  int32_t tokens64;
  int32_t top64;
  LogitShard shard[kMaxRanks];
};
cudaError_t launch_score(const ScoreParams& p, int dtype, bool pdl, cudaStream_t s, int* grid);

// The gradient: each rank's row is written as 16-byte vectors anchored at the
// output, kGradChunk vectors a CTA; elements before and after them one by one.
constexpr int kGradThreads = 256;
constexpr int kGradVecs = 4;
constexpr int kGradChunk = kGradThreads * kGradVecs;
struct GradShard {
  uint64_t in, in_stride;    // bytes
  uint64_t out, out_stride;
  uint32_t first;            // vocabulary index of column 0
  uint32_t width;            // columns, those past the vocabulary included
  uint32_t chunk0;           // this shard's first chunk of a row
  uint32_t pad;
};
struct GradParams {
  uint64_t tokens, lse, entropy, grad_logprobs, grad_entropy;  // the last two f32 [rows] or 0
  uint64_t rows;
  float inv_t;
  uint32_t vocab;
  int32_t P;
  int32_t tokens64;
  uint32_t chunks;           // of one row
  uint32_t pad;
  GradShard shard[kMaxRanks];
};
cudaError_t launch_score_grad(const GradParams& p, int dtype, bool pdl, cudaStream_t s, int* grid);

// ------------------------------------------------------------- paged cache
// A paged cache: element d of head h of token slot o of page g is at
// base + g*page + o*token + h*head + d*element size (strides in bytes).
struct PagedView {
  uint64_t base;
  uint64_t page, token, head;
  uint64_t lo, hi;  // the bytes it spans
};

struct AppendParams {
  uint64_t q, q_token, q_head;          // bytes; 0 if no queries
  uint64_t qo, qo_token, qo_head;
  uint64_t k, k_token, k_head;
  uint64_t v, v_token, v_head;
  uint64_t positions, seqs, table;      // int32
  uint64_t cos_sin;                     // f32 [cos_rows, rot] or 0
  uint64_t tokens;
  int64_t table_stride;                 // entries
  int64_t cos_rows;
  int64_t num_pages;
  uint32_t page_size, table_width, num_seqs;
  int32_t q_heads, kv_heads, dim, rot, interleaved;
  PagedView kc, vc;
};
cudaError_t launch_append(const AppendParams& p, int dtype, int sms, bool pdl, cudaStream_t s, int* grid);

// --------------------------------------------------------------- attention
constexpr int kAttendWarps = 4;
constexpr int kAttendTile = 16;       // tokens a warp takes at a time
constexpr int kAttendJoin = 16;       // pieces that one CTA joins at a time
constexpr int kAttendCluster = 8;     // most CTAs of a cluster, which join their pieces in shared memory
constexpr int kAttendGroups = 8;      // groups of them, at most (128 pieces)
// Arrival counters, at the start of a workspace: an area of one size, whatever
// the workspace's, so that calls on parts of it of different lengths agree on
// what has to be zero.  A unit has one, or, if it may have several groups, one
// for them and one for each group's pieces; units beyond the area's room are
// computed by a CTA each.  Its last word is attention to shared prefixes' (PrefixParams).
constexpr uint64_t kAttendCounterBytes = 1 << 20;
constexpr uint64_t kAttendCounters = kAttendCounterBytes / 4 - 1;
__host__ __device__ constexpr uint32_t attend_counters(uint32_t pieces) {
  return pieces <= static_cast<uint32_t>(kAttendJoin) ? 1u : 1u + (pieces + kAttendJoin - 1) / kAttendJoin;
}

struct AttendParams {
  uint64_t q, q_seq, q_head;            // bytes
  uint64_t out, out_seq, out_head;
  uint64_t lse;                         // f32 [seqs, q_heads] or 0
  uint64_t table, lengths;              // int32
  uint64_t counters;                    // uint32 [units][attend_counters(pieces)], zero between calls
  uint64_t partial;                     // f32 [units][HB * (pieces * (dim + 2) + 2 * kAttendGroups)]
  uint64_t raw, raw_rl;                 // 0, or where the results go instead of out: f32 [seqs][q_heads][dim]
                                        // unnormalised, and [seqs][q_heads] (reference, sum)
  uint64_t ready;                       // (with raw) uint32, as PrefixParams has it
  int64_t table_stride;
  int64_t num_pages;
  uint32_t page_size, table_width;
  int32_t seqs, q_heads, kv_heads, group, head_blocks;
  int32_t hb;                           // heads of a block: attend_head_block
  int32_t window;
  int32_t units;                        // seqs * kv_heads * head_blocks
  int32_t pieces;                       // most pieces of one sequence
  int32_t places;                       // CTAs of a unit: pieces, the cluster they fit in, fewer that take turns, or one
  int32_t cluster;                      // places, or 1: pieces are joined through the workspace
  int32_t page_shift;                   // log2 of the page size, -1 if it is no power of two
  float scale;
  PagedView kc, vc;
};

// The tree over a sequence of n attended tokens has leaves of attend_leaf(n)
// tokens, at most 512 of them; a warp takes 2^level neighbouring leaves and a
// CTA four neighbouring warps' (a piece).  The leaves are a function of n
// alone, the level of how much work there is.
// Leaves of 32 tokens up to 1024, which a cluster's 32 warps share, of 64 up to
// 8192 and 128 above: a leaf costs a climb up the tree, and long sequences have
// leaves enough.  Measured, us.  64 / 32 up to 1024: one sequence of 1024
// tokens, 32/8 heads of 128: 7.2 / 5.9; 64 ragged ones up to 1024: 33.5 / 35.9.
// 64 throughout / 128 above 8192 / 128 above 4096: one of 16384: 22.7 / 19.3 /
// 19.3; 128 ragged ones up to 8192: 347 / 347 / 339; 32 up to 8000, 64/8 heads
// of 64: 54 / 54 / 63.
constexpr uint32_t kAttendTiny = 1024, kAttendShort = 8192;
__host__ __device__ inline uint32_t attend_leaf(uint32_t n) {
  uint32_t leaf = n <= kAttendTiny ? 32 : n <= kAttendShort ? 64 : 128;
  while (n / leaf > 512 || (n / leaf == 512 && n % leaf)) leaf *= 2;
  return leaf;
}
__host__ __device__ inline uint32_t attend_pieces(uint32_t n, uint32_t level) {
  const uint32_t leaf = attend_leaf(n), leaves = n / leaf + (n % leaf != 0), per = 4u << level;
  return (leaves + per - 1) / per;
}
constexpr uint32_t kAttendMaxPieces = 128;  // 512 leaves, one a warp
// Levels that a warp can hold: waiting subtrees live in registers (heads above
// 128 are shared by two or three warps).
__host__ __device__ constexpr int attend_levels(int dim, int hb) { return hb == 8 || dim <= 64 ? 2 : 1; }
// The level for a sequence of `small` pieces at level 0, if all `units` of the
// call were like it: the smallest that leaves at most kAttendCtas CTAs.
constexpr uint32_t kAttendCtas = 608;
__host__ __device__ inline uint32_t attend_level(uint32_t small, uint32_t units, int levels) {
  uint32_t k = 0;
  while (k < static_cast<uint32_t>(levels) && units * ((small + (1u << k) - 1) >> k) > kAttendCtas) ++k;
  return k;
}
// Heads that one CTA serves.  Where a key head has more than 8 query heads: 16,
// which read keys and values once, or 8 while the GPU would hold all of those
// CTAs at once (two read the same keys, the second from L2; same bits).
// Measured, us, 16 / 8: one sequence of 1024, 16/1 heads of 128: 7.5 / 6.2 (16
// CTAs of 8); of 131072: 32.9 / 28.9 (256 CTAs); of 16384, 128/8 heads: 29.3 /
// 31.0 (512); 32 up to 8000, 64/4 heads: 64 / 69.
// (The GPU's SMs by a constant: a workspace's size follows from them, and is asked
// for without a device.)
constexpr uint32_t kAttendSms = 152;
__host__ __device__ constexpr int attend_ctas_per_sm(int dim, int hb) {
  return dim <= 64 && hb == 8 ? 3 : dim <= 128 ? 2 : 1;
}
__host__ __device__ inline int attend_head_block(int group, uint64_t kv_units, uint32_t pieces, int dim) {
  const uint64_t ctas = kv_units * static_cast<uint64_t>((group + 7) / 8) * pieces;
  return group > 8 && ctas > kAttendSms * static_cast<uint64_t>(attend_ctas_per_sm(dim, 8)) ? 16 : 8;
}
cudaError_t launch_attend(const AttendParams& p, int dtype, int dim, bool pdl, cudaStream_t s, int* grid);
cudaError_t launch_attend_parts(const AttendParams& p, int dtype, int dim, bool pdl, cudaStream_t s, int* grid);  // to raw, raw_rl

// ------------------------------------------- log probabilities of a linear head
// Matrix products on the tensor cores: tiles of kLinearM x kLinearN, which a pair
// of CTAs share, kLinearK of the inner dimension a stage.
constexpr int kLinearM = 256, kLinearN = 256, kLinearK = 64;
constexpr uint32_t kLinearPairs = kAttendSms / 2;  // at most, at work
constexpr int kLinearPart = 128;  // columns that one thread reduces of a row of the logits
// The gradient takes up to this many columns of a shard at a time, and cuts the
// products over them into slices, both whatever the call's rows: how a sum is cut
// decides its bits.
constexpr uint32_t kLinearChunk = 24576;
__host__ __device__ inline uint32_t linear_chunk(uint32_t width) {
  const uint32_t n = (width + kLinearChunk - 1) / kLinearChunk, per = n ? (width + n - 1) / n : 0;
  return (per + kLinearN - 1) / kLinearN * kLinearN;
}
__host__ __device__ inline uint32_t linear_groups(uint64_t rows) { return static_cast<uint32_t>((rows + 31) / 32); }
// Bytes of the marks for a chunk whose rows of d take d_stride bytes.
__host__ __device__ inline uint64_t linear_marks(uint64_t rows, uint64_t d_stride) {
  return d_stride / (2 * kLinearN) * linear_groups(rows) * 4;
}
// A row of dh has ceil(size / kLinearN) tiles: with few the sum over a chunk's
// columns is cut into slices, so that short batches have work for the GPU too.
__host__ __device__ inline uint32_t linear_slices(uint32_t size) {
  const uint32_t tiles = (size + kLinearN - 1) / kLinearN;
  return tiles >= 16 ? 1 : 16 / tiles;
}

enum : int { kLinearStats = 0, kLinearDLogits = 1, kLinearGrads = 2 };

// Columns [first, end) of the vocabulary, in tiles from tile0 on (end: without padding).
struct LinearShard {
  uint32_t tile0, first, end, pad;
};

// Both products of a chunk's gradient in one launch: tiles of dh = d W (in
// slices of the chunk's columns), then tiles of dW = d^T h.  CTA pair c of G takes dh
// tiles c, c + G, ..., then the first `few` rounds of dW tiles like all others;
// those that had one dh tile less (c >= rest) go on to `many` rounds.
struct LinearGrads {
  uint32_t h_tiles, h_m, h_n;  // h_m * h_n * slices
  uint32_t slice_blocks, h_blocks;
  uint32_t w_tiles, w_m, w_blocks;
  uint32_t rounds, rest, few, many;
  uint32_t columns;            // of the chunk
  int32_t add, last;           // what `acc` holds is added; the sum is complete (no acc: one slice)
  uint64_t acc;                // f32 [slices][rows][size] or 0
  uint64_t tile;               // f32 [kLinearPairs][kLinearM][kLinearN] or 0: sums of dW's runs
  uint64_t out_h, out_h_stride, out_w, out_w_stride;  // bytes
  uint64_t x, x_stride, w, w_stride;                  // the hidden rows, the chunk's rows of the weights
  uint64_t table, next, sums;  // what dW's rows get back: as LinearLostParams has them (not of kLostFew rows)
};

// One product C [m, n] = A B^T over k, and what becomes of it.
struct LinearParams {
  uint32_t m, n;               // extents of C (kLinearStats: n is not used; kLinearGrads: rows and hidden size)
  uint32_t m_tiles, n_tiles, k_blocks;
  uint32_t run;                // kLinearStats: blocks of a sum on the tensor cores
  uint32_t b_row0;             // first row of the weights (kLinearDLogits, kLinearGrads)
  uint32_t vocab, first;       // the vocabulary index of column 0 (kLinearDLogits, kLinearGrads)
  float inv_t;
  int32_t tokens64;
  int32_t shards;              // kLinearStats
  uint64_t rows;
  uint64_t tokens;
  uint64_t part, target;       // kLinearStats: f32 [2 tiles][rows][4], f32 [rows]
  uint64_t lse, entropy, grad_logprobs, grad_entropy;  // f32 [rows]; the last two or 0
  uint64_t scale;              // f32 [2] or 0: the gradient's power of two and its inverse
  uint64_t d, d_stride;        // kLinearDLogits: [rows] of d_stride bytes
  uint64_t lost;               // f32 [rows]: what d lost of each row's token
  uint64_t marks;              // [tiles of kLinearN columns][groups of 32 rows]: a bit a row that has a gradient and its token there
  uint64_t wait_ns;
  int32_t late;                // test: 1 or 2: the even or odd CTAs' first results are late, 3 or 4: their third copies
  LinearGrads g;               // kLinearGrads
};

// What dW's rows get back of what d lost, for calls of more than kLostFew rows.  A
// column that up to kLostAlone rows have as their token: its first row's number, and
// each row's next one (-1: none).  A column of more: -2 - its place in the sums.
constexpr uint32_t kLostFew = 64, kLostAlone = 16;
struct LinearLostParams {
  uint64_t tokens, lost, marks;
  uint64_t table, next;        // int32 [d_stride / 2], [rows]
  uint64_t sums, places;       // f32 [places][size]
  uint64_t x, x_stride;        // the hidden rows
  uint64_t rows, d_stride;
  uint32_t first, columns, size;
  int32_t tokens64, by_row;    // by_row: a column's place is its first row's, else its own
};
// Places for sums: a chunk's columns, or the rows that can be the first of a column's
// more than kLostAlone.
__host__ __device__ inline uint64_t linear_lost_places(uint64_t rows, uint64_t d_stride) {
  if (rows <= kLostFew) return 0;
  return rows - kLostAlone < d_stride / 2 ? rows - kLostAlone : d_stride / 2;
}

struct LinearFinishParams {
  uint64_t part, target, tokens, logprobs, entropy, lse;  // the last three f32 [rows], two of them or 0
  uint64_t rows;
  uint32_t parts, vocab;
  int32_t tokens64;
  float inv_t;
};

// dh from its slices' sums, which are added in order.
struct LinearSumParams {
  uint64_t acc, out, out_stride, scale;
  uint64_t rows;
  uint32_t size, slices;
};

// The operands as tensors of 16-bit rows.
struct LinearOperand {
  uint64_t base, rows, columns, stride;  // stride in bytes
};
cudaError_t launch_linear(int mode, int dtype, const LinearParams& p, const LinearOperand& a, const LinearOperand* b,
                          const LinearShard* shards, int sms, bool pdl, cudaStream_t s, int* grid);
cudaError_t launch_linear_finish(const LinearFinishParams& p, bool pdl, cudaStream_t s, int* grid);
cudaError_t launch_linear_lost(const LinearLostParams& p, int dtype, bool pdl, cudaStream_t s, int* grid);
cudaError_t launch_linear_sum(const LinearSumParams& p, int dtype, bool pdl, cudaStream_t s, int* grid);
// Fills the schedule of p.g for `pairs` CTA pairs.
void plan_linear_grads(LinearGrads* g, uint32_t pairs);
cudaError_t launch_linear_scale(uint64_t grad_logprobs, uint64_t grad_entropy, uint64_t tokens, bool tokens64, uint64_t rows,
                                float inv_t, uint64_t scale, bool pdl, cudaStream_t s);

// ---------------------------------------------- normed queries and keys
// A token's heads of one kind: element d of head h of token t is at
// base + t*token + h*head + d*element size.
struct HeadsView {
  uint64_t base, token, head;
};

// CTAs of a launch, by a constant: the weights' gradient is added up over them.
constexpr int kNormThreads = 128;
constexpr int kNormCtas = 152 * 6;
constexpr int kNormGradCtas = 152 * 4;
constexpr int kNormMaxDim = 512;  // at most 128 work units a head

// One kind of heads: queries, keys, or values (which are copied).
struct NormJob {
  HeadsView x, y;              // in and out; y of keys and values is the cache where there is one
  HeadsView dy;                // (gradient) of the output; y is that of the input
  uint64_t w;                  // [dim], 0 for values
  uint64_t partial;            // (gradient) f32 [CTAs][dim] or 0
  int32_t heads, split;        // warps that share a token
  uint32_t cta0, ctas;
};

struct NormParams {
  NormJob job[3];
  uint64_t positions, cos_sin; // int32 [tokens], f32 [cos_rows][rot] or 0
  uint64_t tokens;
  int64_t cos_rows;
  // a cache, where keys and values go to one
  uint64_t seqs, table;
  int64_t table_stride, num_pages;
  uint32_t page_size, table_width, num_seqs;
  PagedView kc, vc;
  int32_t jobs, cached;
  int32_t dim, rot, w32;       // w32: the weights are binary32, else of the heads' type
  int32_t units, lanes;        // of a head: work units, and lanes that share it
  int32_t angles_aligned;      // cos_sin: to 16 bytes
  float eps, inv_dim;          // 1 / dim
};
// Fills inv_dim, units, lanes, angles_aligned, split, cta0 and ctas.
void plan_norm(NormParams* p, int dtype, bool interleaved, bool gradient);
cudaError_t launch_norm(const NormParams& p, int dtype, bool interleaved, bool gradient, bool pdl, cudaStream_t s, int* grid);

// The weights' gradients from the CTAs' parts.
struct NormFinishParams {
  uint64_t partial[2], out[2];  // out 0: not wanted
  uint32_t ctas[2];
  int32_t dim, out32;
};
cudaError_t launch_norm_finish(const NormFinishParams& p, int dtype, bool pdl, cudaStream_t s, int* grid);

// -------------------------------------------------- attention to shared prefixes
// A prefix's tokens are cut into chunks, a CTA each for every key head and 128
// query rows (a row: one head of one sequence): as many as fill the GPU once, no
// shorter than a tile and no longer than the tensor cores' sums stay good for (FP16, flat
// scores, values of one sign, 32 key heads, 2^20 tokens, mean error: chunks of 262144
// tokens 1.4e-3, of 24576 1.9e-4, the last rounding's).  The cut follows
// from the prefix's length and the number of key heads, so that how many sequences share
// it changes no bit.
constexpr int kPrefixRows = 128, kPrefixTile = 64;
constexpr uint32_t kPrefixChunk = 24576;
__host__ __device__ inline uint32_t prefix_most_chunks(int kv_heads) {
  const uint32_t n = kAttendSms / static_cast<uint32_t>(kv_heads);
  return n > 1 ? n : 1;
}
__host__ __device__ inline uint32_t prefix_chunk(uint32_t tokens, int kv_heads) {
  const uint32_t most = prefix_most_chunks(kv_heads), per = tokens / most + (tokens % most != 0);
  return per < kPrefixChunk ? (per + kPrefixTile - 1) / kPrefixTile * kPrefixTile : kPrefixChunk;
}
__host__ __device__ inline uint32_t prefix_chunks(uint32_t tokens, int kv_heads) {
  if (tokens == 0) return 0;
  const uint32_t per = prefix_chunk(tokens, kv_heads);
  return tokens / per + (tokens % per != 0);
}

struct PrefixParams {
  uint64_t q, q_seq, q_head;            // bytes
  uint64_t out, out_seq, out_head, lse; // lse: f32 [seqs, q_heads] or 0
  uint64_t table, lengths;              // int32 [prefixes][table_width], [prefixes]
  uint64_t partial, partial_rl;         // f32 [prefixes][kv_heads][chunks][rows][dim], [..][rows] (reference, sum)
  uint64_t raw, raw_rl;                 // the sequences' own tokens, as AttendParams has them
  uint64_t ready;                       // uint32, 0 between calls; 1: what came before the call is done
  int64_t table_stride, num_pages;
  uint32_t page_size, table_width;
  int32_t page_shift;
  int32_t seqs, prefixes, each, q_heads, kv_heads, group;
  int32_t rows, row_tiles;              // of a prefix and key head: each * group
  int32_t chunks;                       // most of one prefix
  int32_t slots;                        // neighbouring tokens that one TMA copy moves; 0: keys and values by cp.async
  float scale;
  int32_t late;                         // test: 1: the first weights are late, 2: the second tile's values
  uint64_t wait_ns;
  PagedView kc, vc;
};
cudaError_t launch_prefix(const PrefixParams& p, int dtype, int dim, bool pdl, cudaStream_t s, int* grid);
cudaError_t launch_prefix_join(const PrefixParams& p, int dtype, int dim, bool pdl, cudaStream_t s, int* grid);

}  // namespace dc
