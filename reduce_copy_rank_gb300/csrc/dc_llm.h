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
// computed by a CTA each.
constexpr uint64_t kAttendCounterBytes = 1 << 20;
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

}  // namespace dc
