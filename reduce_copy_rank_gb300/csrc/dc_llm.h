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
// The vocabulary is cut into segments of kVocabSeg entries, counted over the
// concatenated shards; one warp reduces one segment, and a row's segments are
// folded in one fixed order.  The tree of additions therefore depends on the
// vocabulary alone: not on the rows of the call, the shards or the grid.
constexpr int kVocabSeg = 2048;
constexpr int kScoreWarps = 8;      // warps per CTA
constexpr int kScoreMaxCluster = 8; // CTAs that may share a row
constexpr int kMaxVocab = 1 << 22;  // 24 KB of segment partials
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

constexpr int kAppendThreads = 256;
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
constexpr int kAttendMinChunk = 128;  // tokens of the shortest piece of a sequence
constexpr int kAttendMaxChunk = 4096; // ... and of the longest

struct AttendParams {
  uint64_t q, q_seq, q_head;            // bytes
  uint64_t out, out_seq, out_head;
  uint64_t lse;                         // f32 [seqs, q_heads] or 0
  uint64_t table, lengths;              // int32
  uint64_t counters;                    // uint32 [seqs * kv_heads * head blocks], zero between calls
  uint64_t partial;                     // f32 [seqs * kv_heads * head blocks, splits, HB, dim + 2]
  int64_t table_stride;
  int64_t num_pages;
  uint32_t page_size, table_width;
  int32_t seqs, q_heads, kv_heads, group, head_blocks;
  int32_t window;
  int32_t target;                       // pieces a long sequence is cut into
  int32_t splits;                       // pieces of the longest sequence that the table holds
  uint32_t page_slots;                  // page numbers one piece may touch
  float scale;
  PagedView kc, vc;
};

// Pieces a sequence of n attended tokens is cut into, and their length: a
// function of n and of `target` (which the head counts give) alone.
__host__ __device__ inline uint32_t attend_chunk(uint32_t n, uint32_t target) {
  const uint32_t per = (n / target + (n % target != 0) + 63u) / 64u * 64u;
  return per < kAttendMinChunk ? kAttendMinChunk : per > kAttendMaxChunk ? kAttendMaxChunk : per;
}
__host__ __device__ inline uint32_t attend_splits(uint32_t n, uint32_t target) {
  const uint32_t c = attend_chunk(n, target);
  return n / c + (n % c != 0);
}
// `target` for the units (key heads x head blocks) of one sequence: enough
// pieces that one long sequence alone fills 304 CTAs, two for each of the
// GPU's 152 SMs.
__host__ __device__ inline int attend_target(int units) {
  const int t = 304 / units;
  return t < 16 ? 16 : t > 128 ? 128 : t;
}
constexpr int kAttendMaxSplits = 512; // of the longest sequence (2M tokens)
// Heads that one CTA serves: 8, or 16 where a key head has more than 8 query heads.
__host__ __device__ inline int attend_head_block(int group) { return group > 8 ? 16 : 8; }
cudaError_t launch_attend(const AttendParams& p, int dtype, int dim, bool pdl, cudaStream_t s, int* grid);

}  // namespace dc
