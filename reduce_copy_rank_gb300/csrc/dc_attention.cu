// Attention of one new token per sequence over a paged key-value cache.
//
// Mathematics.  For sequence b with n attended tokens and query head h of
// key head k:  o = sum_t softmax_t(scale q.k_t) v_t.  Any run of tokens keeps,
// per head, a reference r, l = sum 2^(s_t - r) and the unnormalised output
// u = sum 2^(s_t - r) v_t, in binary32 (s_t = scale log2(e) q.k_t).  r is the
// running maximum rounded up to a whole number: changing it multiplies by a
// power of two, which rounds nothing, so a result depends only on the order
// in which the terms are added.  That order is one binary tree over leaves of
// 32 to 128 tokens (more in very long sequences), fixed by n alone; how large a
// subtree a warp, a CTA or a group of CTAs computes is free, and follows from
// how much work there is.  So neither the rest of the batch nor the grid
// changes a bit.  The last CTA to finish joins what is left of the tree.
//
// Bound: memory.  Every key and value is read once; at 8 query heads per key
// head that is 8 multiply-adds per byte, which the matrix pipe does with a
// wide margin (mma.m16n8k16, 16 heads x 8 tokens), so it is fed from shared
// memory by cp.async and never waited for.  A warp owns 16 tokens at a time
// with a ring of its own: no barrier until its subtree is done.  (Above 128
// columns two or three warps share the tokens, a part of the columns each, and
// add their scores up through shared memory.)
//
// Where a unit's pieces fit one cluster and the GPU has room, its CTAs join them
// through shared memory; else through the workspace, the last to arrive doing
// it.  Measured on GB300 (copy rate 6.78 TB/s; launches replayed from a graph), heads
// of 128: 128 ragged sequences up to 8192 tokens, 32/8 heads: 348 us, 6.3 TB/s; one
// of 131072, 64/8 heads: 94 us, 5.7 TB/s; 32 ragged up to 8000, 64/4 heads: 64 us, 3.2
// TB/s; one of 1024, 32/8 heads: 5.6 us.  What is left is latency: a piece of
// 256 tokens spends 0.35 us on its length, 1.3 on its page, query and first
// copies, 2.4 on its tiles (16 cp.async hold a warp for 450 of a tile's 1200
// cycles) and 0.6 on its end, and 8 warps an SM are all that registers allow.
//
// Rounding.  The weights 2^(s-r) enter the second product as a pair of 16-bit
// numbers hi + lo (hi the weight cut to 16 bits, lo the rounded rest), so
// that the output carries one rounding to 16 bits, the last.  With at most 8
// heads to a CTA the pair fills the tile's 16 rows and costs nothing.
// binary16 has no numbers below 2^-24, so there the weights enter times 2^15 and
// lo times 2^11 more, summed apart from hi (in the lower 8 rows; of more heads,
// tile by tile), the powers of two taken out again in binary32.  A weight is then
// held to 2^-20 of itself and 2^-50 of its leaf's largest: with values up to
// 65504 in a leaf of 128 tokens that is 2^-27, less than half the least binary16
// number.  (In units of the weights alone it was 2^-25, and a token far ahead
// with a small value left nothing of the others.)
#include <atomic>

#include "dc_llm.h"
#include "dc_numeric.cuh"

namespace dc {
namespace {

enum : uint32_t {
  kSiteLength = 1, kSiteTable = 2, kSiteQuery = 3, kSiteKey = 4, kSiteValue = 5, kSiteOut = 6, kSitePartial = 7,
};

// A head size's share of a CTA: kAttendWarps runs of tokens, each of one warp,
// or of two or three that hold a part of the columns each where a head has more
// than 128.  (One warp's registers held no subtrees of so many and its ring two
// tiles, and an SM had four warps.  32 ragged sequences up to 8000 tokens, 16/4
// heads of 256, one / two warps: 105 / 90 us; of 192, one / two / three: 73.5 /
// 81 / 70: halves of 192 columns cut the 128-byte lines.)  Shared memory: each
// warp's ring of tiles, then the partial scores of a run's warps.
template <int D, int HB, bool APART>
struct Shape {
  static constexpr int kParts = D == 192 && HB == 8 && !APART ? 3 : D > 128 ? 2 : 1;  // warps per run of tokens
  static constexpr int kThreads = kAttendWarps * kParts * 32;
  static constexpr int kCols = D / kParts;          // columns of a warp
  static constexpr int kRow = kCols * 2 + 16;       // bytes; the 16 keep ldmatrix free of conflicts
  static constexpr int kHalf = kAttendTile * kRow;  // keys or values of one tile
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kStages = 3;
  static constexpr int kRing = kAttendWarps * kParts * kStages * kStage;
  static constexpr int kValues = kCols / 4 * (HB / 8);  // of a head block's output that a lane holds
  static constexpr int kLevels = attend_levels(D, HB);
  static constexpr int kExchange = kParts > 1 ? kAttendWarps * 2 * kParts * (HB / 8) * 512 : 0;
  static constexpr int kBytes = kRing + kExchange;
  static constexpr int kCtas = attend_ctas_per_sm(D, HB);
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void st_shared4(uint32_t a, const float4& v) {
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(a), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w) : "memory");
}
__device__ __forceinline__ float4 ld_shared4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}
// The warps of a run of tokens wait for one another (all take as many tiles).
template <int WARPS>
__device__ __forceinline__ void run_barrier(int run) {
  asm volatile("bar.sync %0, %1;" ::"r"(run + 1), "n"(WARPS * 32) : "memory");
}

// Shared memory of CTA `rank` of the cluster, at this CTA's address `a`.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t a, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 ld_cluster4(uint32_t a, uint32_t rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr(a, rank))
               : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t a, uint32_t rank) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0,%1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(cluster_addr(a, rank)) : "memory");
  return v;
}
// All threads of the cluster.
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// 16 bytes global -> shared, or 16 zero bytes (nothing is read then).
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, uint64_t src, bool read) {
  const uint32_t n = read ? 16u : 0u;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}

template <int DT>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (DT == kF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The weights' units in the second product: hi is weight * kWeightUnit, lo the
// rest of that times kLowUnit.  (A weight is at most 1, so in binary16 hi is at
// most 2^15 and lo, less than 2^-10 of it, below 2^16.)
template <int DT>
constexpr float kWeightUnit = DT == kF16 ? 32768.0f : 1.0f;
template <int DT>
constexpr float kLowUnit = DT == kF16 ? 2048.0f : 1.0f;

// hi: both weights cut to 16 bits; lo: what that left out, rounded.  lo stays
// positive (2^-20 of the weight at least), so that an infinite value gives an
// infinity and not 0 * inf (in binary16, where 2^-24 is the least, for weights
// above 2^-31 of the leaf's largest; below, an infinite value gives NaN).
template <int DT>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t& hi, uint32_t& lo) {
  x *= kWeightUnit<DT>;
  y *= kWeightUnit<DT>;
  if constexpr (DT == kF16)
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(y), "f"(x));
  else
    asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(y), "f"(x));
  constexpr float kLeast = kLowUnit<DT> / (1 << 20);
  lo = Elem<DT>::pack(fmaxf((x - Elem<DT>::lo(hi)) * kLowUnit<DT>, x * kLeast),
                      fmaxf((y - Elem<DT>::hi(hi)) * kLowUnit<DT>, y * kLeast));
}

// Stores `v` as a 16-bit element pair.
template <int DT>
__device__ __forceinline__ void st_pair(uint64_t a, float x, float y, uint64_t lo, uint64_t hi) {
  if (in_bounds(reinterpret_cast<const void*>(a), 4, lo, hi, kSiteOut))
    *reinterpret_cast<uint32_t*>(a) = Elem<DT>::pack(x, y);
}

// 2^(x - M) for whole numbers x <= M; 0 below 2^-126, and for x = -inf.
__device__ __forceinline__ float pow2_diff(float x, float M) {
  const int k = static_cast<int>(fmaxf(x - M, -127.0f));
  return __int_as_float((k + 127) << 23);
}

// A run of tokens: reference, sum and output of a lane's heads.
template <int NV, int R>
struct Run {
  float v[NV];  // [column group][half of the heads][2]
  float ref[R], l[R];
};

// b = a + b, a the earlier tokens.
template <int NV, int R>
__device__ __forceinline__ void join(const Run<NV, R>& a, Run<NV, R>& b) {
#pragma unroll
  for (int h = 0; h < R; ++h) {
    const float M = fmaxf(a.ref[h], b.ref[h]);
    const float fa = pow2_diff(a.ref[h], M), fb = pow2_diff(b.ref[h], M);
    b.ref[h] = M;
    b.l[h] = __fmaf_rn(a.l[h], fa, b.l[h] * fb);
#pragma unroll
    for (int i = h * 2; i < NV; i += 2 * R)
#pragma unroll
      for (int e = 0; e < 2; ++e) b.v[i + e] = __fmaf_rn(a.v[i + e], fa, b.v[i + e] * fb);
  }
}

// The sum of 8 values as the tree of them.
template <class F>
__device__ __forceinline__ float tree8(F x) {
  return ((x(0) + x(1)) + (x(2) + x(3))) + ((x(4) + x(5)) + (x(6) + x(7)));
}

// The sum of 16 values as the tree of them.
template <class F>
__device__ __forceinline__ float tree16(F x) {
  float a[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = x(2 * i) + x(2 * i + 1);
  return ((a[0] + a[1]) + (a[2] + a[3])) + ((a[4] + a[5]) + (a[6] + a[7]));
}

// Where a unit's pieces leave their runs: [piece][head][D] outputs, then
// [piece][head] (reference, sum), then the same of each joined group (whose
// output replaces its first piece's).
struct Pieces {
  float* out;
  float2* rl;
  uint64_t lo, hi;  // their bytes
};

template <int D, int HB>
__device__ __forceinline__ void st_piece(const Pieces& w, uint32_t piece, uint32_t rl, int h, int d, const float4& v,
                                         float ref, float l) {
  float4* a = reinterpret_cast<float4*>(w.out + (static_cast<uint64_t>(piece) * HB + h) * D + d);
  if (in_bounds(a, 16, w.lo, w.hi, kSitePartial)) *a = v;
  if (d == 0) {
    float2* b = w.rl + static_cast<uint64_t>(rl) * HB + h;
    if (in_bounds(b, 8, w.lo, w.hi, kSitePartial)) *b = make_float2(ref, l);
  }
}

// The finished output of head h (of the CTA's), columns d .. d + 3.
template <int DT, int D>
__device__ __forceinline__ void st_result(const AttendParams& p, int seq, int head, int d, const float4& v, float ref,
                                          float l) {
  const float inv = 1.0f / l;
  const uint64_t row = p.out + static_cast<uint64_t>(seq) * p.out_seq + static_cast<uint64_t>(head) * p.out_head;
  st_pair<DT>(row + d * 2, v.x * inv, v.y * inv, row, row + D * 2);
  st_pair<DT>(row + d * 2 + 4, v.z * inv, v.w * inv, row, row + D * 2);
  if (d == 0 && p.lse) {
    float* a = reinterpret_cast<float*>(p.lse) + static_cast<uint64_t>(seq) * p.q_heads + head;
    if (in_bounds(a, 4, p.lse, p.lse + 4ull * p.seqs * p.q_heads, kSiteOut)) *a = (ref + log2f(l)) * kLn2;
  }
}

// True in every thread of the CTA that arrives last of `n`; the counter is
// then 0 again, and what the others wrote before arriving is visible (the
// barrier orders the CTA's writes before thread 0's release; its acquire and
// the second barrier order the other CTAs' writes before this CTA's reads,
// which bypass L1).
__device__ __forceinline__ bool arrive_last(uint32_t* counter, uint32_t n, uint32_t* flag) {
  __syncthreads();
  if (threadIdx.x == 0) {
    uint32_t before;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(before) : "l"(counter) : "memory");
    if (before == n - 1) *counter = 0;
    *flag = before == n - 1 ? 1u : 0u;
  }
  __syncthreads();
  return *flag != 0;
}

// APART: 8 heads that share their keys with 8 others, computed as 16 in a block
// are, with the weights' high and low parts in a product each.
// LOOP: a unit has fewer CTAs than its longest sequence could have pieces, and
// a CTA takes every p.places-th of them.
template <int DT, int D, int HB, bool LOOP, bool APART>
__global__ __launch_bounds__(Shape<D, HB, APART>::kThreads, Shape<D, HB, APART>::kCtas) void dc_attend_kernel(const __grid_constant__ AttendParams p) {
  using S = Shape<D, HB, APART>;
  constexpr int R = HB / 8;
  using State = Run<S::kValues, R>;
  constexpr int C = S::kCols;
  constexpr int kThreads = S::kThreads;
  constexpr int kSteps = C / 16;  // k-steps of q.k, and 16-element column groups of the output
  constexpr bool kLowApart = kLowUnit<DT> != 1.0f;  // hi and lo do not add up as they are
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float w_ref[kAttendWarps][HB], w_l[kAttendWarps][HB];
  __shared__ uint32_t last_flag;
  const int lane = threadIdx.x & 31;
  // run of tokens `warp`, columns [col0, col0 + C)
  const int warp = static_cast<int>(threadIdx.x >> 5) / S::kParts, column = static_cast<int>(threadIdx.x >> 5) % S::kParts;
  const int col0 = column * C;

  __shared__ float2 c_rl[HB];  // this CTA's piece, for its cluster
  uint32_t piece = blockIdx.x % static_cast<uint32_t>(p.places);
  const uint32_t unit = blockIdx.x / static_cast<uint32_t>(p.places);  // (sequence, key head, head block)
  const int hb = static_cast<int>(unit % static_cast<uint32_t>(p.head_blocks));
  const int kh = static_cast<int>(unit / static_cast<uint32_t>(p.head_blocks) % static_cast<uint32_t>(p.kv_heads));
  const int seq = static_cast<int>(unit / static_cast<uint32_t>(p.head_blocks) / static_cast<uint32_t>(p.kv_heads));
  const int h0 = kh * p.group + hb * HB;          // first query head
  const int nh = min(HB, p.group - hb * HB);      // query heads of this CTA
  pdl_enter();

  const int32_t* lp = reinterpret_cast<const int32_t*>(p.lengths) + seq;
  int32_t len = in_bounds(lp, 4, p.lengths, p.lengths + 4ull * p.seqs, kSiteLength) ? *lp : 0;
  // a length past the table: the tokens that exist are not known, the output is NaN
  const uint64_t room = static_cast<uint64_t>(p.table_width) * p.page_size;
  bool bad = len > 0 && static_cast<uint64_t>(len) > room;
  if (len < 0) len = 0;
  if (bad) len = 1;
  const uint32_t start = p.window > 0 && len > p.window ? static_cast<uint32_t>(len - p.window) : 0u;
  const uint32_t n = static_cast<uint32_t>(len) - start;
  const uint32_t leaf = attend_leaf(n);
  const uint32_t small = attend_pieces(n, 0);     // pieces of one leaf per warp
  const uint32_t level = attend_level(small, static_cast<uint32_t>(p.units), S::kLevels);
  const uint32_t pieces = attend_pieces(n, level);
  const bool in_cluster = p.cluster > 1 && pieces > 1;  // the unit's CTAs are one cluster
  if (piece >= pieces) {
    if (piece == 0) {  // nothing to attend to: zeros
      for (int i = threadIdx.x; i < nh * (D / 2); i += kThreads) {
        const uint64_t row = p.out + static_cast<uint64_t>(seq) * p.out_seq +
                             static_cast<uint64_t>(h0 + i / (D / 2)) * p.out_head;
        st_pair<DT>(row + static_cast<uint64_t>(i % (D / 2)) * 4, 0.0f, 0.0f, row, row + D * 2);
      }
      if (p.lse && threadIdx.x < nh) {
        float* a = reinterpret_cast<float*>(p.lse) + static_cast<uint64_t>(seq) * p.q_heads + h0 + threadIdx.x;
        if (in_bounds(a, 4, p.lse, p.lse + 4ull * p.seqs * p.q_heads, kSiteOut)) *a = neg_inf();
      }
    }
    if (in_cluster) {  // (all of a cluster take part in its two barriers)
      cluster_barrier();
      cluster_barrier();
    }
    return;
  }
  uint32_t qf[kSteps][2 * R];
  do {
  // this warp's tokens [t0, t1): a subtree of 2^level leaves
  const uint32_t run = leaf << level;
  const uint64_t first = static_cast<uint64_t>(start) + (static_cast<uint64_t>(piece) * kAttendWarps + warp) * run;
  const uint32_t t0 = static_cast<uint32_t>(min(first, static_cast<uint64_t>(len)));
  const uint32_t t1 = static_cast<uint32_t>(min(first + run, static_cast<uint64_t>(len)));
  const uint32_t tiles = (t1 - t0 + kAttendTile - 1) / kAttendTile;

  // A copy instruction moves 128 bytes of each of 4 rows (64 of 8 where rows
  // are no multiple of 128 bytes).  Most tiles lie in one page: their rows are
  // a stride apart.  In the others lanes 0..15 look up where the keys of the
  // tile's tokens are, lanes 16..31 their values, and hand the addresses on.
  constexpr int kLanes = C % 64 == 0 ? 8 : 4;       // lanes that copy one row
  constexpr int kRows = 32 / kLanes;                // rows an instruction touches
  constexpr int kGroups = kAttendTile / kRows;
  const uint32_t ring = smem_addr(smem) + static_cast<uint32_t>((warp * S::kParts + column) * S::kStages * S::kStage);
  const uint64_t table_row = p.table + static_cast<uint64_t>(seq) * static_cast<uint64_t>(p.table_stride) * 4;
  const uint64_t k_head = p.kc.base + static_cast<uint64_t>(kh) * p.kc.head + col0 * 2;
  const uint64_t v_head = p.vc.base + static_cast<uint64_t>(kh) * p.vc.head + col0 * 2;
  int32_t next_id = -1;     // the page of this lane's token of the next tile to copy, -1: no token
  uint32_t next_slot = 0;   // ... and its place in the page
  bool next_whole = false;  // the tile is 16 tokens of one page, next_slot its first token's place
  auto look_up = [&](uint32_t i) {
    if (i >= tiles) return;
    const uint32_t tile = t0 + i * kAttendTile;
    uint32_t pg = p.page_shift >= 0 ? tile >> p.page_shift : tile / p.page_size;
    next_slot = tile - pg * p.page_size;
    next_whole = tile + kAttendTile <= t1 && next_slot + kAttendTile <= p.page_size;
    if (!next_whole) {
      const uint32_t t = tile + (lane & 15);
      pg = p.page_shift >= 0 ? t >> p.page_shift : t / p.page_size;
      next_slot = t - pg * p.page_size;
      next_id = -1;
      if (t >= t1) return;
    }
    const int32_t* a = reinterpret_cast<const int32_t*>(table_row) + pg;
    next_id = in_bounds(a, 4, table_row, table_row + 4ull * p.table_width, kSiteTable) ? *a : -1;
  };
  auto copy = [&](uint32_t dst, int half, uint64_t src, bool read) {
#pragma unroll
    for (int c = 0; c < C / 8 / kLanes; ++c) {
      const uint64_t x = src + c * kLanes * 16;
      const bool ok = read && in_bounds(reinterpret_cast<const void*>(x), 16, half ? p.vc.lo : p.kc.lo,
                                        half ? p.vc.hi : p.kc.hi, half ? kSiteValue : kSiteKey);
      cp_async16_or_zero(dst + half * S::kHalf + c * kLanes * 16, ok ? x : p.kc.base, ok);
    }
  };
  auto issue = [&](uint32_t i) {
    if (i < tiles) {
      const uint32_t dst = ring + (i % S::kStages) * S::kStage + (lane / kLanes) * S::kRow + (lane % kLanes) * 16;
      // (a page outside the cache is never touched; ids past a sequence's end are not looked at)
      const bool there = next_id >= 0 && next_id < p.num_pages;
      if (!there && (next_whole || t0 + i * kAttendTile + (lane & 15) < t1)) bad = true;
      if (next_whole && there) {
        const uint64_t at = next_slot + lane / kLanes;
        uint64_t k = k_head + static_cast<uint64_t>(next_id) * p.kc.page + at * p.kc.token + (lane % kLanes) * 16;
        uint64_t v = v_head + static_cast<uint64_t>(next_id) * p.vc.page + at * p.vc.token + (lane % kLanes) * 16;
#pragma unroll
        for (int r = 0; r < kGroups; ++r) {
          copy(dst + r * kRows * S::kRow, 0, k, true);
          k += kRows * p.kc.token;
        }
#pragma unroll
        for (int r = 0; r < kGroups; ++r) {
          copy(dst + r * kRows * S::kRow, 1, v, true);
          v += kRows * p.vc.token;
        }
      } else {
        // (no row starts at 0; a whole tile of a missing page is 16 missing rows)
        const uint64_t row = !there ? 0 : (lane < 16 ? k_head : v_head) +
                                              static_cast<uint64_t>(next_id) * (lane < 16 ? p.kc.page : p.vc.page) +
                                              next_slot * (lane < 16 ? p.kc.token : p.vc.token);
#pragma unroll
        for (int r = 0; r < 2 * kGroups; ++r) {
          const uint64_t at = __shfl_sync(~0u, row, lane / kLanes + kRows * (r % kGroups) + 16 * (r / kGroups));
          copy(dst + r % kGroups * kRows * S::kRow, r / kGroups, at + (lane % kLanes) * 16, at != 0);
        }
      }
    }
    cp_async_commit();
    look_up(i + 1);
  };
  look_up(0);

  // query fragments: rows 0..7 heads h0.., rows 8..15 heads h0 + 8.. (HB 16)
  {
    const uint64_t q_seq = p.q + static_cast<uint64_t>(seq) * p.q_seq + static_cast<uint64_t>(h0) * p.q_head;
#pragma unroll
    for (int half = 0; half < R; ++half) {
      const int h = (lane >> 2) + 8 * half;
      const uint64_t row = q_seq + static_cast<uint64_t>(h) * p.q_head;
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t* a =
              reinterpret_cast<const uint32_t*>(row + static_cast<uint64_t>(col0 + k * 16 + i * 8 + (lane & 3) * 2) * 2);
          // a[0]: row g, first 8 columns; a[1]: row g + 8; a[2], a[3]: the next 8 columns
          qf[k][R * i + half] = h < nh && in_bounds(a, 4, row, row + D * 2, kSiteQuery) ? *a : 0u;
        }
    }
  }
#pragma unroll
  for (int i = 0; i < S::kStages - 1; ++i) issue(i);

  float m[R], l[R], o[C / 8][4];
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      m[i] = neg_inf();
      l[i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < C / 8; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.0f;
  };
  clear();
  const float sc = p.scale * kLog2E;

  // subtrees that wait for their right neighbour: slot b holds 2^b leaves
  State cur;
  State held[S::kLevels];
  [[maybe_unused]] const uint32_t exchange = smem_addr(smem) + S::kRing + static_cast<uint32_t>(warp * 2 * S::kParts * R * 512 + lane * 16);

  const uint32_t leaf_tiles = leaf / kAttendTile;
  uint32_t in_leaf = 0, leaves = 0;
  for (uint32_t i = 0; i < tiles; ++i) {
    cp_async_wait<S::kStages - 2>();
    __syncwarp();
    const uint32_t kt = ring + (i % S::kStages) * S::kStage, vt = kt + S::kHalf;
    // scores: 16 heads x 16 tokens, even and odd k-steps apart
    float s[2][2][4] = {};
    {
      const uint32_t a = kt + ((lane >> 4) * 8 + (lane & 7)) * S::kRow + ((lane >> 3) & 1) * 16;
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        uint32_t b[4];
        ldmatrix4(a + k * 32, b);
        uint32_t q[4];
        if constexpr (HB == 16) {
#pragma unroll
          for (int j = 0; j < 4; ++j) q[j] = qf[k][j];
        } else {
          q[0] = qf[k][0];
          q[1] = 0;
          q[2] = qf[k][1];
          q[3] = 0;
        }
        mma<DT>(s[k & 1][0], q, b[0], b[1]);
        mma<DT>(s[k & 1][1], q, b[2], b[3]);
      }
    }
    issue(i + S::kStages - 1);  // (its stage was read in the last round)
    if constexpr (S::kParts > 1) {
      // the sums over all columns: the warps' shares in order (two buffers: a
      // warp writes one again only after the others have read it)
      const uint32_t at = exchange + (i & 1) * (S::kParts * R * 512);
#pragma unroll
      for (int half = 0; half < R; ++half)
        st_shared4(at + (column * R + half) * 512,
                   make_float4(s[0][0][2 * half] + s[1][0][2 * half], s[0][0][2 * half + 1] + s[1][0][2 * half + 1],
                               s[0][1][2 * half] + s[1][1][2 * half], s[0][1][2 * half + 1] + s[1][1][2 * half + 1]));
      run_barrier<S::kParts>(warp);
#pragma unroll
      for (int half = 0; half < R; ++half) {
        float4 v = ld_shared4(at + half * 512);
#pragma unroll
        for (int c = 1; c < S::kParts; ++c) {
          const float4 w = ld_shared4(at + (c * R + half) * 512);
          v = make_float4(v.x + w.x, v.y + w.y, v.z + w.z, v.w + w.w);
        }
        s[0][0][2 * half] = v.x;
        s[0][0][2 * half + 1] = v.y;
        s[0][1][2 * half] = v.z;
        s[0][1][2 * half + 1] = v.w;
      }
    }
    const uint32_t base = t0 + i * kAttendTile;
    const bool partial = base + kAttendTile > t1;
    uint32_t phi[4], plo[4];
#pragma unroll
    for (int half = 0; half < R; ++half) {
      float x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        x[j] = (s[0][j >> 1][2 * half + (j & 1)] + (S::kParts == 1 ? s[1][j >> 1][2 * half + (j & 1)] : 0.0f)) * sc;
      if (partial) {
        const uint32_t t = base + (lane & 3) * 2;
        if (t >= t1) x[0] = neg_inf();
        if (t + 1 >= t1) x[1] = neg_inf();
        if (t + 8 >= t1) x[2] = neg_inf();
        if (t + 9 >= t1) x[3] = neg_inf();
      }
      float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
      mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 2));
      if (__any_sync(~0u, mx > m[half])) {
        const float mn = fmaxf(m[half], ceilf(mx));
        const float f = pow2_diff(m[half], mn);
        l[half] *= f;
#pragma unroll
        for (int c = 0; c < C / 8; ++c) {
          if constexpr (HB == 16) {
            o[c][2 * half] *= f;
            o[c][2 * half + 1] *= f;
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) o[c][j] *= f;
          }
        }
        m[half] = mn;
      }
      const float ref = m[half] == neg_inf() ? 0.0f : m[half];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j] = ex2(x[j] - ref);
        l[half] += x[j];
      }
      split_pair<DT>(x[0], x[1], phi[half], plo[half]);
      split_pair<DT>(x[2], x[3], phi[2 + half], plo[2 + half]);
    }
    {
      const uint32_t a = vt + (((lane >> 3) & 1) * 8 + (lane & 7)) * S::kRow + (lane >> 4) * 16;
      uint32_t w[4];
      if constexpr (HB == 8) {
        w[0] = phi[0];
        w[1] = APART && !kLowApart ? 0 : plo[0];
        w[2] = phi[2];
        w[3] = APART && !kLowApart ? 0 : plo[2];
      }
      [[maybe_unused]] const uint32_t low[4] = {plo[0], 0, plo[2], 0};  // (APART)
#pragma unroll
      for (int c = 0; c < kSteps; ++c) {
        uint32_t b[4];
        ldmatrix4_t(a + c * 32, b);
        if constexpr (HB == 16) {
          mma<DT>(o[2 * c], phi, b[0], b[1]);
          mma<DT>(o[2 * c + 1], phi, b[2], b[3]);
          if constexpr (kLowApart) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float t[4] = {};
              mma<DT>(t, plo, b[2 * i], b[2 * i + 1]);
#pragma unroll
              for (int j = 0; j < 4; ++j) o[2 * c + i][j] = __fmaf_rn(t[j], 1.0f / kLowUnit<DT>, o[2 * c + i][j]);
            }
          } else {
            mma<DT>(o[2 * c], plo, b[0], b[1]);
            mma<DT>(o[2 * c + 1], plo, b[2], b[3]);
          }
        } else {
          mma<DT>(o[2 * c], w, b[0], b[1]);
          mma<DT>(o[2 * c + 1], w, b[2], b[3]);
          if constexpr (APART && kLowApart) {  // the tile's low parts, added as 16 heads' are
#pragma unroll
            for (int i = 2 * c; i < 2 * c + 2; ++i)
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                o[i][j] = __fmaf_rn(o[i][2 + j], 1.0f / kLowUnit<DT>, o[i][j]);
                o[i][2 + j] = 0.0f;
              }
          } else if constexpr (APART) {
            mma<DT>(o[2 * c], low, b[0], b[1]);
            mma<DT>(o[2 * c + 1], low, b[2], b[3]);
          }
        }
      }
    }
    __syncwarp();
    if (++in_leaf == leaf_tiles || i + 1 == tiles) {  // a leaf is done: up the tree
      in_leaf = 0;
#pragma unroll
      for (int half = 0; half < R; ++half) {
        l[half] += __shfl_xor_sync(~0u, l[half], 1);
        l[half] += __shfl_xor_sync(~0u, l[half], 2);
        cur.ref[half] = m[half];
        cur.l[half] = l[half];
      }
      constexpr float kUnit = 1.0f / kWeightUnit<DT>, kLow = kUnit / kLowUnit<DT>;
#pragma unroll
      for (int c = 0; c < C / 8; ++c) {
        if constexpr (HB == 16) {
#pragma unroll
          for (int j = 0; j < 4; ++j) cur.v[4 * c + j] = o[c][j] * kUnit;
        } else {  // rows 8..15 hold the low parts (nothing if those have a product of their own)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            cur.v[2 * c + j] = APART ? o[c][j] * kUnit : __fmaf_rn(o[c][2 + j], kLow, o[c][j] * kUnit);
        }
      }
      // (at most 2^kLevels leaves; the last one's subtree stays in cur)
      if (leaves & 1) join(held[0], cur);
      if constexpr (S::kLevels > 1)
        if ((leaves & 3) == 3) join(held[1], cur);
      ++leaves;
      if (i + 1 < tiles) {
        if (leaves & 1) held[0] = cur;
        else if constexpr (S::kLevels > 1) held[1] = cur;
        clear();
      }
    }
  }
  cp_async_wait<0>();
  if (tiles == 0) {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      cur.ref[i] = neg_inf();
      cur.l[i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < S::kValues; ++i) cur.v[i] = 0.0f;
  } else if constexpr (S::kLevels > 1) {
    if (leaves == 3) join(held[1], cur);  // a last leaf without a neighbour
  }

  // the piece: the warps' subtrees
  if ((lane & 3) == 0 && column == 0) {
#pragma unroll
    for (int half = 0; half < R; ++half) {
      w_ref[warp][(lane >> 2) + 8 * half] = cur.ref[half];
      w_l[warp][(lane >> 2) + 8 * half] = cur.l[half];
    }
  }
  bad = __syncthreads_or(bad);  // every warp has read its last tile: the ring is free
  float* wo = reinterpret_cast<float*>(smem);  // [warp][head][D]
  static_assert(kAttendWarps * HB * D * 4 <= S::kRing, "the warps' outputs fit in the ring");
  {
    const int g = lane >> 2;
#pragma unroll
    for (int c = 0; c < C / 8; ++c)
#pragma unroll
      for (int half = 0; half < R; ++half)
        *reinterpret_cast<float2*>(wo + (warp * HB + g + 8 * half) * D + col0 + c * 8 + (lane & 3) * 2) =
            make_float2(cur.v[c * 2 * R + 2 * half], cur.v[c * 2 * R + 2 * half + 1]);
  }
  __syncthreads();
  Pieces w;
  {
    const uint64_t floats = static_cast<uint64_t>(HB) * (static_cast<uint64_t>(p.pieces) * (D + 2) + 2 * kAttendGroups);
    w.out = reinterpret_cast<float*>(p.partial) + unit * floats;
    w.rl = reinterpret_cast<float2*>(w.out + static_cast<uint64_t>(p.pieces) * HB * D);
    w.lo = reinterpret_cast<uint64_t>(w.out);
    w.hi = w.lo + floats * 4;
  }
  for (int i = threadIdx.x; i < nh * (D / 4); i += kThreads) {
    const int h = i / (D / 4), d = i % (D / 4) * 4;
    float M = w_ref[0][h], f[kAttendWarps];
#pragma unroll
    for (int k = 1; k < kAttendWarps; ++k) M = fmaxf(M, w_ref[k][h]);
    float4 x[kAttendWarps];
    float ls[kAttendWarps];
#pragma unroll
    for (int k = 0; k < kAttendWarps; ++k) {
      f[k] = pow2_diff(w_ref[k][h], M);
      x[k] = *reinterpret_cast<const float4*>(wo + (k * HB + h) * D + d);
      ls[k] = w_l[k][h] * f[k];
    }
    static_assert(kAttendWarps == 4, "the tree below is of four");
    float l4 = (ls[0] + ls[1]) + (ls[2] + ls[3]);
    if (bad) l4 = __int_as_float(0x7FC00000);
    const float4 v = make_float4((x[0].x * f[0] + x[1].x * f[1]) + (x[2].x * f[2] + x[3].x * f[3]),
                                 (x[0].y * f[0] + x[1].y * f[1]) + (x[2].y * f[2] + x[3].y * f[3]),
                                 (x[0].z * f[0] + x[1].z * f[1]) + (x[2].z * f[2] + x[3].z * f[3]),
                                 (x[0].w * f[0] + x[1].w * f[1]) + (x[2].w * f[2] + x[3].w * f[3]));
    if (pieces == 1) st_result<DT, D>(p, seq, h0 + h, d, v, M, l4);
    else if (in_cluster) {
      // for the cluster: in place of what this thread alone has read
      *reinterpret_cast<float4*>(wo + h * D + d) = v;
      if (d == 0) c_rl[h] = make_float2(M, l4);
    } else st_piece<D, HB>(w, piece, piece, h, d, v, M, l4);
  }
  if (pieces == 1) return;

  const uint32_t per_unit = attend_counters(static_cast<uint32_t>(p.pieces));
  uint32_t* counters = reinterpret_cast<uint32_t*>(p.counters) + static_cast<uint64_t>(unit) * per_unit;
  if (in_cluster) {
    // the pieces are one cluster's CTAs: each joins a share of the columns
    // from all of them, through shared memory
    const uint32_t count = pieces, rank = piece;
    cluster_barrier();
    const uint32_t wo_at = smem_addr(wo), rl_at = smem_addr(c_rl);
    for (int i = static_cast<int>(rank) * kThreads + threadIdx.x; i < nh * (D / 4); i += static_cast<int>(count) * kThreads) {
      const int h = i / (D / 4), d = i % (D / 4) * 4;
      float4 x[kAttendCluster];
      float2 rl[kAttendCluster];
#pragma unroll
      for (uint32_t k = 0; k < kAttendCluster; ++k) {
        x[k] = k < count ? ld_cluster4(wo_at + static_cast<uint32_t>(h * D + d) * 4, k) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        rl[k] = k < count ? ld_cluster2(rl_at + h * 8, k) : make_float2(neg_inf(), 0.0f);
      }
      float M = rl[0].x, f[kAttendCluster];
#pragma unroll
      for (int k = 1; k < kAttendCluster; ++k) M = fmaxf(M, rl[k].x);
#pragma unroll
      for (int k = 0; k < kAttendCluster; ++k) f[k] = pow2_diff(rl[k].x, M);
      const float l8 = tree8([&](int k) { return rl[k].y * f[k]; });
      const float4 v = make_float4(tree8([&](int k) { return x[k].x * f[k]; }), tree8([&](int k) { return x[k].y * f[k]; }),
                                   tree8([&](int k) { return x[k].z * f[k]; }), tree8([&](int k) { return x[k].w * f[k]; }));
      st_result<DT, D>(p, seq, h0 + h, d, v, M, l8);
    }
    cluster_barrier();  // no CTA leaves while another reads its shared memory
    return;
  }

  // the last of 16 neighbouring pieces joins them, the last such group the groups
  const uint32_t groups = (pieces + kAttendJoin - 1) / kAttendJoin;
  uint32_t base = piece / kAttendJoin * kAttendJoin, step = 1;
  uint32_t count = min(static_cast<uint32_t>(kAttendJoin), pieces - base);
  const bool alone = LOOP && p.places == 1;  // this CTA has computed them all, in order
  bool last;
  if (alone) {
    __syncthreads();  // its threads' parts of the pieces
    last = piece + 1 == base + count;
  } else {
    last = arrive_last(counters + (per_unit > 1 ? 1 : 0) + piece / kAttendJoin, count, &last_flag);
  }
  while (last) {
    const bool done = step > 1 || groups == 1;
    for (int i = threadIdx.x; i < nh * (D / 4); i += kThreads) {
      const int h = i / (D / 4), d = i % (D / 4) * 4;
      // every load is issued before the first is used: one latency
      float4 x[kAttendJoin];
      float2 rl[kAttendJoin];
#pragma unroll
      for (uint32_t k = 0; k < kAttendJoin; ++k) {
        const float4* a = reinterpret_cast<const float4*>(w.out + ((static_cast<uint64_t>(base) + k * step) * HB + h) * D + d);
        const float2* b = w.rl + (static_cast<uint64_t>(step == 1 ? base : p.pieces) + k) * HB + h;
        const bool read = k < count && in_bounds(a, 16, w.lo, w.hi, kSitePartial) &&
                          in_bounds(b, 8, w.lo, w.hi, kSitePartial);
        x[k] = read ? __ldcg(a) : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        rl[k] = read ? __ldcg(b) : make_float2(neg_inf(), 0.0f);
      }
      float M = rl[0].x, f[kAttendJoin];
#pragma unroll
      for (int k = 1; k < kAttendJoin; ++k) M = fmaxf(M, rl[k].x);
#pragma unroll
      for (int k = 0; k < kAttendJoin; ++k) f[k] = pow2_diff(rl[k].x, M);
      const float l16 = tree16([&](int k) { return rl[k].y * f[k]; });
      const float4 v = make_float4(tree16([&](int k) { return x[k].x * f[k]; }), tree16([&](int k) { return x[k].y * f[k]; }),
                                   tree16([&](int k) { return x[k].z * f[k]; }), tree16([&](int k) { return x[k].w * f[k]; }));
      if (done) st_result<DT, D>(p, seq, h0 + h, d, v, M, l16);
      else st_piece<D, HB>(w, base, p.pieces + base / kAttendJoin, h, d, v, M, l16);
    }
    if (done) break;
    if (alone) {
      __syncthreads();
      last = piece + 1 == pieces;
    } else {
      last = arrive_last(counters, groups, &last_flag);
    }
    base = 0;
    step = kAttendJoin;
    count = groups;
  }
  if (LOOP) __syncthreads();  // the ring is free for the CTA's next piece
  } while (LOOP && (piece += static_cast<uint32_t>(p.places)) < pieces);
}

template <int DT, int D, int HB, bool LOOP, bool APART>
cudaError_t launch_one(const AttendParams& p, bool pdl, cudaStream_t s, int grid) {
  constexpr int kSmem = Shape<D, HB, APART>::kBytes;
  static_assert(kSmem + 4096 <= 227 * 1024, "the ring and the partial scores fit");
  static std::atomic<uint64_t> allowed{0};  // devices whose limit is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(allowed.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(dc_attend_kernel<DT, D, HB, LOOP, APART>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    allowed.fetch_or(bit, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(Shape<D, HB, APART>::kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  unsigned n = 0;
  if (p.cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = static_cast<unsigned>(p.cluster);
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = n ? attr : nullptr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, dc_attend_kernel<DT, D, HB, LOOP, APART>, p);
}

template <int DT, int D>
cudaError_t launch_hb(const AttendParams& p, bool pdl, cudaStream_t s, int grid) {
  const bool loop = p.places < p.pieces;
  if (p.hb == 16)
    return loop ? launch_one<DT, D, 16, true, false>(p, pdl, s, grid) : launch_one<DT, D, 16, false, false>(p, pdl, s, grid);
  // (few CTAs, or there would be 16 heads to a block: never in turns)
  if (p.group > 8) return loop ? cudaErrorInvalidValue : launch_one<DT, D, 8, false, true>(p, pdl, s, grid);
  return loop ? launch_one<DT, D, 8, true, false>(p, pdl, s, grid) : launch_one<DT, D, 8, false, false>(p, pdl, s, grid);
}

template <int DT>
cudaError_t launch_dim(const AttendParams& p, int dim, bool pdl, cudaStream_t s, int grid) {
  switch (dim) {
    case 64: return launch_hb<DT, 64>(p, pdl, s, grid);
    case 96: return launch_hb<DT, 96>(p, pdl, s, grid);
    case 128: return launch_hb<DT, 128>(p, pdl, s, grid);
    case 192: return launch_hb<DT, 192>(p, pdl, s, grid);
    default: return launch_hb<DT, 256>(p, pdl, s, grid);
  }
}

}  // namespace

cudaError_t launch_attend(const AttendParams& p, int dtype, int dim, bool pdl, cudaStream_t s, int* grid) {
  *grid = p.seqs * p.kv_heads * p.head_blocks * p.places;
  return dtype == kF16 ? launch_dim<kF16>(p, dim, pdl, s, *grid) : launch_dim<kBF16>(p, dim, pdl, s, *grid);
}

DC_BOUNDS_READER(take_bounds_attention)

}  // namespace dc
