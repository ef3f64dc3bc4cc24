// Log probabilities of tokens from hidden rows and a head's weights, without
// keeping the logits, and the gradient of that.
//
// Mathematics.  x = h W^T over a vocabulary, z = x / temperature; lse =
// log sum exp z, log p_y = z_y - lse, entropy = lse - sum p z.  With upstream
// gradients g and e of a row's log probability and entropy the logits' gradient
// is d_j = (g ([j = y] - p_j) - e p_j (log p_j + entropy)) / temperature, and
// dh = d W, dW = d^T h.
//
// The products run on the tensor cores (tcgen05.mma, operands by TMA, binary32
// accumulators in tensor memory).  A pair of CTAs on two SMs takes tiles of 256 x
// 256 in turn, each with 128 of the rows and half of B's columns in its shared
// memory; while one is computed eight warps reduce the one before from tensor
// memory:
//  * forward: a row's part of the tile as its largest logit m, sum 2^(z-r) and sum
//    2^(z-r) (z-r), z in units of log2 and r that of m, written as 16 bytes; a
//    second kernel adds a row's parts up in one fixed order, which depends on the
//    shards' widths alone.
//  * backward, for up to 24576 columns of a shard at a time: the logits again,
//    from which d is written in 16 bits; then d W, added to binary32 sums, and
//    d^T h in one launch, whose tiles are shared out so that all CTAs end together.
// Neither the number of rows nor the grid changes a bit of a row's results (DC_F16's
// gradient: beyond its power of two, which all rows' upstream gradients decide).  How the
// vocabulary is cut into shards and chunks decides the order of dh's sums.
//
// Rounding: d is rounded to 16 bits before its products (half a step of each: 2^-8
// of it for DC_BF16, 2^-11 for DC_F16), as an activation's gradient is; the sums are
// binary32.  What that takes from the largest element of most rows, the token's, is
// kept in 32 bits and put back into both products where they are stored: d e_y^T is
// one row of the weights for dh, and one row of h for the token's row of dW.  The
// gradients' errors are then those of their last rounding where single tokens make
// them up (4096 rows, 127900 columns: 0.0017 of the gradients, 0.0025 without).  For
// DC_F16 d is multiplied by one power of two for all rows, so that the largest possible
// is between 2^14 and 2^15: what is 2^-29 of that is still a normal number.
//
// Bound: the tensor cores for training batches, the weights' bytes for few rows.
// Measured, BF16, 4096 rows of 4096 against 128000 columns: forward 2.62 to 2.69
// ms, 1.6 PFLOP/s, gradient 8.0 to 8.4 ms, 1.53 to 1.61 (tiles of 128 x 256 a CTA, without the pair:
// 2.71 and 8.84); 128 rows against 131072 columns on 8 shards: 194 to 201 us, 5.3 to 5.5 TB/s (179 and 6.0
// with tiles of 128 x 256 and one run: a row of tiles has half of its rows to spare here, and
// shorter runs are read more often).
#include <algorithm>
#include <atomic>
#include <cstddef>

#include "dc_llm.h"
#include "dc_numeric.cuh"
#include "dc_tc.cuh"

namespace dc {
namespace {

using namespace tc;

enum : uint32_t { kSitePart = 1, kSiteRow = 2, kSiteD = 3, kSiteAcc = 4, kSiteOut = 5 };

__device__ unsigned int g_linear_fault_bits;

constexpr int kStages = 6;
constexpr int kTileBytes = 64 * 128;                  // 64 rows of 64 elements: what one TMA copy loads
constexpr int kHalfM = kLinearM / 2, kHalfN = kLinearN / 2;  // a CTA's rows of A and of B
constexpr int kABytes = kHalfM / 64 * kTileBytes, kBBytes = kHalfN / 64 * kTileBytes;
constexpr int kStageBytes = kABytes + kBBytes;        // of one CTA
constexpr int kSmem = kStages * kStageBytes + 1024;   // (the ring starts at a multiple of 1024)
// The tensor cores' sums lose more than a rounding a step (the error grows with
// their number, not its root).  The logits of the forward are therefore summed 512
// elements at a time, or 256 of hidden sizes up to 1024 (whose binary32 sums would be
// that good), and those sums added up, rounded, in registers.  Measured, 1543 rows of
// 4040 against 41592 columns, runs of 512 / 768 / 1024 elements: relative error of
// the log probabilities 1.7e-7 / 2.6e-7 / 3.5e-7 and the entropies 2.6e-7 / 3.9e-7 /
// 5.4e-7 (a binary32 matrix product: 3.3e-7, 3.1e-7); 4096 rows of 4096 against
// 128000: 2.66 / 2.60 / 2.57 ms, of 256: 2.96 ms.  4 rows of 512, runs of 512 / 256:
// entropies 5e-7 / 1.5e-7, 10.2 us either way.
constexpr uint32_t kRunBlocks = 8, kShortRunBlocks = 4, kShortBlocks = 16;
// The gradient's products are rounded to 16 bits afterwards: 24576 rows (or columns
// of a chunk) at a time.  Measured, FP16, dW of terms of one sign, 131072 / 2^20 rows,
// error against its last rounding's 2.1e-4: in one run 5.9e-4 / 4.5e-3.
constexpr uint32_t kGradBlocks = kLinearChunk / kLinearK;
constexpr int kResultThreads = 256;                   // eight warps of results: a row and half of the columns a thread
constexpr int kThreads = 64 + kResultThreads;         // one warp loads, one issues products
constexpr uint32_t kColumns = 2 * kLinearN;           // of tensor memory: two tiles' accumulators

template <int NB>
struct LinearArgs {
  CUtensorMap a, b[NB];
  LinearParams p;
  LinearShard shard[NB];
};

__device__ __forceinline__ int64_t token_of(uint64_t tokens, int tokens64, uint64_t row) {
  return tokens64 ? reinterpret_cast<const int64_t*>(tokens)[row] : reinterpret_cast<const int32_t*>(tokens)[row];
}
__device__ __forceinline__ float ld_row(uint64_t base, uint64_t row, uint64_t rows) {
  const float* a = reinterpret_cast<const float*>(base) + row;
  return in_bounds(a, 4, base, base + rows * 4, kSiteRow) ? *a : 0.0f;
}

// ------------------------------------------------------------- the results ---
// Each runs in a thread that has row `row` of C and kLinearPart columns of the
// tile's accumulators from `at` on in tensor memory.

// Forward: one row's part of a tile, its logits in v.  limit: the columns that exist.
__device__ __forceinline__ void stats(const LinearParams& p, float (&v)[kLinearPart], uint64_t row, uint32_t part, uint32_t column0,
                                      uint32_t limit) {
  const float c = p.inv_t * kLog2E;
  const int64_t mine = token_of(p.tokens, p.tokens64, row) - static_cast<int64_t>(column0);  // the token's column, if it is here
  if (limit < kLinearPart) {
#pragma unroll
    for (int j = 0; j < kLinearPart; ++j) v[j] = static_cast<uint32_t>(j) < limit ? v[j] : neg_inf();
  }
  if (mine >= 0 && mine < static_cast<int64_t>(limit)) {
    float z = 0.0f;
#pragma unroll
    for (int j = 0; j < kLinearPart; ++j) z = mine == j ? v[j] : z;
    float* a = reinterpret_cast<float*>(p.target) + row;
    if (in_bounds(a, 4, p.target, p.target + p.rows * 4, kSitePart)) *a = z;
  }
  float m[4] = {neg_inf(), neg_inf(), neg_inf(), neg_inf()};
#pragma unroll
  for (int j = 0; j < kLinearPart; j += 2) m[j / 2 & 3] = max3(m[j / 2 & 3], v[j], v[j + 1]);
  const float most = fmaxf(max3(m[0], m[1], m[2]), m[3]), top = most * c;
  // Exponents are taken from top, one fused multiply-add each, and what its rounding took
  // is put back into the sums; where that is more than a quarter (logits of millions, or
  // temperatures that make them so) from the logits' differences.
  float base = most == neg_inf() ? 0.0f : top, off = most == neg_inf() ? 0.0f : __fmaf_rn(most, c, -top);
  if (most != neg_inf() && !(fabsf(top) < 4194304.0f)) {
#pragma unroll
    for (int j = 0; j < kLinearPart; ++j) v[j] -= most;
    base = off = 0.0f;
  }
  float s[4] = {}, t[4] = {};
#pragma unroll
  for (int j = 0; j < kLinearPart; ++j) {
    const float x = __fmaf_rn(v[j], c, -base), e = ex2(x);
    s[j & 3] += e;
    t[j & 3] = __fmaf_rn(e, fmaxf(x, -1e4f), t[j & 3]);  // (e is 0 or NaN where that matters)
  }
  const float sum = (s[0] + s[1]) + (s[2] + s[3]), f = ex2(-off);
  float4* a = reinterpret_cast<float4*>(p.part) + static_cast<uint64_t>(part) * p.rows + row;
  if (in_bounds(a, 16, p.part, p.target, kSitePart))
    *a = make_float4(most, f * sum, f * __fmaf_rn(-off, sum, (t[0] + t[1]) + (t[2] + t[3])), 0.0f);
}

// Adds the tile's accumulators to v.
__device__ __forceinline__ void gather_part(uint32_t at, float (&v)[kLinearPart]) {
#pragma unroll
  for (int j0 = 0; j0 < kLinearPart; j0 += 16) {  // (16 at a time: v leaves room for no more)
    float x[16];
    tmem_ld16(at + j0, x);
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j0 + j] += x[j];
  }
}

// 32 bytes, to a multiple of 32.
__device__ __forceinline__ void st32(uint64_t at, const uint4& a, const uint4& b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(a.x), "r"(a.y), "r"(a.z), "r"(a.w),
               "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

// Stores 32 results of a row as 16-bit elements; `left` of them exist (a
// multiple of 8, or more than 32).
template <int DT>
__device__ __forceinline__ void st_row32(uint64_t at, const float (&v)[32], int left, uint64_t lo, uint64_t hi, uint32_t site) {
  uint4 w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float x[8] = {v[8 * j], v[8 * j + 1], v[8 * j + 2], v[8 * j + 3], v[8 * j + 4], v[8 * j + 5], v[8 * j + 6], v[8 * j + 7]};
    w[j] = repack<DT>(x);
  }
  if (left >= 32 && at % 32 == 0) {  // whole sectors of memory at a time
#pragma unroll
    for (int j = 0; j < 4; j += 2)
      if (in_bounds(reinterpret_cast<const void*>(at + j * 16), 32, lo, hi, site)) st32(at + j * 16, w[j], w[j + 1]);
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint4* a = reinterpret_cast<uint4*>(at + j * 16);
    if (8 * j < left && in_bounds(a, 16, lo, hi, site)) st16(a, w[j]);
  }
}

// Backward: the gradient of one row's logits in a tile.
template <int DT>
__device__ __forceinline__ void dlogits(const LinearParams& p, uint32_t at, uint64_t row, bool own, uint32_t n0) {
  float lse = 0.0f, a0 = 0.0f, a1 = 0.0f, hot = 0.0f;
  int64_t token = -1;
  bool none = false;  // a row without a finite logit, or without upstream gradients, has no gradient
  if (own) {
    token = token_of(p.tokens, p.tokens64, row);
    const float unit = p.scale ? *reinterpret_cast<const float*>(p.scale) : 1.0f;
    const float e = p.grad_entropy ? ld_row(p.grad_entropy, row, p.rows) : 0.0f;
    float g = p.grad_logprobs && token >= 0 ? ld_row(p.grad_logprobs, row, p.rows) : 0.0f;
    if (token >= static_cast<int64_t>(p.vocab) && (g != 0.0f || e != 0.0f)) g = __int_as_float(0x7FC00000);
    const float h = p.grad_entropy ? ld_row(p.entropy, row, p.rows) : 0.0f;
    lse = ld_row(p.lse, row, p.rows);
    const float f = p.inv_t * unit;
    hot = g * f;
    a0 = -(g + e * h) * f;   // d = p (a0 + a1 log2 p), and hot at the token
    a1 = -(e * kLn2) * f;
    none = lse <= -1e30f || (hot == 0.0f && a0 == 0.0f && a1 == 0.0f);
  }
  const int64_t column = token - static_cast<int64_t>(p.first) - n0;
  const uint32_t mine = column >= 0 && column < kLinearPart ? static_cast<uint32_t>(column) : kLinearPart;
  const uint32_t ld = static_cast<uint32_t>(p.d_stride / 2);
  const uint32_t exist = !none && p.vocab > p.first + n0 ? p.vocab - p.first - n0 : 0;  // columns before the padding
  const uint64_t lo = p.d + row * p.d_stride;
  if (n0 % kLinearN == 0) {
    const uint32_t marked = __ballot_sync(~0u, own && !none && column >= 0 && column < min(kLinearN, static_cast<int>(p.n - n0)));
    uint32_t* a = reinterpret_cast<uint32_t*>(p.marks) + static_cast<uint64_t>(n0 / kLinearN) * linear_groups(p.rows) + row / 32;
    if ((threadIdx.x & 31) == 0 && in_bounds(a, 4, p.marks, p.marks + linear_marks(p.rows, p.d_stride), kSiteRow)) *a = marked;
  }
#pragma unroll 1
  for (uint32_t j0 = 0; j0 < kLinearPart && n0 + j0 < ld; j0 += 32) {
    float v[32], exact = 0.0f;
    __syncwarp();
    tmem_ld32(at + j0, v);
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const float x = __fmaf_rn(v[j], p.inv_t, -lse) * kLog2E;
      v[j] = ex2(x) * __fmaf_rn(a1, x < -1e4f ? -1e4f : x, a0);
      if (j0 + j == mine) v[j] += hot;
      if (j0 + j >= exist) v[j] = 0.0f;
      if (j0 + j == mine) exact = v[j];
    }
    if (own && mine - j0 < 32) {
      const float off = exact - Elem<DT>::one(Elem<DT>::bits(exact));
      float* a = reinterpret_cast<float*>(p.lost) + row;
      if (in_bounds(a, 4, p.lost, p.lost + p.rows * 4, kSiteRow)) *a = fabsf(off) < -neg_inf() ? off : 0.0f;
    }
    if (own) st_row32<DT>(lo + (n0 + j0) * 2, v, static_cast<int>(ld - n0 - j0), lo, lo + p.d_stride, kSiteD);
  }
}

// What the rounding of d took from a row of a gradient.  dh: a factor times a row of
// the weights, its own token's.  dW: the same of the rows of the batch whose token this
// column is, in order, up to kLostAlone of them (or any of kLostFew rows in all), or one
// row of binary32 sums where there are more (dc_linear_lost_kernel).
struct Lost {
  float f[2];
  uint64_t row[2];  // 0: none
  uint4 w[8];       // 32 elements of each, or 32 sums
  uint32_t hits;
  bool sum;
};
// The rows' numbers for a warp's 32 columns: of kLostFew rows in all a byte each.
union LostList {
  uint32_t some[32][kLostAlone];
  uint8_t few[32][kLostFew];
};

// 32 elements of a row of `size`, from `first` on, of 16 bits (4 vectors) or 32 (8).
template <int BYTES>
__device__ __forceinline__ void ld_row32(uint4* w, uint64_t row, uint32_t first, uint32_t size) {
  constexpr uint32_t kPer = 16 / BYTES;
#pragma unroll
  for (uint32_t j = 0; j < 2 * BYTES; ++j) {
    const uint4* a = reinterpret_cast<const uint4*>(row + static_cast<uint64_t>(first) * BYTES) + j;
    w[j] = row && first + kPer * j < size && in_bounds(a, 16, row, row + static_cast<uint64_t>(size) * BYTES, kSiteRow) ? *a : make_uint4(0, 0, 0, 0);
  }
}
__device__ __forceinline__ void ld_lost(Lost& x, uint32_t first, uint32_t size) {
  if (x.sum) {
    ld_row32<4>(x.w, x.row[0], first, size);
  } else {
    ld_row32<2>(x.w, x.row[0], first, size);
    ld_row32<2>(x.w + 4, x.row[1], first, size);
  }
}
template <int DT>
__device__ __forceinline__ void add_lost(float (&v)[32], const Lost& x) {
  if (x.sum) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[4 * j] += __uint_as_float(x.w[j].x);
      v[4 * j + 1] += __uint_as_float(x.w[j].y);
      v[4 * j + 2] += __uint_as_float(x.w[j].z);
      v[4 * j + 3] += __uint_as_float(x.w[j].w);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (x.f[i] == 0.0f) continue;  // (whatever the row holds)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float y[8];
      unpack<DT>(x.w[4 * i + j], y);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[8 * j + k] = __fmaf_rn(x.f[i], y[k], v[8 * j + k]);
    }
  }
}
// The lane's rows k and k + 1 of the list.
__device__ __forceinline__ void lost_pair(const LinearParams& p, Lost& x, uint32_t k, const LostList& list) {
  const uint32_t lane = threadIdx.x & 31;
#pragma unroll
  for (uint32_t i = 0; i < 2; ++i) {
    const bool there = k + i < x.hits;
    const uint64_t row = !there ? 0 : p.rows <= kLostFew ? list.few[lane][k + i] : list.some[lane][k + i];
    x.f[i] = there ? ld_row(p.lost, row, p.rows) : 0.0f;
    x.row[i] = there ? p.g.x + row * p.g.x_stride : 0;
  }
}

// Looked up before the products are there: `row` of C, k0 and blocks of dh's inner dimension.
__device__ __forceinline__ void look_up(const LinearParams& p, uint64_t row, bool own, uint32_t n0, bool weights, uint32_t k0,
                                        uint32_t blocks, LostList& list, Lost* x) {
  const LinearGrads& g = p.g;
  const uint32_t lane = threadIdx.x & 31;
  *x = Lost{};
  if (!weights) {
    if (own) {
      const int64_t column = token_of(p.tokens, p.tokens64, row) - static_cast<int64_t>(p.first);
      if (column >= k0 && column < min(g.columns, k0 + blocks * kLinearK)) {
        x->f[0] = ld_row(p.lost, row, p.rows);
        x->row[0] = x->f[0] != 0.0f ? g.w + static_cast<uint64_t>(column) * g.w_stride : 0;
      }
    }
    x->hits = x->row[0] != 0;
  } else if (p.rows <= kLostFew) {
    for (uint32_t r0 = 0; r0 < p.rows; r0 += 32) {
      const int64_t t = r0 + lane < p.rows ? token_of(p.tokens, p.tokens64, r0 + lane) - static_cast<int64_t>(p.first) : -1;
      for (uint32_t k = 0; k < min(32u, static_cast<uint32_t>(p.rows) - r0); ++k)
        if (__shfl_sync(~0u, t, k) == static_cast<int64_t>(row) && own) list.few[lane][x->hits++] = static_cast<uint8_t>(r0 + k);
    }
  } else if (own) {
    const int32_t* a = reinterpret_cast<const int32_t*>(g.table) + row;
    int32_t at = in_bounds(a, 4, g.table, g.table + g.columns * 4ull, kSiteRow) ? *a : -1;
    if (at < -1) {
      x->sum = true;
      x->row[0] = g.sums + static_cast<uint64_t>(-2 - at) * p.n * 4;
      x->hits = 1;
    }
    while (at >= 0 && x->hits < kLostAlone) {
      list.some[lane][x->hits++] = static_cast<uint32_t>(at);
      a = reinterpret_cast<const int32_t*>(g.next) + at;
      at = in_bounds(a, 4, g.next, g.next + p.rows * 4, kSiteRow) ? *a : -1;
    }
  }
  if (weights && !x->sum) lost_pair(p, *x, 0, list);
  if (x->hits) ld_lost(*x, n0, p.n);
}

// A row of a gradient.  Plus what `acc` (dh: of chunks and slices, dW: of this
// tile's runs) holds of it, to `acc` or (complete) to the output.
template <int DT>
__device__ __forceinline__ void result(const LinearParams& p, uint32_t at, uint64_t row, bool own, uint32_t n0, bool weights,
                                       uint32_t slice, bool empty, bool again, bool whole, Lost& lost, const LostList& list) {
  const LinearGrads& g = p.g;
  const float unit = p.scale ? reinterpret_cast<const float*>(p.scale)[1] : 1.0f;
  const uint64_t out = weights ? g.out_w + row * g.out_w_stride : g.out_h + row * g.out_h_stride;
  const uint64_t tile = static_cast<uint64_t>(kLinearM) * kLinearN * 4;
  const uint64_t acc_lo = weights ? g.tile + blockIdx.x / 2 * tile : g.acc + static_cast<uint64_t>(slice) * p.rows * p.n * 4;
  const uint64_t acc_hi = acc_lo + (weights ? tile : p.rows * p.n * 4);
  const uint64_t acc_row = weights ? row % kLinearM * kLinearN + n0 % kLinearN : row * p.n + n0;
  const bool sums = !weights && g.acc, add = weights ? again : sums && g.add, last = weights ? whole : !sums || g.last;
#pragma unroll 1
  for (uint32_t j0 = 0; j0 < kLinearPart && n0 + j0 < p.n; j0 += 32) {
    float v[32];
    __syncwarp();
    tmem_ld32(at + j0, v);
    const int left = static_cast<int>(min(p.n - n0 - j0, 32u));
    if (empty) {  // (a slice behind the last column: nothing was multiplied)
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = 0.0f;
    }
    if (lost.hits && (last || !weights)) {  // (dW: with the last run)
      add_lost<DT>(v, lost);
      for (uint32_t k = 2; k < lost.hits; k += 2) {
        lost_pair(p, lost, k, list);
        ld_lost(lost, n0 + j0, p.n);
        add_lost<DT>(v, lost);
      }
      if (lost.hits > 2) lost_pair(p, lost, 0, list);
      if (j0 + 32 < kLinearPart) ld_lost(lost, n0 + j0 + 32, p.n);  // (for the next columns)
    }
    if (!own) continue;
    float4* a = reinterpret_cast<float4*>(acc_lo) + (acc_row + j0) / 4;
    if (add) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (4 * j < left && in_bounds(a + j, 16, acc_lo, acc_hi, kSiteAcc)) {
          const float4 x = a[j];
          v[4 * j] += x.x;
          v[4 * j + 1] += x.y;
          v[4 * j + 2] += x.z;
          v[4 * j + 3] += x.w;
        }
    }
    if (!last) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (4 * j < left && in_bounds(a + j, 16, acc_lo, acc_hi, kSiteAcc))
          a[j] = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
      continue;
    }
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] *= unit;
    st_row32<DT>(out + (n0 + j0) * 2, v, left, out, out + p.n * 2ull, kSiteOut);
  }
}

// Tile t of fast x slow, in bands of `band` of the first, so that the tiles that run at
// the same time share their operands and a band's stay in L2.  Bands of 16 rows of
// tiles for the logits, of 8 for dh, of 8 columns for dW.  Measured, BF16, against all
// rows first (dW: all of the vocabulary first): 4096 rows of 4096 and 128000 columns,
// gradient 8.67 -> 8.03 ms; 16384 rows and 64000 columns, forward 5.15 -> 4.62 (1.86
// PFLOP/s), gradient 17.2 -> 15.0 ms (1.72).  Bands of 8 for the logits cost that
// forward nothing and 4096 rows 3 %; of 16 for dh and dW: 8.11 and 15.4 ms.
struct Spot {
  uint32_t fast, slow;
};
__device__ __forceinline__ Spot spot(uint32_t t, uint32_t fast, uint32_t slow, uint32_t band) {
  const uint32_t b = t / (band * slow), r = t - b * (band * slow), w = max(1u, min(band, fast - b * band));
  return {b * band + r % w, r / w};
}
constexpr uint32_t kLogitBand = 16, kGradBand = 8;

// What a CTA has to tell its pair before both may leave.
struct Leave {
  uint32_t told;            // the other has given up
  uint32_t filled;          // stages that this CTA's loader filled
  uint32_t used, runs;      // (even CTA) stages that products read, and sums of them
};

// A wait of the pair has run out.  Every thread of both CTAs has stopped; their copies
// and products in flight are waited for, and the arrivals that those bring.  A stage's
// barrier is told by both CTAs' copies: where one loader was ahead, what the other
// would have copied or announced is made up for.
__device__ __noinline__ void give_up(const Leave* leave, uint32_t rank, uint32_t full, uint32_t empty, uint32_t done, uint32_t over) {
  const uint32_t at = smem_addr(leave);
  bool ended = true;
  auto drain = [&](uint32_t bar, uint32_t parity) { ended = tma::mbar_wait_bounded(bar, parity, kDrainNs) && ended; };
  if (threadIdx.x == 32) {  // (the thread that issued the products)
    if (rank == 0) commit_pair(over);
    drain(over, 0);
    const uint32_t even = cluster_addr(at, 0);
    const uint32_t used = ld_cluster(even + offsetof(Leave, used)), runs = ld_cluster(even + offsetof(Leave, runs));
    for (uint32_t k = used > kStages ? used - kStages : 0; k < used; ++k) drain(empty + 8 * (k % kStages), (k / kStages) & 1);
    for (uint32_t k = runs > 2 ? runs - 2 : 0; k < runs; ++k) drain(done + 8 * (k & 1), (k / 2) & 1);
  }
  if (threadIdx.x == 0 && rank == 0) {
    const uint32_t mine = leave->filled, other = ld_cluster(cluster_addr(at, 1) + offsetof(Leave, filled));
    const uint32_t both = min(mine, other), end = max(mine, other);
    for (uint32_t k = both; k < end; ++k) {
      const uint32_t bar = full + 8 * (k % kStages);
      if (k < mine) tma::mbar_complete_tx(bar, kStageBytes);
      else tma::mbar_arrive_expect_tx(bar, kStageBytes);
    }
    for (uint32_t k = end > kStages ? end - kStages : 0; k < end; ++k) drain(full + 8 * (k % kStages), (k / kStages) & 1);
  }
  if (!ended) atomicOr(&g_linear_fault_bits, kFaultTensorDrain);
  __syncwarp();
  cluster_barrier();
}

template <int MODE, int DT, int NB>
__global__ __launch_bounds__(kThreads, 1) void dc_linear_kernel(const __grid_constant__ LinearArgs<NB> args) {
  // whether B's rows run across the inner dimension (A's do for dW)
  constexpr bool kAcrossB = MODE == kLinearGrads;
  const LinearParams& p = args.p;
  // blocks of the inner dimension that the tensor cores sum
  const uint32_t run = MODE == kLinearStats ? p.run : MODE == kLinearGrads ? kGradBlocks : 1u << 30;
  extern __shared__ uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[2 * kStages + 5];
  __shared__ uint32_t tmem_at;
  __shared__ volatile uint32_t stop;
  __shared__ Leave leave;
  __shared__ LostList lists[MODE == kLinearGrads ? kResultThreads / 32 : 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ring = (smem_addr(smem) + 1023u) & ~1023u;
  const uint32_t full = smem_addr(bars), empty = full + 8 * kStages;
  const uint32_t done = empty + 8 * kStages, drained = done + 16, over = drained + 16;
  const uint32_t rank = cluster_rank();
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      tma::mbar_init(full + 8 * i, 1);
      tma::mbar_init(empty + 8 * i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      tma::mbar_init(done + 8 * i, 1);
      tma::mbar_init(drained + 8 * i, 2 * kResultThreads / 32);
    }
    tma::mbar_init(over, 1);
    tma::mbar_init_fence();
    stop = 0;
    leave = Leave{};
    prefetch_map(&args.a);
    prefetch_map(&args.b[0]);
  }
  __syncwarp();
  if (warp == 1) tmem_alloc_pair(smem_addr(&tmem_at), kColumns);
  fence_before();
  __syncthreads();
  cluster_barrier();  // (each CTA's barriers are used by the other)
  fence_after();
  const uint32_t tmem = tmem_at;
  pdl_enter();
  tma::fence_proxy_async_global();  // (the operands may be an earlier kernel's stores)

  const Waits waits{&stop, p.wait_ns};
  // This pair's n-th tile: its rows, its columns, the tensor that those belong to,
  // its blocks of the inner dimension.
  struct Place {
    uint32_t m0, n0, k0, blocks;
    uint32_t tile;    // kLinearStats: of columns; kLinearGrads: slice
    int r;            // kLinearStats: shard; kLinearGrads: 0 dh, 1 dW
    bool there;
  };
  auto place = [&](uint32_t n) {
    Place x{0, 0, 0, p.k_blocks, 0, 0, true};
    const uint32_t c = blockIdx.x / 2, G = gridDim.x / 2;
    if constexpr (MODE == kLinearGrads) {
      const LinearGrads& g = p.g;
      const uint32_t mine = g.rounds + (c < g.rest);
      if (n < mine) {
        const uint32_t t = c + n * G, s = t / (g.h_m * g.h_n);
        const Spot at = spot(t - s * (g.h_m * g.h_n), g.h_m, g.h_n, kGradBand);
        x.m0 = at.fast * kLinearM;
        x.n0 = at.slow * kLinearN;
        x.k0 = s * g.slice_blocks;
        x.blocks = min(g.slice_blocks, g.h_blocks > x.k0 ? g.h_blocks - x.k0 : 0u);
        x.tile = s;
      } else {
        const uint32_t k = n - mine, t = k < g.few ? k * G + c : g.few * G + (k - g.few) * (G - g.rest) + c - g.rest;
        x.there = (k < g.few || (c >= g.rest && k < g.many)) && t < g.w_tiles;
        const Spot at = spot(t, g.h_n, g.w_m, kGradBand);
        x.m0 = at.slow * kLinearM;
        x.n0 = at.fast * kLinearN;
        x.blocks = g.w_blocks;
        x.r = 1;
      }
    } else {
      const uint64_t t = c + static_cast<uint64_t>(n) * G;
      x.there = t < static_cast<uint64_t>(p.m_tiles) * p.n_tiles;
      const Spot at = spot(static_cast<uint32_t>(t), p.m_tiles, p.n_tiles, kLogitBand);
      x.m0 = at.fast * kLinearM;
      x.n0 = x.tile = at.slow;
      if constexpr (MODE == kLinearStats) {
        if constexpr (NB > 1)
          while (x.r + 1 < p.shards && args.shard[x.r + 1].tile0 <= x.n0) ++x.r;
        x.n0 -= args.shard[x.r].tile0;
      }
      x.n0 *= kLinearN;
    }
    return x;
  };

  if (warp == 0) {
    if (lane == 0) {
      uint32_t i = 0;  // stages filled so far
      for (uint32_t n = 0; !stop; ++n) {
        const Place x = place(n);
        if (!x.there) break;
        const bool across_a = MODE == kLinearGrads && x.r == 1;
        // (dh: the weights' rows are the inner dimension; the logits: they are the columns)
        const int32_t off = static_cast<int32_t>(MODE == kLinearGrads && x.r == 1 ? 0 : p.b_row0);
        for (uint32_t kb = 0; kb < x.blocks; ++kb, ++i) {
          const uint32_t st = i % kStages, bar = full + 8 * st, to = ring + st * kStageBytes;
          if (i >= kStages && !wait(waits, empty + 8 * st, (i / kStages - 1) & 1)) break;
          if (i == 2 && p.late == static_cast<int32_t>(3 + rank)) {
            come_late(p.wait_ns);
            if (stop) break;
          }
          // (the products wait at the even CTA, for both CTAs' operands)
          if (rank == 0) tma::mbar_arrive_expect_tx(bar, 2 * kStageBytes);
          const uint32_t told = cluster_addr(bar, 0);
          const int32_t k0 = static_cast<int32_t>((x.k0 + kb) * kLinearK);
#pragma unroll
          for (int j = 0; j < kHalfM / 64; ++j) {
            const int32_t mj = static_cast<int32_t>(x.m0 + rank * kHalfM) + 64 * j;
            load_tile_pair(to + j * kTileBytes, &args.a, told, across_a ? mj : k0, across_a ? k0 : mj);
          }
#pragma unroll
          for (int j = 0; j < kHalfN / 64; ++j) {
            const int32_t nj = static_cast<int32_t>(x.n0 + rank * kHalfN) + 64 * j;
            load_tile_pair(to + kABytes + j * kTileBytes, &args.b[NB > 1 ? x.r : 0], told, kAcrossB ? nj : k0,
                           kAcrossB ? k0 + off : nj + off);
          }
        }
      }
      leave.filled = i;
      // (the even CTA's products tell this barrier too: it may go when they have)
      for (uint32_t k = i > kStages ? i - kStages : 0; k < i && !stop; ++k) wait(waits, empty + 8 * (k % kStages), (k / kStages) & 1);
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      uint32_t i = 0, runs = 0;  // stages used, and runs of them that were summed, so far
      for (uint32_t n = 0; !stop; ++n) {
        const Place x = place(n);
        if (!x.there) break;
        const bool across_a = MODE == kLinearGrads && x.r == 1;
        const uint32_t idesc = instruction<DT>(kLinearM, kLinearN, (across_a ? kMajorA : 0u) | (kAcrossB ? kMajorB : 0u));
        uint32_t kb = 0;
        do {
          const uint32_t buf = runs & 1, acc = tmem + buf * kLinearN;
          const uint32_t from = kb, to = min(kb + run, x.blocks);
          if (runs >= 2 && !wait(waits, drained + 8 * buf, (runs / 2 - 1) & 1)) break;
          fence_after();
          for (; kb < to; ++kb, ++i) {
            const uint32_t st = i % kStages, a = ring + st * kStageBytes, b = a + kABytes;
            if (!wait(waits, full + 8 * st, (i / kStages) & 1)) break;
            fence_after();
#pragma unroll
            for (int k = 0; k < kLinearK / 16; ++k)
              mma_pair(acc, across_a ? desc_mn(a + k * 2048, kTileBytes) : desc_k(a + k * 32),
                       kAcrossB ? desc_mn(b + k * 2048, kTileBytes) : desc_k(b + k * 32), idesc, (kb - from | k) != 0);
            commit_pair(empty + 8 * st);
          }
          commit_pair(done + 8 * buf);
          ++runs;
        } while (kb < x.blocks && !stop);
      }
      leave.used = i;
      leave.runs = runs;
    }
  } else {
    // the lanes of tensor memory that this warp reads, and which half of the columns
    const uint32_t quarter = static_cast<uint32_t>(warp & 3) * 32, half = static_cast<uint32_t>(warp - 2) / 4;
    uint32_t runs = 0;
    bool there = true;
    for (uint32_t n = 0; there; ++n) {
      const Place x = place(n);
      if (!x.there) break;
      const uint32_t row0 = x.m0 + rank * kHalfM + quarter, n0 = x.n0 + half * kLinearPart;
      const uint64_t row = row0 + lane;
      const uint32_t rows = MODE == kLinearGrads && x.r == 1 ? p.g.columns : p.m;
      const bool own = row < rows;
      [[maybe_unused]] float v[MODE == kLinearStats ? kLinearPart : 1] = {};
      [[maybe_unused]] Lost lost;
      if constexpr (MODE == kLinearGrads)
        if (row0 < rows) look_up(p, row, own, n0, x.r == 1, x.k0 * kLinearK, x.blocks, lists[warp - 2], &lost);
      uint32_t kb = 0;
      do {
        const uint32_t buf = runs & 1, at = tmem + buf * kLinearN + half * kLinearPart + (quarter << 16);
        there = __all_sync(~0u, wait(waits, done + 8 * buf, (runs / 2) & 1));
        if (!there) break;
        fence_after();
        if (p.late == static_cast<int32_t>(1 + rank) && runs == 0) come_late(p.wait_ns);
        if (row0 < rows) {
          if constexpr (MODE == kLinearStats) gather_part(at, v);
          else if constexpr (MODE == kLinearDLogits) dlogits<DT>(p, at, row, own, n0);
          else result<DT>(p, at, row, own, n0, x.r == 1, x.tile, x.blocks == 0, kb > 0, kb + run >= x.blocks, lost, lists[warp - 2]);
        }
        fence_before();
        __syncwarp();
        if (lane == 0) arrive_cluster(cluster_addr(drained + 8 * buf, 0));  // (of every thread, 512 of them took longer than the reading)
        ++runs;
        kb += run;
      } while (kb < x.blocks);
      if constexpr (MODE == kLinearStats) {
        const LinearShard& s = args.shard[NB > 1 ? x.r : 0];
        const uint32_t column0 = s.first + n0;
        if (there && own)
          stats(p, v, row, 2 * x.tile + half, column0, column0 < s.end ? min(s.end - column0, static_cast<uint32_t>(kLinearPart)) : 0u);
      }
    }
  }
  __syncwarp();
  __syncthreads();
  if (threadIdx.x == 0 && stop) {
    atomicOr(&g_linear_fault_bits, kFaultTensorWait);
    st_cluster(cluster_addr(smem_addr(&leave.told), rank ^ 1), 1);
  }
  fence_before();
  cluster_barrier();  // no CTA leaves while the other's products read its shared memory, or its barriers are told
  if (stop || *const_cast<volatile uint32_t*>(&leave.told)) give_up(&leave, rank, full, empty, done, over);
  fence_after();
  if (warp == 1) tmem_free_pair(tmem, kColumns);
}

// A CTA adds a row's parts up: thread t takes parts t, t + 128, ..., then the lanes
// join in pairs and the warps in order.
constexpr int kFinishThreads = 128;
__global__ __launch_bounds__(kFinishThreads) void dc_linear_finish_kernel(const __grid_constant__ LinearFinishParams p) {
  pdl_enter();
  __shared__ float4 joined[kFinishThreads / 32];
  const uint64_t row = blockIdx.x;
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float ref = neg_inf(), s = 0.0f, t = 0.0f;
  const float c = p.inv_t * kLog2E;
  auto add = [&](float r, float s1, float t1) {
    // t = sum 2^(z-ref) (z-ref): moving ref by k adds k times the sum (2^-10000 is 0, and NaN is in the sums)
    const float m = fmaxf(ref, r);
    const float k0 = ref == neg_inf() ? 0.0f : fmaxf((ref - m) * c, -1e4f), k1 = r == neg_inf() ? 0.0f : fmaxf((r - m) * c, -1e4f);
    const float f0 = ex2(k0), f1 = ex2(k1);
    t = __fmaf_rn(f0, __fmaf_rn(s, k0, t), f1 * __fmaf_rn(s1, k1, t1));
    s = __fmaf_rn(f0, s, f1 * s1);
    ref = m;
  };
  constexpr int kAtOnce = 4;
  for (uint32_t i0 = threadIdx.x; i0 < p.parts; i0 += kAtOnce * kFinishThreads) {
    float4 x[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const uint32_t i = i0 + k * kFinishThreads;
      const float4* a = reinterpret_cast<const float4*>(p.part) + static_cast<uint64_t>(i) * p.rows + row;
      x[k] = i < p.parts && in_bounds(a, 16, p.part, p.part + static_cast<uint64_t>(p.parts) * p.rows * 16, kSitePart)
                 ? *a : make_float4(neg_inf(), 0.0f, 0.0f, 0.0f);
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k)
      if (i0 + k * kFinishThreads < p.parts) add(x[k].x, x[k].y, x[k].z);
  }
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const float r1 = __shfl_xor_sync(~0u, ref, d), s1 = __shfl_xor_sync(~0u, s, d), t1 = __shfl_xor_sync(~0u, t, d);
    add(r1, s1, t1);
  }
  if (lane == 0) joined[warp] = make_float4(ref, s, t, 0.0f);
  __syncthreads();
  if (threadIdx.x) return;
  for (int w = 1; w < kFinishThreads / 32; ++w) add(joined[w].x, joined[w].y, joined[w].z);
  const bool none = ref == neg_inf() && s == 0.0f;  // nothing but -inf
  const float log_2 = log2f(s), log_s = log_2 * kLn2, nan = __int_as_float(0x7FC00000);
  const int64_t token = token_of(p.tokens, p.tokens64, row);
  auto put = [&](uint64_t base, float v) {
    float* a = reinterpret_cast<float*>(base) + row;
    if (in_bounds(a, 4, base, base + p.rows * 4, kSiteOut)) *a = v;
  };
  float lp = 0.0f;
  if (token >= static_cast<int64_t>(p.vocab)) lp = nan;
  else if (token >= 0) lp = none ? neg_inf() : __fmaf_rn(ld_row(p.target, row, p.rows) - ref, p.inv_t, -log_s);
  put(p.logprobs, lp);
  if (p.entropy) put(p.entropy, none ? 0.0f : (log_2 - t / s) * kLn2);
  if (p.lse) put(p.lse, none ? neg_inf() : __fmaf_rn(ref, p.inv_t, log_s));
}

// Where dW's columns find what d lost of the rows whose token they are, for calls of
// more than kLostFew rows: a column of up to kLostAlone such rows the first of them, each
// row the next (in order), and a column of more the sum, in binary32, of what d lost times
// the hidden rows.  So no tile's results take longer the more rows share a token.
// A CTA has 256 columns (the marks say which rows have their token there) and every
// gridDim.y-th 256 elements of the hidden rows.  kLostRows rows at a time are put in order
// by column and, in one, the rows' order; the CTA's warps sum a column's rows and join in
// order.
// Measured, BF16, 16384 rows of 4096 against 64000 columns, tokens spread evenly / half of
// the rows one token's / as often as the n-th word of a text: 16.3 / 16.5 / 16.9 ms (all of
// it by the tile's own warps: 15.5 / 30.9 / 18.0 to 21.5); 509 rows of 1000 against 50021:
// 208 / 235 / 242 us (200 / 534 / 284).  13 and 5 us a chunk of columns.
constexpr int kLostThreads = 256, kLostWarps = kLostThreads / 32;
constexpr uint32_t kLostRows = 4096, kLostWords = kLostRows / 32;
constexpr uint32_t kLostAtOnce = 8;  // rows whose loads a warp has in flight

// Exclusive sums over the CTA; every thread gets the total.
__device__ __forceinline__ uint32_t scan_cta(uint32_t n, uint32_t* warps, uint32_t* total) {
  const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t s = n;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const uint32_t t = __shfl_up_sync(~0u, s, d);
    if (lane >= static_cast<uint32_t>(d)) s += t;
  }
  __syncthreads();  // (warps: of the call before)
  if (lane == 31) warps[warp] = s;
  __syncthreads();
  uint32_t before = 0, all = 0;
#pragma unroll
  for (uint32_t w = 0; w < kLostWarps; ++w) {
    before += w < warp ? warps[w] : 0u;
    all += warps[w];
  }
  *total = all;
  return before + s - n;
}

template <int DT>
__global__ __launch_bounds__(kLostThreads) void dc_linear_lost_kernel(const __grid_constant__ LinearLostParams p) {
  static_assert(kLostThreads == kLinearN, "a thread a column");
  pdl_enter();
  __shared__ uint32_t hits[kLostRows];    // the marked rows: row of these kLostRows, column (8 bits)
  __shared__ uint16_t order[kLostRows];   // their rows, by column
  __shared__ float joined[kLostWarps][kLinearN];
  __shared__ uint32_t count[kLinearN], start[kLinearN], warps[kLostWarps];
  __shared__ int32_t place[kLinearN];     // of a column's sum, -1: it has none yet
  __shared__ uint16_t many[kLinearN];     // the columns that have sums
  const uint32_t t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const uint32_t column0 = blockIdx.x * kLinearN, groups = linear_groups(p.rows);
  const uint64_t marks = p.marks + static_cast<uint64_t>(blockIdx.x) * groups * 4, marks_hi = marks + groups * 4ull;
  const int64_t first = static_cast<int64_t>(p.first) + column0;
  auto mark = [&](uint32_t g) {
    const uint32_t* a = reinterpret_cast<const uint32_t*>(marks) + g;
    return g < groups && in_bounds(a, 4, marks, marks_hi, kSiteRow) ? *a : 0u;
  };
  // (a mark says that the row's token is one of these)
  auto column_of = [&](uint64_t row) { return static_cast<uint32_t>(token_of(p.tokens, p.tokens64, row) - first) & (kLinearN - 1); };

  // which columns have sums: how many rows each has, counted first where those come in parts
  const bool links = blockIdx.y == 0, parts = groups > kLostWords;
  bool shared = false;
  uint32_t n_many = 0;
  auto decide = [&](uint32_t rows) {
    shared = rows > kLostAlone;
    const uint32_t at = scan_cta(shared, warps, &n_many);
    if (shared) many[at] = static_cast<uint16_t>(t);
  };
  count[t] = 0;
  place[t] = -1;
  if (parts) {
    __syncthreads();
    for (uint32_t g0 = warp * 32; g0 < groups; g0 += kLostThreads) {
      const uint32_t word = mark(g0 + lane);
      uint32_t some = __ballot_sync(~0u, word != 0);
      while (some) {
        constexpr int kWords = 4;
        uint32_t column[kWords];
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
          const uint32_t at = some ? static_cast<uint32_t>(__ffs(static_cast<int>(some)) - 1) : 0u;
          const uint32_t bits = __shfl_sync(~0u, word, static_cast<int>(at));
          column[k] = some && (bits >> lane & 1) ? column_of(32ull * (g0 + at) + lane) : static_cast<uint32_t>(kLinearN);
          some &= some - 1;
        }
#pragma unroll
        for (int k = 0; k < kWords; ++k)
          if (column[k] < kLinearN) atomicAdd(&count[column[k]], 1u);
      }
    }
    __syncthreads();
    decide(count[t]);
    if (!links && n_many == 0) return;
  }

  int32_t head = -1, last = -1;  // this thread's column's first row, and the last so far
  for (uint32_t g0 = 0; g0 < groups; g0 += kLostWords) {
    const uint32_t row0 = 32 * g0;
    uint32_t word = t < kLostWords ? mark(g0 + t) : 0u, n, all;
    uint32_t at = scan_cta(static_cast<uint32_t>(__popc(word)), warps, &n);
    if (n == 0) continue;
    count[t] = 0;
    for (; word; word &= word - 1) hits[at++] = 32 * t + static_cast<uint32_t>(__ffs(static_cast<int>(word)) - 1);
    __syncthreads();
    for (uint32_t k = t; k < n; k += kLostThreads) {
      const uint32_t column = column_of(row0 + hits[k]);
      hits[k] = hits[k] << 8 | column;
      atomicAdd(&count[column], 1u);
    }
    __syncthreads();
    const uint32_t mine = count[t];
    if (!parts) {
      decide(mine);
      if (!links && n_many == 0) return;
    }
    at = scan_cta(mine, warps, &all);
    start[t] = at;
    for (uint32_t k = 0, left = mine; left && k < n; ++k) {  // (all threads read the same one)
      if ((hits[k] & 255) != t) continue;
      const uint32_t r = hits[k] >> 8;
      order[at++] = static_cast<uint16_t>(r);
      --left;
      const int32_t row = static_cast<int32_t>(row0 + r);
      if (head < 0) head = row;
      else if (links && !shared) {
        int32_t* a = reinterpret_cast<int32_t*>(p.next) + last;
        if (in_bounds(a, 4, p.next, p.next + p.rows * 4, kSitePart)) *a = row;
      }
      last = row;
    }
    __syncthreads();
    // (the next scan waits for all threads before anything of this is written again)
    for (uint32_t s = blockIdx.y; n_many && s * kLinearN < p.size; s += gridDim.y) {
      const uint32_t e0 = s * kLinearN + lane * 8;
      for (uint32_t i = 0; i < n_many; ++i) {
        const uint32_t column = many[i], rows = count[column];
        if (rows == 0) continue;
        float acc[8] = {};
        for (uint32_t k0 = warp * kLostAtOnce; k0 < rows; k0 += kLostWarps * kLostAtOnce) {
          float f[kLostAtOnce];
          uint4 x[kLostAtOnce];
#pragma unroll
          for (uint32_t j = 0; j < kLostAtOnce; ++j) {
            const bool there = k0 + j < rows;
            const uint64_t row = row0 + order[start[column] + (there ? k0 + j : k0)], from = p.x + row * p.x_stride;
            const uint4* a = reinterpret_cast<const uint4*>(from + e0 * 2ull);
            f[j] = there ? ld_row(p.lost, row, p.rows) : 0.0f;
            x[j] = there && e0 < p.size && in_bounds(a, 16, from, from + p.size * 2ull, kSiteRow) ? *a : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (uint32_t j = 0; j < kLostAtOnce; ++j) {
            float y[8];
            unpack<DT>(x[j], y);
#pragma unroll
            for (int v = 0; v < 8; ++v) acc[v] = __fmaf_rn(f[j], y[v], acc[v]);
          }
        }
        float4* to = reinterpret_cast<float4*>(&joined[warp][lane * 8]);
        to[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        to[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
        __syncthreads();
        const uint32_t e = s * kLinearN + t;
        // one place for each column, whatever the order: its first row's, or its own, of which there are fewer
        const int32_t old = place[column], now = old >= 0 ? old : static_cast<int32_t>(p.by_row ? row0 + order[start[column]] : column0 + column);
        float* a = reinterpret_cast<float*>(p.sums) + static_cast<uint64_t>(now) * p.size + e;
        if (e < p.size && in_bounds(a, 4, p.sums, p.sums + p.places * p.size * 4, kSiteAcc)) {
          float sum = joined[0][t];
          for (int w = 1; w < kLostWarps; ++w) sum += joined[w][t];
          *a = old >= 0 ? *a + sum : sum;
        }
        __syncthreads();
      }
    }
    __syncthreads();
    if (shared && mine && place[t] < 0) place[t] = p.by_row ? head : static_cast<int32_t>(column0 + t);
  }
  if (!links) return;
  if (head >= 0 && !shared) {
    int32_t* a = reinterpret_cast<int32_t*>(p.next) + last;
    if (in_bounds(a, 4, p.next, p.next + p.rows * 4, kSitePart)) *a = -1;
  }
  int32_t* a = reinterpret_cast<int32_t*>(p.table) + column0 + t;
  if (in_bounds(a, 4, p.table, p.table + p.d_stride * 2, kSitePart)) *a = shared ? -2 - place[t] : head;
}

template <int DT>
__global__ __launch_bounds__(256) void dc_linear_sum_kernel(const __grid_constant__ LinearSumParams p) {
  pdl_enter();
  const uint64_t per = p.size / 8, item = static_cast<uint64_t>(blockIdx.x) * 256 + threadIdx.x, row = item / per;
  if (row >= p.rows) return;
  const uint32_t c = static_cast<uint32_t>(item % per) * 8;
  const float unit = p.scale ? reinterpret_cast<const float*>(p.scale)[1] : 1.0f;
  const uint64_t slice = p.rows * p.size * 4, hi = p.acc + p.slices * slice;
  float v[8] = {};
#pragma unroll 4
  for (uint32_t s = 0; s < p.slices; ++s) {
    const float4* a = reinterpret_cast<const float4*>(p.acc + s * slice + (row * p.size + c) * 4);
    if (!in_bounds(a, 32, p.acc, hi, kSiteAcc)) continue;
    const float4 x = a[0], y = a[1];
    const float w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] += w[j];
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] *= unit;
  const uint64_t out = p.out + row * p.out_stride;
  uint4* a = reinterpret_cast<uint4*>(out + c * 2);
  if (in_bounds(a, 16, out, out + p.size * 2ull, kSiteOut)) st16(a, repack<DT>(v));
}

// The power of two for DC_F16: no |d_j| is above (|g| + 16 |e|) / temperature,
// as p |log p| <= 1/e and p entropy <= log DC_MAX_VOCAB < 16.
__global__ __launch_bounds__(1024) void dc_linear_scale_kernel(uint64_t grad_logprobs, uint64_t grad_entropy, uint64_t tokens,
                                                               int tokens64, uint64_t rows, float inv_t, uint64_t scale) {
  pdl_enter();
  __shared__ float most[32];
  float m = 0.0f;
  for (uint64_t i = threadIdx.x; i < rows; i += blockDim.x) {
    float b = 0.0f;
    if (grad_logprobs && token_of(tokens, tokens64, i) >= 0) b += fabsf(ld_row(grad_logprobs, i, rows));
    if (grad_entropy) b += 16.0f * fabsf(ld_row(grad_entropy, i, rows));
    m = fmaxf(m, b * inv_t);
  }
#pragma unroll
  for (int d = 16; d > 0; d /= 2) m = fmaxf(m, __shfl_xor_sync(~0u, m, d));
  if ((threadIdx.x & 31) == 0) most[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x) return;
  for (int i = 1; i < 32; ++i) m = fmaxf(m, most[i]);
  int k = 0;
  if (m > 0.0f && m < __int_as_float(0x7F800000)) k = max(-100, min(100, 14 - ilogbf(m)));
  float* to = reinterpret_cast<float*>(scale);
  to[0] = __int_as_float((127 + k) << 23);
  to[1] = __int_as_float((127 - k) << 23);
}

template <int MODE, int DT, int NB>
cudaError_t launch_one(const LinearParams& p, const LinearOperand& a, const LinearOperand* b, const LinearShard* shards,
                       int sms, bool pdl, cudaStream_t s, int* grid) {
  static std::atomic<uint64_t> allowed{0};  // devices whose limit is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(allowed.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(dc_linear_kernel<MODE, DT, NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    allowed.fetch_or(bit, std::memory_order_relaxed);
  }
  LinearArgs<NB> args{};
  args.p = p;
  e = make_map(&args.a, DT, a.base, a.rows, a.columns, a.stride, 64);
  const int nb = MODE == kLinearStats ? p.shards : NB;
  for (int r = 0; r < nb && e == cudaSuccess; ++r) {
    e = make_map(&args.b[r], DT, b[r].base, b[r].rows, b[r].columns, b[r].stride, 64);
    if (MODE == kLinearStats) args.shard[r] = shards[r];
  }
  if (e != cudaSuccess) return e;
  const uint64_t tiles = MODE == kLinearGrads ? static_cast<uint64_t>(p.g.h_tiles) + p.g.w_tiles
                                              : static_cast<uint64_t>(p.m_tiles) * p.n_tiles;
  args.p.run = p.k_blocks <= kShortBlocks ? kShortRunBlocks : kRunBlocks;
  const uint64_t pairs = std::min<uint64_t>(tiles, std::min(std::max(static_cast<uint32_t>(sms) / 2, 1u), kLinearPairs));
  if constexpr (MODE == kLinearGrads) plan_linear_grads(&args.p.g, static_cast<uint32_t>(pairs));
  *grid = static_cast<int>(2 * pairs);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(*grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, dc_linear_kernel<MODE, DT, NB>, args);
}

template <int DT>
cudaError_t launch_mode(int mode, const LinearParams& p, const LinearOperand& a, const LinearOperand* b,
                        const LinearShard* shards, int sms, bool pdl, cudaStream_t s, int* grid) {
  switch (mode) {
    case kLinearStats:
      // (a parameter block of 64 tensor maps has 9 KB)
      return p.shards == 1   ? launch_one<kLinearStats, DT, 1>(p, a, b, shards, sms, pdl, s, grid)
             : p.shards <= 8 ? launch_one<kLinearStats, DT, 8>(p, a, b, shards, sms, pdl, s, grid)
                             : launch_one<kLinearStats, DT, kMaxRanks>(p, a, b, shards, sms, pdl, s, grid);
    case kLinearDLogits: return launch_one<kLinearDLogits, DT, 1>(p, a, b, shards, sms, pdl, s, grid);
    default: return launch_one<kLinearGrads, DT, 2>(p, a, b, shards, sms, pdl, s, grid);
  }
}

}  // namespace

namespace tc {

namespace {
using Encode = decltype(&cuTensorMapEncodeTiled);
cudaError_t encode_tiled(CUtensorMap* map, int dtype, uint64_t base, int dims, const cuuint64_t* size, const cuuint64_t* stride,
                         const cuuint32_t* box) {
  static std::atomic<Encode> encode{nullptr};  // the CUDA driver's function, looked up once
  Encode f = encode.load(std::memory_order_acquire);
  if (!f) {
    void* at = nullptr;
    cudaDriverEntryPointQueryResult found;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &at, 12000, cudaEnableDefault, &found);
    if (e != cudaSuccess) return e;
    if (!at || found != cudaDriverEntryPointSuccess) return cudaErrorNotSupported;
    f = reinterpret_cast<Encode>(at);
    encode.store(f, std::memory_order_release);
  }
  const cuuint32_t step[4] = {1, 1, 1, 1};
  const CUresult r = f(map, dtype == kF16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                       static_cast<cuuint32_t>(dims), reinterpret_cast<void*>(base), size, stride, box, step,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}
}  // namespace

cudaError_t make_map(CUtensorMap* map, int dtype, uint64_t base, uint64_t rows, uint64_t columns, uint64_t row_stride,
                     uint32_t tile_rows) {
  const cuuint64_t size[2] = {columns, rows}, stride[1] = {row_stride};
  const cuuint32_t box[2] = {64, tile_rows};
  return encode_tiled(map, dtype, base, 2, size, stride, box);
}

cudaError_t make_paged_map(CUtensorMap* map, int dtype, const PagedView& v, int dim, int heads, uint32_t page_size,
                           int64_t pages, uint32_t slots) {
  const cuuint64_t size[4] = {static_cast<cuuint64_t>(dim), static_cast<cuuint64_t>(heads), page_size, static_cast<cuuint64_t>(pages)};
  // (the stride of a dimension of one place is not used, but has to be a valid one)
  const cuuint64_t stride[3] = {heads > 1 ? v.head : 16, page_size > 1 ? v.token : 16, pages > 1 ? v.page : 16};
  const cuuint32_t box[4] = {64, 1, slots, 1};
  return encode_tiled(map, dtype, v.base, 4, size, stride, box);
}

}  // namespace tc

cudaError_t launch_linear(int mode, int dtype, const LinearParams& p, const LinearOperand& a, const LinearOperand* b,
                          const LinearShard* shards, int sms, bool pdl, cudaStream_t s, int* grid) {
  return dtype == kF16 ? launch_mode<kF16>(mode, p, a, b, shards, sms, pdl, s, grid)
                       : launch_mode<kBF16>(mode, p, a, b, shards, sms, pdl, s, grid);
}

void plan_linear_grads(LinearGrads* g, uint32_t pairs) {
  g->rounds = g->h_tiles / pairs;
  g->rest = g->h_tiles % pairs;
  // The number of common rounds after which those who had a dh tile less end with the others.
  const uint32_t on = pairs - g->rest;
  uint64_t best = ~0ull;
  for (uint32_t few = 0; few <= (g->rest ? g->w_tiles / pairs : 0); ++few) {
    const uint32_t many = few + (g->w_tiles - few * pairs + on - 1) / on;
    const uint64_t end = std::max((g->rest ? g->slice_blocks : 0) + static_cast<uint64_t>(few) * g->w_blocks,
                                  static_cast<uint64_t>(many) * g->w_blocks);
    if (end >= best) continue;
    best = end;
    g->few = few;
    g->many = many;
  }
}

cudaError_t launch_linear_sum(const LinearSumParams& p, int dtype, bool pdl, cudaStream_t s, int* grid) {
  *grid = static_cast<int>((p.rows * (p.size / 8) + 255) / 256);
  return dtype == kF16 ? launch_ex(dc_linear_sum_kernel<kF16>, *grid, 256, pdl, s, p)
                       : launch_ex(dc_linear_sum_kernel<kBF16>, *grid, 256, pdl, s, p);
}

cudaError_t launch_linear_lost(const LinearLostParams& p, int dtype, bool pdl, cudaStream_t s, int* grid) {
  const dim3 g((p.columns + kLinearN - 1) / kLinearN, (p.size + kLinearN - 1) / kLinearN);
  *grid = static_cast<int>(g.x * g.y);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = g;
  cfg.blockDim = dim3(kLostThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = pdl ? attr : nullptr;
  cfg.numAttrs = pdl ? 1 : 0;
  return dtype == kF16 ? cudaLaunchKernelEx(&cfg, dc_linear_lost_kernel<kF16>, p) : cudaLaunchKernelEx(&cfg, dc_linear_lost_kernel<kBF16>, p);
}

cudaError_t launch_linear_finish(const LinearFinishParams& p, bool pdl, cudaStream_t s, int* grid) {
  *grid = static_cast<int>(p.rows);
  return launch_ex(dc_linear_finish_kernel, *grid, kFinishThreads, pdl, s, p);
}

cudaError_t launch_linear_scale(uint64_t grad_logprobs, uint64_t grad_entropy, uint64_t tokens, bool tokens64, uint64_t rows,
                                float inv_t, uint64_t scale, bool pdl, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(1024);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = pdl ? attr : nullptr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, dc_linear_scale_kernel, grad_logprobs, grad_entropy, tokens, tokens64 ? 1 : 0, rows, inv_t, scale);
}

DC_BOUNDS_READER(take_bounds_linear)

DC_FAULT_READER(take_linear_faults, g_linear_fault_bits)

}  // namespace dc
