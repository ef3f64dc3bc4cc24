// Attention of one new token per sequence over a paged key-value cache.
//
// Mathematics.  For sequence b with n attended tokens and query head h of
// key head k:  o = sum_t softmax_t(scale q.k_t) v_t.  The tokens are cut into
// pieces whose length follows from n and the head counts alone, so what else
// is in the batch changes no bit.  A piece keeps, per head, its maximum m,
// its sum l = sum 2^(s_t - m) and its unnormalised output, all in binary32
// (s_t = scale log2(e) q.k_t); the last piece to finish joins them in order:
// M = max m, o = sum 2^(m-M) o_piece / sum 2^(m-M) l.
//
// Bound: memory.  Every key and value is read once; at 8 query heads per key
// head that is 8 multiply-adds per byte, which the matrix pipe does with a
// wide margin (mma.m16n8k16, 16 heads x 8 tokens), so it is fed from shared
// memory by cp.async and never waited for.  A warp owns 16 tokens at a time
// with a ring of its own: no barrier until the piece is done.
//
// Rounding.  The weights 2^(s-m) enter the second product as a pair of 16-bit
// numbers hi + lo (hi the weight cut to 16 bits, lo the rounded rest), so
// that the output carries one rounding to 16 bits, the last.  With at most 8 heads to
// a CTA the pair fills the tile's 16 rows and costs nothing.
#include <atomic>

#include "dc_llm.h"
#include "dc_numeric.cuh"

namespace dc {
namespace {

enum : uint32_t {
  kSiteLength = 1, kSiteTable = 2, kSiteQuery = 3, kSiteKey = 4, kSiteValue = 5, kSiteOut = 6, kSitePartial = 7,
};

constexpr int kThreads = kAttendWarps * 32;

template <int D>
struct Ring {
  static constexpr int kRow = D * 2 + 16;                      // bytes; the 16 keep ldmatrix free of conflicts
  static constexpr int kHalf = kAttendTile * kRow;             // keys or values of one tile
  static constexpr int kStage = 2 * kHalf;
  static constexpr int kStages = D > 128 ? 2 : 3;
  static constexpr int kBytes = kAttendWarps * kStages * kStage;
};

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
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

// hi: both weights cut to 16 bits; lo: what that left out, rounded.  lo stays
// positive (2^-20 of the weight at least), so that an infinite value gives an
// infinity and not 0 * inf.
template <int DT>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t& hi, uint32_t& lo) {
  if constexpr (DT == kF16)
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(y), "f"(x));
  else
    asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(y), "f"(x));
  constexpr float kLeast = 1.0f / (1 << 20);
  lo = Elem<DT>::pack(fmaxf(x - Elem<DT>::lo(hi), x * kLeast), fmaxf(y - Elem<DT>::hi(hi), y * kLeast));
}

// Stores `v` as a 16-bit element pair.
template <int DT>
__device__ __forceinline__ void st_pair(uint64_t a, float x, float y, uint64_t lo, uint64_t hi) {
  if (in_bounds(reinterpret_cast<const void*>(a), 4, lo, hi, kSiteOut))
    *reinterpret_cast<uint32_t*>(a) = Elem<DT>::pack(x, y);
}

template <int DT, int D, int HB>
__global__ __launch_bounds__(kThreads) void dc_attend_kernel(const __grid_constant__ AttendParams p) {
  using R = Ring<D>;
  constexpr int kSteps = D / 16;          // k-steps of q.k, and 16-element column groups of the output
  constexpr int kVecs = D / 8;            // 16-byte vectors of a token's key
  constexpr int kCopies = kAttendTile * kVecs / 32;
  static_assert(kAttendTile * kVecs % 32 == 0, "a tile is whole copies of a warp");
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float w_m[kAttendWarps][HB], w_l[kAttendWarps][HB];
  __shared__ uint32_t last_piece;
  int32_t* pages = reinterpret_cast<int32_t*>(smem + R::kBytes);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;

  const uint32_t split = blockIdx.x % static_cast<uint32_t>(p.splits);
  const uint32_t unit = blockIdx.x / static_cast<uint32_t>(p.splits);  // (sequence, key head, head block)
  const int hb = static_cast<int>(unit % static_cast<uint32_t>(p.head_blocks));
  const int kh = static_cast<int>(unit / static_cast<uint32_t>(p.head_blocks) % static_cast<uint32_t>(p.kv_heads));
  const int seq = static_cast<int>(unit / static_cast<uint32_t>(p.head_blocks) / static_cast<uint32_t>(p.kv_heads));
  const int h0 = kh * p.group + hb * HB;                        // first query head
  const int nh = min(HB, p.group - hb * HB);                    // query heads of this CTA
  pdl_enter();

  const int32_t* lp = reinterpret_cast<const int32_t*>(p.lengths) + seq;
  int32_t len = in_bounds(lp, 4, p.lengths, p.lengths + 4ull * p.seqs, kSiteLength) ? *lp : 0;
  // a length past the table: the tokens that exist are not known, the output is NaN
  const uint64_t room = static_cast<uint64_t>(p.table_width) * p.page_size;
  bool bad = len > 0 && static_cast<uint64_t>(len) > room;
  if (len < 0) len = 0;
  if (bad) len = static_cast<int32_t>(min(room, static_cast<uint64_t>(1)));
  const uint32_t start = p.window > 0 && len > p.window ? static_cast<uint32_t>(len - p.window) : 0u;
  const uint32_t n = static_cast<uint32_t>(len) - start;
  const uint32_t chunk = attend_chunk(n, static_cast<uint32_t>(p.target));
  const uint32_t pieces = n / chunk + (n % chunk != 0);
  const uint64_t out_row = p.out + static_cast<uint64_t>(seq) * p.out_seq;
  if (split >= pieces) {
    if (split == 0) {  // nothing to attend to: zeros
      for (int i = threadIdx.x; i < nh * (D / 2); i += kThreads) {
        const uint64_t row = out_row + static_cast<uint64_t>(h0 + i / (D / 2)) * p.out_head;
        st_pair<DT>(row + static_cast<uint64_t>(i % (D / 2)) * 4, 0.0f, 0.0f, row, row + D * 2);
      }
      if (p.lse && threadIdx.x < nh) {
        float* a = reinterpret_cast<float*>(p.lse) + static_cast<uint64_t>(seq) * p.q_heads + h0 + threadIdx.x;
        if (in_bounds(a, 4, p.lse, p.lse + 4ull * p.seqs * p.q_heads, kSiteOut)) *a = neg_inf();
      }
    }
    return;
  }
  const uint32_t t0 = start + split * chunk;
  const uint32_t t1 = min(t0 + chunk, static_cast<uint32_t>(len));

  // the piece's page numbers; a page outside the cache is never touched
  const uint32_t page0 = t0 / p.page_size, npages = (t1 - 1) / p.page_size - page0 + 1;
  for (uint32_t i = threadIdx.x; i < npages; i += kThreads) {
    const int32_t* a = reinterpret_cast<const int32_t*>(p.table) + seq * p.table_stride + page0 + i;
    const uint64_t hi = p.table + (static_cast<uint64_t>(p.seqs - 1) * p.table_stride + p.table_width) * 4;
    int32_t id = in_bounds(a, 4, p.table, hi, kSiteTable) ? *a : -1;
    if (id < 0 || id >= p.num_pages) {
      id = -1;
      bad = true;
    }
    pages[i] = id;
  }

  // query fragments: rows 0..7 heads h0.., rows 8..15 heads h0 + 8.. (HB 16)
  uint32_t qf[kSteps][HB == 16 ? 4 : 2];
  {
    const int g = lane >> 2;
#pragma unroll
    for (int half = 0; half < HB / 8; ++half) {
      const int h = g + 8 * half;
      const uint64_t row = p.q + static_cast<uint64_t>(seq) * p.q_seq + static_cast<uint64_t>(h0 + h) * p.q_head;
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t* a =
              reinterpret_cast<const uint32_t*>(row + static_cast<uint64_t>(k * 16 + i * 8 + (lane & 3) * 2) * 2);
          // a[0]: row g, first 8 columns; a[1]: row g + 8; a[2], a[3]: the next 8 columns
          qf[k][HB == 16 ? 2 * i + half : i] =
              h < nh && in_bounds(a, 4, row, row + D * 2, kSiteQuery) ? *a : 0u;
        }
    }
  }
  bad = __syncthreads_or(bad);

  const uint32_t tiles = (t1 - t0 + kAttendTile - 1) / kAttendTile;
  const uint32_t mine = tiles > static_cast<uint32_t>(warp) ? (tiles - warp - 1) / kAttendWarps + 1 : 0;
  const uint32_t ring = smem_addr(smem) + static_cast<uint32_t>(warp * R::kStages * R::kStage);

  // issues the copies of this warp's tile i; lanes 0..15 look up the tokens'
  // keys, lanes 16..31 their values
  auto issue = [&](uint32_t i) {
    if (i < mine) {
      const uint32_t t = t0 + (i * kAttendWarps + warp) * kAttendTile + (lane & 15);
      uint64_t row = 0;
      if (t < t1) {
        const uint32_t pg = t / p.page_size;
        const int32_t id = pages[pg - page0];
        const PagedView& c = lane < 16 ? p.kc : p.vc;
        if (id >= 0)
          row = c.base + static_cast<uint64_t>(id) * c.page + static_cast<uint64_t>(t - pg * p.page_size) * c.token +
                static_cast<uint64_t>(kh) * c.head;
      }
      const uint32_t dst = ring + (i % R::kStages) * R::kStage;
#pragma unroll
      for (int half = 0; half < 2; ++half)
#pragma unroll
        for (int j = 0; j < kCopies; ++j) {
          const int v = j * 32 + lane, r = v / kVecs, col = v % kVecs;
          const uint64_t a = __shfl_sync(~0u, row, r + 16 * half);
          const uint64_t src = a ? a + col * 16 : (half ? p.vc.base : p.kc.base);
          const bool read = a != 0 && in_bounds(reinterpret_cast<const void*>(src), 16, half ? p.vc.lo : p.kc.lo,
                                                half ? p.vc.hi : p.kc.hi, half ? kSiteValue : kSiteKey);
          cp_async16_or_zero(dst + half * R::kHalf + r * R::kRow + col * 16, src, read);
        }
    }
    cp_async_commit();
  };

  float m[HB / 8], l[HB / 8], o[D / 8][4];
#pragma unroll
  for (int i = 0; i < HB / 8; ++i) {
    m[i] = neg_inf();
    l[i] = 0.0f;
  }
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) o[i][j] = 0.0f;
  const float sc = p.scale * kLog2E;

#pragma unroll
  for (int i = 0; i < R::kStages - 1; ++i) issue(i);
  for (uint32_t i = 0; i < mine; ++i) {
    issue(i + R::kStages - 1);
    cp_async_wait<R::kStages - 1>();
    __syncwarp();
    const uint32_t kt = ring + (i % R::kStages) * R::kStage, vt = kt + R::kHalf;
    // scores: 16 heads x 16 tokens
    float s[2][4] = {};
    {
      const uint32_t a = kt + ((lane >> 4) * 8 + (lane & 7)) * R::kRow + ((lane >> 3) & 1) * 16;
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
        mma<DT>(s[0], q, b[0], b[1]);
        mma<DT>(s[1], q, b[2], b[3]);
      }
    }
    const uint32_t base = t0 + (i * kAttendWarps + warp) * kAttendTile;
    const bool partial = base + kAttendTile > t1;
    uint32_t phi[4], plo[4];
#pragma unroll
    for (int half = 0; half < HB / 8; ++half) {
      float x[4] = {s[0][2 * half] * sc, s[0][2 * half + 1] * sc, s[1][2 * half] * sc, s[1][2 * half + 1] * sc};
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
      const float mn = fmaxf(m[half], mx);
      if (__any_sync(~0u, mn > m[half])) {
        const float f = m[half] == neg_inf() ? 0.0f : ex2(m[half] - mn);
        l[half] *= f;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
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
      const float ref = mn == neg_inf() ? 0.0f : mn;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j] = ex2(x[j] - ref);
        l[half] += x[j];
      }
      split_pair<DT>(x[0], x[1], phi[half], plo[half]);
      split_pair<DT>(x[2], x[3], phi[2 + half], plo[2 + half]);
    }
    {
      const uint32_t a = vt + (((lane >> 3) & 1) * 8 + (lane & 7)) * R::kRow + (lane >> 4) * 16;
      uint32_t w[4];
      if constexpr (HB == 8) {
        w[0] = phi[0];
        w[1] = plo[0];
        w[2] = phi[2];
        w[3] = plo[2];
      }
#pragma unroll
      for (int c = 0; c < kSteps; ++c) {
        uint32_t b[4];
        ldmatrix4_t(a + c * 32, b);
        if constexpr (HB == 16) {
          mma<DT>(o[2 * c], phi, b[0], b[1]);
          mma<DT>(o[2 * c + 1], phi, b[2], b[3]);
          mma<DT>(o[2 * c], plo, b[0], b[1]);
          mma<DT>(o[2 * c + 1], plo, b[2], b[3]);
        } else {
          mma<DT>(o[2 * c], w, b[0], b[1]);
          mma<DT>(o[2 * c + 1], w, b[2], b[3]);
        }
      }
    }
    __syncwarp();
  }
  cp_async_wait<0>();

  // the piece: the warps' maxima, sums and outputs joined in warp order
#pragma unroll
  for (int half = 0; half < HB / 8; ++half) {
    l[half] += __shfl_xor_sync(~0u, l[half], 1);
    l[half] += __shfl_xor_sync(~0u, l[half], 2);
    if ((lane & 3) == 0) {
      w_m[warp][(lane >> 2) + 8 * half] = m[half];
      w_l[warp][(lane >> 2) + 8 * half] = l[half];
    }
  }
  __syncthreads();  // every warp has read its last tile: the ring is free
  float* wo = reinterpret_cast<float*>(smem);  // [warp][head][D]
  static_assert(kAttendWarps * HB * D * 4 <= R::kBytes, "the warps' outputs fit in the ring");
  {
    const int g = lane >> 2;
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {
      float* a = wo + (warp * HB + g) * D + c * 8 + (lane & 3) * 2;
      if constexpr (HB == 16) {
        *reinterpret_cast<float2*>(a) = make_float2(o[c][0], o[c][1]);
        *reinterpret_cast<float2*>(a + 8 * D) = make_float2(o[c][2], o[c][3]);
      } else {  // rows 8..15 hold the low parts
        *reinterpret_cast<float2*>(a) = make_float2(o[c][0] + o[c][2], o[c][1] + o[c][3]);
      }
    }
  }
  __syncthreads();
  const uint64_t unit_floats = static_cast<uint64_t>(p.splits) * HB * (D + 2);
  float* part = reinterpret_cast<float*>(p.partial) + unit * unit_floats;
  const uint64_t part_lo = reinterpret_cast<uint64_t>(part), part_hi = part_lo + unit_floats * 4;
  float* part_ml = part + static_cast<uint64_t>(p.splits) * HB * D;
  for (int i = threadIdx.x; i < nh * (D / 4); i += kThreads) {
    const int h = i / (D / 4), d = i % (D / 4) * 4;
    float M = w_m[0][h];
#pragma unroll
    for (int w = 1; w < kAttendWarps; ++w) M = fmaxf(M, w_m[w][h]);
    float lsum = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kAttendWarps; ++w) {
      const float f = w_m[w][h] == neg_inf() ? 0.0f : ex2(w_m[w][h] - M);
      const float4 x = *reinterpret_cast<const float4*>(wo + (w * HB + h) * D + d);
      lsum = __fmaf_rn(w_l[w][h], f, lsum);
      acc.x = __fmaf_rn(x.x, f, acc.x);
      acc.y = __fmaf_rn(x.y, f, acc.y);
      acc.z = __fmaf_rn(x.z, f, acc.z);
      acc.w = __fmaf_rn(x.w, f, acc.w);
    }
    // scores that are all NaN leave no maximum; they and a missing page give NaN
    if (bad) lsum = __int_as_float(0x7FC00000);
    if (pieces == 1) {
      const float inv = 1.0f / lsum;
      const uint64_t row = out_row + static_cast<uint64_t>(h0 + h) * p.out_head;
      st_pair<DT>(row + d * 2, acc.x * inv, acc.y * inv, row, row + D * 2);
      st_pair<DT>(row + d * 2 + 4, acc.z * inv, acc.w * inv, row, row + D * 2);
      if (d == 0 && p.lse) {
        float* a = reinterpret_cast<float*>(p.lse) + static_cast<uint64_t>(seq) * p.q_heads + h0 + h;
        if (in_bounds(a, 4, p.lse, p.lse + 4ull * p.seqs * p.q_heads, kSiteOut)) *a = (M + log2f(lsum)) * kLn2;
      }
    } else {
      float* a = part + (static_cast<uint64_t>(split) * HB + h) * D + d;
      if (in_bounds(a, 16, part_lo, part_hi, kSitePartial)) *reinterpret_cast<float4*>(a) = acc;
      if (d == 0) {
        float* b = part_ml + (static_cast<uint64_t>(split) * HB + h) * 2;
        if (in_bounds(b, 8, part_lo, part_hi, kSitePartial)) *reinterpret_cast<float2*>(b) = make_float2(M, lsum);
      }
    }
  }
  if (pieces == 1) return;

  // the last piece to arrive joins them all, in order
  __threadfence();
  __syncthreads();
  uint32_t* counter = reinterpret_cast<uint32_t*>(p.counters) + unit;
  if (threadIdx.x == 0) last_piece = atomicAdd(counter, 1u) == pieces - 1 ? 1u : 0u;
  __syncthreads();
  if (!last_piece) return;
  __threadfence();
  if (threadIdx.x == 0) *counter = 0;  // ready for the next call
  float* jw = reinterpret_cast<float*>(smem);  // weights [piece][HB]; then M and 1/L of every head
  for (int h = warp; h < nh; h += kAttendWarps) {
    float M = neg_inf();
    for (uint32_t i = lane; i < pieces; i += 32) M = max_nan(M, __ldcg(part_ml + (i * HB + h) * 2));
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) M = max_nan(M, __shfl_xor_sync(~0u, M, x));
    const float ref = M == neg_inf() ? 0.0f : M;
    float L = 0.0f;
    for (uint32_t i = lane; i < pieces; i += 32) {
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(part_ml + (i * HB + h) * 2));
      const float f = ex2(ml.x - ref);
      jw[i * HB + h] = f;
      L = __fmaf_rn(ml.y, f, L);
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) L += __shfl_xor_sync(~0u, L, x);
    if (lane == 0) {
      w_m[0][h] = M;
      w_l[0][h] = L;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < nh * (D / 4); i += kThreads) {
    const int h = i / (D / 4), d = i % (D / 4) * 4;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
    for (uint32_t s = 0; s < pieces; ++s) {
      const float4* a = reinterpret_cast<const float4*>(part + (static_cast<uint64_t>(s) * HB + h) * D + d);
      const float4 x = in_bounds(a, 16, part_lo, part_hi, kSitePartial) ? __ldcg(a) : float4{};
      const float f = jw[s * HB + h];
      acc.x = __fmaf_rn(x.x, f, acc.x);
      acc.y = __fmaf_rn(x.y, f, acc.y);
      acc.z = __fmaf_rn(x.z, f, acc.z);
      acc.w = __fmaf_rn(x.w, f, acc.w);
    }
    const float inv = 1.0f / w_l[0][h];
    const uint64_t row = out_row + static_cast<uint64_t>(h0 + h) * p.out_head;
    st_pair<DT>(row + d * 2, acc.x * inv, acc.y * inv, row, row + D * 2);
    st_pair<DT>(row + d * 2 + 4, acc.z * inv, acc.w * inv, row, row + D * 2);
    if (d == 0 && p.lse) {
      float* a = reinterpret_cast<float*>(p.lse) + static_cast<uint64_t>(seq) * p.q_heads + h0 + h;
      if (in_bounds(a, 4, p.lse, p.lse + 4ull * p.seqs * p.q_heads, kSiteOut)) *a = (w_m[0][h] + log2f(w_l[0][h])) * kLn2;
    }
  }
}

template <int DT, int D, int HB>
cudaError_t launch_one(const AttendParams& p, bool pdl, cudaStream_t s, int grid) {
  constexpr int kMost = Ring<D>::kBytes + (kAttendMaxChunk + 4) * 4;
  static_assert(kMost + 2048 <= 227 * 1024, "the ring and the page numbers fit");
  static_assert(kAttendMaxSplits * HB * 4 <= Ring<D>::kBytes, "the pieces' weights fit in the ring");
  const size_t smem = static_cast<size_t>(Ring<D>::kBytes) + static_cast<size_t>(p.page_slots) * 4;
  static std::atomic<uint64_t> allowed{0};  // devices whose limit is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(allowed.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(dc_attend_kernel<DT, D, HB>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost);
    if (e != cudaSuccess) return e;
    allowed.fetch_or(bit, std::memory_order_relaxed);
  }
  return launch_ex(dc_attend_kernel<DT, D, HB>, grid, kThreads, pdl, s, p, smem);
}

template <int DT, int D>
cudaError_t launch_hb(const AttendParams& p, bool pdl, cudaStream_t s, int grid) {
  return attend_head_block(p.group) == 16 ? launch_one<DT, D, 16>(p, pdl, s, grid) : launch_one<DT, D, 8>(p, pdl, s, grid);
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
  *grid = p.seqs * p.kv_heads * p.head_blocks * p.splits;
  return dtype == kF16 ? launch_dim<kF16>(p, dim, pdl, s, *grid) : launch_dim<kBF16>(p, dim, pdl, s, *grid);
}

DC_BOUNDS_READER(take_bounds_attention)

}  // namespace dc
