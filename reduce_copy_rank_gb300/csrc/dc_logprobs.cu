// Log probabilities of given tokens over vocabulary shards, with entropy and
// the likeliest alternatives, and their gradient.
//
// Mathematics.  With z_i = x_i / T over the whole vocabulary,
//     lse = log sum_i exp(z_i),  logprob(y) = z_y - lse,
//     H   = lse - sum_i p_i z_i,
//     d/dx_i = (1/T) [ g (1[i = y] - p_i) - h p_i (log p_i + H) ]
// for upstream gradients g of the log probability and h of the entropy.  A
// segment of the vocabulary is reduced around its largest logit m in base 2:
//     a_i = (x_i - m) log2(e)/T,   s = sum 2^a_i,   t = sum 2^a_i a_i,
// and segments join around the row's largest logit M, with d = (m - M)
// log2(e)/T:   S = sum 2^d s,   U = sum 2^d (t + d s).  Then
//     lse = M/T + ln S,   logprob = (x_y - M)/T - ln S,   H = ln S - ln2 U/S.
// The difference is taken first, so the largest logit's exponent is exactly 0
// and logits of any finite size (masks of the type's lowest value) do not
// overflow.  All of it in binary32.
//
// Bound: memory for many rows.  The logits are read once (and the gradient
// written once); an element costs about five instructions, one of them the
// exponential: pairs of elements share the additions and products, which took
// 8192 x 128000 bf16 from 322 to 301 us.  For few rows a cluster of up to 8
// CTAs shares a row and the time is the chain of one load, one reduction, the
// cluster's barrier and (with alternatives) the search for them.  Between, a
// row's CTA spends as long on that chain as on its logits.
//
// Measured on GB300 (copy rate 6.78 TB/s; launches replayed from a graph), scores:
// 8192 x 128000 bf16 303 us, 6.9 TB/s; 1021 x 50021 f32 on 3 ranks with 5
// alternatives 51 us, 4.0 TB/s; 128 x 131072 bf16 on 8 ranks with 20 16.7 us; 4 x
// 32768 with 1 6.3 us.  Gradient: 8192 x 127900 bf16 on 8 ranks 611 us, 6.9 TB/s;
// 509 x 50021 f16 17 us, 5.9 TB/s; narrow shards (2849 x 14007 bf16 on 8 ranks: 219
// vectors a row of a shard, for CTAs of up to 1024) 60 us, 2.7 TB/s, issue slots 87 %
// busy with what a CTA does once.
#include <cfloat>

#include "dc_llm.h"
#include "dc_numeric.cuh"

namespace dc {
namespace {

enum : uint32_t {
  kSiteLogit = 1, kSiteToken = 2, kSiteScore = 3, kSiteTop = 4, kSiteGradIn = 5, kSiteGradOut = 6, kSiteRow = 7,
};

// Entry `i` of an array of n, and its store, checked in the checked build.
template <class T>
__device__ __forceinline__ T ld_entry(uint64_t base, uint64_t i, uint64_t n, uint32_t site) {
  const T* a = reinterpret_cast<const T*>(base) + i;
  return in_bounds(a, sizeof(T), base, base + n * sizeof(T), site) ? *a : T{};
}
template <class T>
__device__ __forceinline__ void st_entry(uint64_t base, uint64_t i, uint64_t n, T v, uint32_t site) {
  T* a = reinterpret_cast<T*>(base) + i;
  if (in_bounds(a, sizeof(T), base, base + n * sizeof(T), site)) *a = v;
}
// A token index of either width.
__device__ __forceinline__ int64_t ld_token(uint64_t base, uint64_t i, uint64_t n, bool is64) {
  return is64 ? ld_entry<int64_t>(base, i, n, kSiteToken)
              : static_cast<int64_t>(ld_entry<int32_t>(base, i, n, kSiteToken));
}

// ------------------------------------------------------------- clusters ---
__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
// The address of this CTA's shared `local` in the cluster's CTA 0.
__device__ __forceinline__ uint32_t leader_addr(uint32_t local) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(local));
  return a;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_cluster64(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// ------------------------------------------------- sorted lists of a warp ---
// Keys, one a lane, largest first; a key is (ordered value, ~index), so equal
// values rank by the lowest index.
__device__ __forceinline__ uint64_t exchange(uint64_t k, int partner_xor, bool keep_max) {
  const uint64_t o = __shfl_xor_sync(~0u, k, partner_xor);
  return (k > o) == keep_max ? k : o;
}
__device__ __forceinline__ uint64_t bitonic_tail(uint64_t k, int lane) {
#pragma unroll
  for (int j = 16; j > 0; j >>= 1) k = exchange(k, j, (lane & j) == 0);
  return k;
}
__device__ __forceinline__ uint64_t sort_desc(uint64_t k, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int j = size >> 1; j > 0; j >>= 1) k = exchange(k, j, ((lane & j) == 0) == ((lane & size) == 0));
  return k;
}
// The 32 largest of two sorted lists, sorted.
__device__ __forceinline__ uint64_t merge_desc(uint64_t a, uint64_t b, int lane) {
  const uint64_t r = __shfl_sync(~0u, b, 31 - lane);
  return bitonic_tail(a > r ? a : r, lane);
}
// Entries of a sorted list of 32 that are larger than `key`.
__device__ __forceinline__ uint32_t larger_in(const uint64_t* list, uint64_t key) {
  uint32_t n = 0;
#pragma unroll
  for (uint32_t s = 16; s > 0; s >>= 1)
    if (list[n + s - 1] > key) n += s;
  return n + (list[n] > key ? 1u : 0u);
}

constexpr uint32_t kFewCandidates = 256;  // of a CTA

struct TopList {
  uint64_t key;    // this lane's entry of the list, largest in lane 0
  uint32_t count;  // candidates waiting in the buffer
  float thr;       // nothing below it can be among the k largest
};

// Sorts the first 32 waiting candidates into the list.
__device__ __noinline__ void flush_candidates(TopList& t, uint64_t* buf, int k, int lane) {
  const uint32_t n = t.count < 32u ? t.count : 32u;
  __syncwarp();
  const uint64_t c = lane < static_cast<int>(n) ? buf[lane] : 0;
  const uint64_t rest = static_cast<uint32_t>(lane) + n < t.count ? buf[lane + n] : 0;
  __syncwarp();
  t.count -= n;
  if (static_cast<uint32_t>(lane) < t.count) buf[lane] = rest;
  __syncwarp();
  t.key = merge_desc(t.key, sort_desc(c, lane), lane);
  const uint64_t kth = __shfl_sync(~0u, t.key, k - 1);
  if (kth != 0) t.thr = fmaxf(t.thr, from_ordered(static_cast<uint32_t>(kth >> 32)));
}

// Loads where `ok`, without a branch; the rest keep what they hold.
__device__ __forceinline__ void ld_where(uint32_t& v, uint64_t a, bool ok) {
  asm volatile("{ .reg .pred q; setp.ne.u32 q, %2, 0; @q ld.global.nc.u32 %0, [%1]; }"
               : "+r"(v) : "l"(a), "r"(static_cast<uint32_t>(ok)));
}
__device__ __forceinline__ void ld16_where(uint4& v, uint64_t a, bool ok) {
  asm volatile("{ .reg .pred q; setp.ne.u32 q, %5, 0; @q ld.global.nc.v4.u32 {%0, %1, %2, %3}, [%4]; }"
               : "+r"(v.x), "+r"(v.y), "+r"(v.z), "+r"(v.w) : "l"(a), "r"(static_cast<uint32_t>(ok)));
}

// --------------------------------------------------------- one segment ---
// How a segment's entries lie in a warp: 16-bit types as 8 vectors of 8
// entries a lane, vector j at (j * 32 + lane) * 8; binary32 as 32 single
// entries, entry j at j * 32 + lane.  (Rows of binary32 logits start at any
// multiple of 4 bytes: single entries load at full width from all of them.
// 16-bit rows that do not start at a multiple of 16 bytes read the two blocks
// around each vector and shift.)  The layout is the same for every alignment
// and sharding, and with it the order of the additions.
template <int DT>
struct SegLoader {
  static constexpr int kPer = Elem<DT>::kPerVec;
  static constexpr uint32_t kSeg = vocab_seg(DT);
  static constexpr int kVecs = static_cast<int>(kSeg) / kPer / 32;  // 16-byte groups a lane holds

  // The index in the segment of element i of group j.
  __device__ static __forceinline__ uint32_t index(int j, int i, int lane) {
    if constexpr (DT == kF32) return static_cast<uint32_t>((j * 4 + i) * 32 + lane);
    else return static_cast<uint32_t>((j * 32 + lane) * kPer + i);
  }

  template <int W>  // byte offset / 4 of the vectors in their 16-byte blocks
  __device__ static __forceinline__ void load_shifted(const uint4* b, uint32_t bits, uint64_t lo, uint64_t hi,
                                                      uint4 (&raw)[kVecs]) {
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const uint4 x = in_bounds(b + 32 * j, 16, lo, hi, kSiteLogit) ? ld_nc_cached(b + 32 * j) : uint4{};
      const uint4 y = in_bounds(b + 32 * j + 1, 16, lo, hi, kSiteLogit) ? ld_nc_cached(b + 32 * j + 1) : uint4{};
      const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
      raw[j] = make_uint4(__funnelshift_r(w[W], w[W + 1], bits), __funnelshift_r(w[W + 1], w[W + 2], bits),
                          __funnelshift_r(w[W + 2], w[W + 3], bits), __funnelshift_r(w[W + 3], w[W + 4], bits));
    }
  }

  // Lane `lane`'s part of segment `seg` of row `row`; entries past the
  // vocabulary read -inf.  r: the shard of the previous segment of this warp
  // (segments come in order).
  __device__ static __forceinline__ void load(const ScoreParams& p, uint64_t row, int seg, int lane, int& r,
                                              uint4 (&raw)[kVecs]) {
    const uint32_t e0 = static_cast<uint32_t>(seg) * kSeg;
    while (p.shard[r].end <= e0) ++r;
    const LogitShard& sh = p.shard[r];
    const uint64_t bytes = (p.rows - 1) * sh.stride + static_cast<uint64_t>(sh.end - sh.first) * Elem<DT>::kBytes;
    if (e0 + kSeg <= sh.end) {
      const uint64_t a0 = sh.base + row * sh.stride + static_cast<uint64_t>(e0 - sh.first) * Elem<DT>::kBytes;
      if constexpr (DT == kF32) {
        const uint32_t* a = reinterpret_cast<const uint32_t*>(a0) + lane;
        const uint64_t lo = sh.base, hi = sh.base + bytes;
        auto get = [&](int k) {
          uint32_t v = 0;
          if (in_bounds(a + 32 * k, 4, lo, hi, kSiteLogit))
            asm volatile("ld.global.nc.u32 %0, [%1];" : "=r"(v) : "l"(a + 32 * k));
          return v;
        };
#pragma unroll
        for (int j = 0; j < kVecs; ++j) raw[j] = make_uint4(get(4 * j), get(4 * j + 1), get(4 * j + 2), get(4 * j + 3));
      } else {
        const uint64_t lo = hull_lo(sh.base), hi = hull_hi(sh.base, bytes);
        const uint64_t a = a0 + static_cast<uint64_t>(lane) * 16;
        const uint32_t s = static_cast<uint32_t>(a & 15u), bits = (s & 3u) * 8;
        const uint4* b = reinterpret_cast<const uint4*>(a - s);
        if (s == 0) {
#pragma unroll
          for (int j = 0; j < kVecs; ++j)
            raw[j] = in_bounds(b + 32 * j, 16, lo, hi, kSiteLogit) ? ld_nc_stream(b + 32 * j) : uint4{};
        } else if (s < 8) {
          if (s < 4) load_shifted<0>(b, bits, lo, hi, raw);
          else load_shifted<1>(b, bits, lo, hi, raw);
        } else {
          if (s < 12) load_shifted<2>(b, bits, lo, hi, raw);
          else load_shifted<3>(b, bits, lo, hi, raw);
        }
      }
      return;
    }
    // A segment that crosses shards or ends the vocabulary: two shards at a
    // time, every load of theirs in flight at once (each lane picks the shard
    // of its entry and loads under a predicate: as branches per shard and
    // vector they waited for one another; 1024 x 128256 bf16 on 8 ranks, 7 of
    // 63 segments, 78 us that way and 46 this way).  A vector that a shard's
    // end cuts is put together by lanes 0..7 (8..15 for the second shard's
    // end), an entry each.
#pragma unroll
    for (int j = 0; j < kVecs; ++j)
      raw[j] = make_uint4(Elem<DT>::kNegInfWord, Elem<DT>::kNegInfWord, Elem<DT>::kNegInfWord, Elem<DT>::kNegInfWord);
    for (int q = r; q < p.P && p.shard[q].first < e0 + kSeg; q += 2) {
      const bool pair = q + 1 < p.P;
      const LogitShard& s0 = p.shard[q];
      const LogitShard& s1 = p.shard[pair ? q + 1 : q];
      const uint32_t cut = s0.end, end = pair ? s1.end : s0.end;
      // addresses of column 0
      const uint64_t at0 = s0.base + row * s0.stride - static_cast<uint64_t>(s0.first) * Elem<DT>::kBytes;
      const uint64_t at1 = s1.base + row * s1.stride - static_cast<uint64_t>(s1.first) * Elem<DT>::kBytes;
      if constexpr (DT == kF32) {
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
          uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            const uint32_t e = e0 + index(j, i, lane);
            const uint64_t x = (e < cut ? at0 : at1) + static_cast<uint64_t>(e) * 4;
            ld_where(w[i], x, e >= s0.first && e < end && inside(p, e < cut ? s0 : s1, x, 4));
          }
          raw[j] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      } else {
        uint32_t odd = Elem<DT>::kNegInfWord;  // this lane's entry of a cut vector
        const uint32_t of = (lane < 8 ? cut : end) - e0;  // where the cut is in the segment
        {
          const uint32_t e = e0 + of / kPer * kPer + (lane & 7);
          if (lane < 16 && of < kSeg && of % kPer != 0 && e < p.vocab) {
            int n = r;
            while (p.shard[n].end <= e) ++n;
            const LogitShard& t = p.shard[n];
            const uint64_t x = t.base + row * t.stride + static_cast<uint64_t>(e - t.first) * 2;
            if (inside(p, t, x, 2)) odd = *reinterpret_cast<const uint16_t*>(x);
          }
        }
        const uint32_t o0 = static_cast<uint32_t>(at0 + static_cast<uint64_t>(e0) * 2) & 15u,
                       o1 = static_cast<uint32_t>(at1 + static_cast<uint64_t>(e0) * 2) & 15u;
        auto whole = [&](uint32_t e) { return e >= s0.first && (e + kPer <= cut || (e >= cut && e + kPer <= end)); };
        if ((o0 | o1) == 0) {
#pragma unroll
          for (int j = 0; j < kVecs; ++j) {
            const uint32_t e = e0 + index(j, 0, lane);
            const uint64_t x = (e < cut ? at0 : at1) + static_cast<uint64_t>(e) * 2;
            ld16_where(raw[j], x, whole(e) && inside(p, e < cut ? s0 : s1, x, 16));
          }
        } else {
          constexpr int kBatch = 2;  // (4: registers spill, and with alternatives that costs more than it saves)
#pragma unroll
          for (int j0 = 0; j0 < kVecs; j0 += kBatch) {
            uint4 next[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
              const uint32_t e = e0 + index(j0 + k, 0, lane);
              const uint32_t o = e < cut ? o0 : o1;
              const uint64_t x = (e < cut ? at0 : at1) + static_cast<uint64_t>(e) * 2 - o;
              const bool ok = whole(e) && inside(p, e < cut ? s0 : s1, x + o, 16);
              ld16_where(raw[j0 + k], x, ok);
              next[k] = raw[j0 + k];
              ld16_where(next[k], x + 16, ok && o != 0);
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
              const uint32_t e = e0 + index(j0 + k, 0, lane);
              if (whole(e)) raw[j0 + k] = realign16_sel(raw[j0 + k], next[k], e < cut ? o0 : o1);
            }
          }
        }
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const uint32_t at = __shfl_sync(~0u, of, 8 * b);
          if (at >= kSeg || at % kPer == 0) continue;
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            w[i] = (__shfl_sync(~0u, odd, 8 * b + 2 * i) & 0xFFFFu) | (__shfl_sync(~0u, odd, 8 * b + 2 * i + 1) << 16);
#pragma unroll
          for (int j = 0; j < kVecs; ++j)
            if (at / kPer == static_cast<uint32_t>(j * 32 + lane)) raw[j] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
  }

  // Whether [x, x + n) is of shard `t` (always, but in the checked build).
  __device__ static __forceinline__ bool inside(const ScoreParams& p, const LogitShard& t, uint64_t x, uint32_t n) {
    return in_bounds(reinterpret_cast<const void*>(x), n, t.base,
                     t.base + (p.rows - 1) * t.stride + static_cast<uint64_t>(t.end - t.first) * Elem<DT>::kBytes,
                     kSiteLogit);
  }
};

template <int DT>
__device__ __forceinline__ uint32_t vec_max(const uint4& v) {
  return Elem<DT>::max2(Elem<DT>::max2(v.x, v.y), Elem<DT>::max2(v.z, v.w));
}

// Element i of a vector, chosen at run time.
template <int DT>
__device__ __forceinline__ float pick(const uint4& v, int i) {
  if constexpr (DT == kF32) {
    return __uint_as_float(i < 2 ? (i == 0 ? v.x : v.y) : (i == 2 ? v.z : v.w));
  } else {
    const int h = i >> 1;
    const uint32_t w = h < 2 ? (h == 0 ? v.x : v.y) : (h == 2 ? v.z : v.w);
    return (i & 1) ? Elem<DT>::hi(w) : Elem<DT>::lo(w);
  }
}

// The entries of a segment that reach the bound, into a warp's own list: the
// slow way, for rows with many logits near or equal to the bound.  (Out of
// line: its code and registers are not the common path's.)
template <int DT>
__device__ __noinline__ void list_segment(const ScoreParams& p, uint64_t row, int seg, int lane, TopList& top,
                                          uint64_t* waiting) {
  using L = SegLoader<DT>;
  uint4 raw[L::kVecs];
  int r = 0;
  L::load(p, row, seg, lane, r, raw);
  const uint32_t e0 = static_cast<uint32_t>(seg) * L::kSeg;
#pragma unroll
  for (int j = 0; j < L::kVecs; ++j)
#pragma unroll 1
    for (int i = 0; i < L::kPer; ++i) {  // an entry of every lane at a time: at most 32 join the 31 that wait
      const float x = pick<DT>(raw[j], i);
      const bool take = x >= top.thr && e0 + L::index(j, i, lane) < p.vocab;
      const uint32_t who = __ballot_sync(~0u, take);
      if (who == 0) continue;
      if (take)
        waiting[top.count + __popc(who & ((1u << lane) - 1u))] =
            (static_cast<uint64_t>(ordered(x)) << 32) | (0xFFFFFFFFu - (e0 + L::index(j, i, lane)));
      top.count += __popc(who);
      if (top.count >= 32) flush_candidates(top, waiting, p.top, lane);
    }
}

// Two binary32 numbers, added and multiplied by one instruction each.
struct Two {
  uint64_t v;
};
__device__ __forceinline__ Two two(float a, float b) {
  Two r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void apart(const Two& x, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x.v));
}
__device__ __forceinline__ Two add2(const Two& a, const Two& b) {
  Two r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Two mul2(const Two& a, const Two& b) {
  Two r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ Two fma2(const Two& a, const Two& b, const Two& c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}

// s = sum 2^a, t = sum 2^a a over a lane's part of a segment, a = (x - m) c.
// 16-bit logits are first raised, two at a time, to `floor2` (two copies of a
// number far enough below m that 2^a is 0 there), so that a masked logit adds
// 0 and not 0 * -inf; CLAMP does it on every exponent instead.
template <int DT, bool CLAMP>
__device__ __forceinline__ void lane_sums(const uint4 (&raw)[SegLoader<DT>::kVecs], float m, float c, uint32_t floor2,
                                          float& s, float& t) {
  const Two nm = two(-m, -m), cc = two(c, c);
  Two s2[2] = {two(0.0f, 0.0f), two(0.0f, 0.0f)}, t2[2] = {two(0.0f, 0.0f), two(0.0f, 0.0f)};
#pragma unroll
  for (int j = 0; j < SegLoader<DT>::kVecs; ++j) {
    uint4 v = raw[j];
    if constexpr (!CLAMP && DT != kF32)
      v = make_uint4(Elem<DT>::max2(v.x, floor2), Elem<DT>::max2(v.y, floor2), Elem<DT>::max2(v.z, floor2),
                     Elem<DT>::max2(v.w, floor2));
    float x[SegLoader<DT>::kPer];
    unpack<DT>(v, x);
#pragma unroll
    for (int i = 0; i < SegLoader<DT>::kPer; i += 2) {
      Two a = mul2(add2(two(x[i], x[i + 1]), nm), cc);
      float a0, a1;
      apart(a, a0, a1);
      if constexpr (CLAMP || DT == kF32) {
        a0 = max_nan(a0, -400.0f);
        a1 = max_nan(a1, -400.0f);
        a = two(a0, a1);
      }
      const Two e = two(ex2(a0), ex2(a1));
      s2[(i >> 1) & 1] = add2(s2[(i >> 1) & 1], e);
      t2[(i >> 1) & 1] = fma2(e, a, t2[(i >> 1) & 1]);
    }
  }
  float a, b, d, e;
  apart(add2(s2[0], s2[1]), a, b);
  apart(add2(t2[0], t2[1]), d, e);
  s = a + b;
  t = d + e;
}

template <int DT, bool TOP>
__global__ __launch_bounds__(kScoreWarps * 32, 4) void dc_score_kernel(const __grid_constant__ ScoreParams p) {
  using L = SegLoader<DT>;
  extern __shared__ float part[];  // leader: m, s, t of every segment; then (TOP) this CTA's segments' m
  __shared__ __align__(16) uint64_t cand[TOP ? kScoreWarps : 1][64];
  __shared__ uint64_t lists[TOP ? kScoreWarps : 1][32];
  __shared__ uint64_t cta_lists[TOP ? kScoreMaxCluster : 1][32];
  __shared__ float4 maxima[TOP ? 32 : 1];  // at most 128 groups
  __shared__ float bound;
  __shared__ uint32_t cta_count;
  __shared__ float row_m, row_log_s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = static_cast<int>(blockDim.x >> 5);
  const uint32_t cl = static_cast<uint32_t>(p.cluster);
  const uint64_t row = blockIdx.x / cl;
  const int rank = static_cast<int>(blockIdx.x % cl);
  pdl_enter();
  if (cl > 1) cluster_arrive();  // the leader has started before anyone writes to it

  int64_t token = -1;
  float x_token = 0.0f;
  if (rank == 0 && threadIdx.x == 0) {
    token = ld_token(p.tokens, row, p.rows, p.tokens64 != 0);
    if (token >= 0 && token < static_cast<int64_t>(p.vocab)) {
      int q = 0;
      while (static_cast<int64_t>(p.shard[q].end) <= token) ++q;
      const LogitShard& sh = p.shard[q];
      const uint64_t a = sh.base + row * sh.stride + static_cast<uint64_t>(token - sh.first) * Elem<DT>::kBytes;
      if (in_bounds(reinterpret_cast<const void*>(a), Elem<DT>::kBytes, sh.base,
                    sh.base + (p.rows - 1) * sh.stride + static_cast<uint64_t>(sh.end - sh.first) * Elem<DT>::kBytes,
                    kSiteLogit))
        x_token = load_elem<DT>(a);
    }
  }

  const float c = p.inv_t * kLog2E;
  const uint32_t dst = leader_addr(smem_addr(part));
  float thread_max = neg_inf();
  if (TOP && threadIdx.x == 0) cta_count = 0;
  int r_shard = 0;
  bool waited = cl == 1;
  const int seg0 = rank * warps + warp, step = warps * static_cast<int>(cl);
  int last = -1;
  uint4 raw[L::kVecs];
  for (int seg = seg0; seg < p.nseg; seg += step) {
    last = seg;
    L::load(p, row, seg, lane, r_shard, raw);
    uint32_t mw = vec_max<DT>(raw[0]);
#pragma unroll
    for (int j = 1; j < L::kVecs; ++j) mw = Elem<DT>::max2(mw, vec_max<DT>(raw[j]));
    const float lane_max = word_max<DT>(mw);
    thread_max = fmaxf(thread_max, lane_max);  // (a lane with NaN has no say)
    float m = lane_max;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(~0u, m, o));
    const float ref = m == neg_inf() ? 0.0f : m;
    float s, t;
    if constexpr (DT == kF32) {
      lane_sums<DT, true>(raw, ref, c, 0u, s, t);
    } else {
      // 2^-400 is 0 in binary32; the step below the rounded number makes sure that it is low enough
      // (and its exponent finite: at very low temperatures one step of the type may be beyond binary32)
      const uint32_t floor2 = Elem<DT>::below2(ref - 400.0f / c);
      if (floor2 != Elem<DT>::kNegInfWord && (Elem<DT>::lo(floor2) - ref) * c >= -FLT_MAX)
        lane_sums<DT, false>(raw, ref, c, floor2, s, t);
      else lane_sums<DT, true>(raw, ref, c, 0u, s, t);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s += __shfl_xor_sync(~0u, s, o);
      t += __shfl_xor_sync(~0u, t, o);
    }
    if (!waited) {
      cluster_wait();
      waited = true;
    }
    if (lane < 3) {
      const float v = lane == 0 ? m : lane == 1 ? s : t;
      st_cluster(dst + static_cast<uint32_t>(seg * 3 + lane) * 4, __float_as_uint(v));
    }
    if (TOP && lane == 0) part[3 * p.nseg + seg] = m;
  }
  if (!waited) cluster_wait();

  if constexpr (TOP) {
    // A bound for the k-th largest logit of this CTA's part of the row: the
    // k-th largest of the maxima of groups of lanes, of which k are at least
    // that.  (64 groups or more, of 4 lanes, 2 or 1 as there are warps with
    // something to look at; one warp's 32 lanes.)  A second look at the
    // segments that reach it (from L2; the last one is still in registers)
    // then meets little more than the k entries that are wanted: 20 of 64
    // groups hold about the 24 largest.
    const int busy = min(warps, p.nseg - rank * warps);  // warps with a segment (may be negative: none)
    const int wide = busy >= 8 ? 4 : busy >= 4 ? 2 : 1, groups = busy > 0 ? (busy * 32) >> (wide >> 1) : 0;
    float v = thread_max;
    for (int o = 1; o < wide; o <<= 1) v = fmaxf(v, __shfl_xor_sync(~0u, v, o));
    float* const mx = reinterpret_cast<float*>(maxima);
    if (warp < busy && (lane & (wide - 1)) == 0) mx[static_cast<int>(threadIdx.x) >> (wide >> 1)] = v;
    if (threadIdx.x < 32) lists[0][lane] = 0;
    __syncthreads();
    {
      // a group's place: 4, 2 or 1 threads compare it with a part of the others each
      const int share = 4 * groups <= static_cast<int>(blockDim.x) ? 4 : 2 * groups <= static_cast<int>(blockDim.x) ? 2 : 1;
      const int t = static_cast<int>(threadIdx.x) >> (share >> 1), part_of = static_cast<int>(threadIdx.x) & (share - 1);
      const float mine = t < groups ? mx[t] : 0.0f;
      int rank_of = 0;  // groups before this one, equal ones by their number
      for (int i = part_of; i < groups / 4; i += share) {
        const float4 q = maxima[i];
        const int n = t - 4 * i;
        rank_of += (q.x > mine || (q.x == mine && n > 0)) + (q.y > mine || (q.y == mine && n > 1)) +
                   (q.z > mine || (q.z == mine && n > 2)) + (q.w > mine || (q.w == mine && n > 3));
      }
      for (int o = 1; o < share; o <<= 1) rank_of += __shfl_xor_sync(~0u, rank_of, o);
      if (t < groups && part_of == 0 && rank_of == p.top - 1) bound = mine;
    }
    __syncthreads();
    const float thr = bound;
    // From the last segment back: begin(n) with the candidates of a segment
    // that each lane has, then put(key) for each of them.  Their keys are the
    // entries that reach the bound.
    auto scan = [&](auto begin, auto put) {
      for (int seg = last; seg >= seg0 && seg >= 0; seg -= step) {
        if (part[3 * p.nseg + seg] < thr) continue;
        int r = 0;
        if (seg != last) L::load(p, row, seg, lane, r, raw);
        const uint32_t e0 = static_cast<uint32_t>(seg) * L::kSeg;
        static_assert(L::kVecs * L::kPer <= 64, "a bit per entry");
        uint32_t bits[2] = {0, 0};
#pragma unroll
        for (int j = 0; j < L::kVecs; ++j) {
          if (!__any_sync(~0u, !(word_max<DT>(vec_max<DT>(raw[j])) < thr))) continue;
          float x[L::kPer];
          unpack<DT>(raw[j], x);
          uint32_t mask = 0;
#pragma unroll
          for (int i = 0; i < L::kPer; ++i)
            if (x[i] >= thr && e0 + L::index(j, i, lane) < p.vocab) mask |= 1u << i;
          bits[j * L::kPer / 32] |= mask << (j * L::kPer % 32);
        }
        begin(__popc(bits[0]) + __popc(bits[1]));
#pragma unroll
        for (int j = 0; j < L::kVecs; ++j) {
          uint32_t mask = (bits[j * L::kPer / 32] >> (j * L::kPer % 32)) & ((1u << L::kPer) - 1u);
          while (mask != 0) {
            const int i = __ffs(static_cast<int>(mask)) - 1;
            mask &= mask - 1;
            put((static_cast<uint64_t>(ordered(pick<DT>(raw[j], i))) << 32) | (0xFFFFFFFFu - (e0 + L::index(j, i, lane))));
          }
        }
      }
    };
    // most often the CTA's candidates are few: each is ranked among all
    uint32_t at = 0;
    scan(
        [&](uint32_t mine) {
          // the lanes' places: from a vote where no lane has two, else a sum over the lanes
          const uint32_t who = __ballot_sync(~0u, mine != 0);
          uint32_t before = __popc(who & ((1u << lane) - 1u)), all = __popc(who);
          if (__any_sync(~0u, mine > 1)) {
            uint32_t upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const uint32_t x = __shfl_up_sync(~0u, upto, o);
              if (lane >= o) upto += x;
            }
            before = upto - mine;
            all = __shfl_sync(~0u, upto, 31);
          }
          if (lane == 0 && all != 0) at = atomicAdd(&cta_count, all);
          at = __shfl_sync(~0u, at, 0) + before;
        },
        [&](uint64_t key) {
          if (at < kFewCandidates) (&cand[0][0])[at] = key;
          ++at;
        });
    __syncthreads();
    const uint32_t found = cta_count;
    if (found <= kFewCandidates) {
      const ulonglong2* all = reinterpret_cast<const ulonglong2*>(&cand[0][0]);
      for (uint32_t t = threadIdx.x; t < found; t += blockDim.x) {
        const uint64_t key = (&cand[0][0])[t];
        uint32_t place = 0;
#pragma unroll 4
        for (uint32_t i = 0; i < (found + 1) / 2; ++i) {  // (keys are distinct; an odd one's neighbour does not count)
          const ulonglong2 k2 = all[i];
          place += (k2.x > key ? 1u : 0u) + (k2.y > key && 2 * i + 1 < found ? 1u : 0u);
        }
        if (place < 32) lists[0][place] = key;
      }
      __syncthreads();
    } else {
      // many logits near or equal to the bound: every warp keeps its own list
      __syncthreads();
      TopList top{0, 0, thr};
      for (int seg = seg0; seg < p.nseg; seg += step)
        if (!(part[3 * p.nseg + seg] < thr)) list_segment<DT>(p, row, seg, lane, top, cand[warp]);
      if (top.count) flush_candidates(top, cand[warp], p.top, lane);
      lists[warp][lane] = top.key;
      __syncthreads();
      for (int n = warps / 2; n > 0; n >>= 1) {
        if (warp < n) {
          top.key = merge_desc(top.key, lists[warp + n][lane], lane);
          lists[warp][lane] = top.key;
        }
        __syncthreads();
      }
    }
    if (warp == 0) st_cluster64(leader_addr(smem_addr(&cta_lists[rank][lane])), lists[0][lane]);
  }
  if (cl > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  if (rank != 0 || (!TOP && warp != 0)) return;

  // the row's segments: the largest logit, then lane l folds segments l,
  // l + 32, ... in order and the lanes join in a fixed exchange
  const bool scored = warp == 0;
  if (scored) {
    float M = neg_inf();
    for (int i = lane; i < p.nseg; i += 32) M = max_nan(M, part[3 * i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = max_nan(M, __shfl_xor_sync(~0u, M, o));
    float S = 0.0f, U = 0.0f;
    for (int i = lane; i < p.nseg; i += 32) {
      const float mi = part[3 * i];
      if (mi == neg_inf()) continue;
      const float d = max_nan((mi - M) * c, -400.0f);
      const float w = ex2(d), si = part[3 * i + 1];
      S = __fmaf_rn(si, w, S);
      U = __fmaf_rn(w, __fmaf_rn(si, d, part[3 * i + 2]), U);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      S += __shfl_xor_sync(~0u, S, o);
      U += __shfl_xor_sync(~0u, U, o);
    }
    const bool none = M == neg_inf();  // every entry of the row is masked
    const float log_s = logf(S);
    if (lane == 0) {
      row_m = M;
      row_log_s = log_s;
      float lp;
      if (token < 0) lp = 0.0f;
      else if (token >= static_cast<int64_t>(p.vocab)) lp = __int_as_float(0x7FC00000);
      else if (none) lp = neg_inf();
      else lp = __fmaf_rn(x_token - M, p.inv_t, -log_s);
      st_entry<float>(p.logprobs, row, p.rows, lp, kSiteScore);
      if (p.lse) st_entry<float>(p.lse, row, p.rows, none ? neg_inf() : __fmaf_rn(M, p.inv_t, log_s), kSiteScore);
      if (p.entropy) st_entry<float>(p.entropy, row, p.rows, none ? 0.0f : log_s - U / S * kLn2, kSiteScore);
    }
  }
  if constexpr (TOP) {
    // a key's place among all lists: its place in its own and how many of
    // each other one are larger
    static_assert(kScoreMaxCluster <= kScoreWarps, "a thread per key: clusters have CTAs of all warps");
    uint64_t key = 0;
    uint32_t place = lane;
    if (warp < static_cast<int>(cl)) {
      key = cta_lists[warp][lane];
      for (int i = 0; i < static_cast<int>(cl); ++i)
        if (i != warp) place += larger_in(cta_lists[i], key);
    }
    const uint32_t filled = __syncthreads_count(key != 0);  // (row_m and row_log_s are visible after this)
    // places that no number fills: token -1
    const bool fill = threadIdx.x < static_cast<uint32_t>(p.top) && threadIdx.x >= filled;
    const float M = row_m;
    for (int k = 0; k < 2; ++k) {
      if (k == 0 ? key == 0 || place >= static_cast<uint32_t>(p.top) : !fill) continue;
      const uint64_t at = row * static_cast<uint64_t>(p.top) + (k == 0 ? place : threadIdx.x);
      const int64_t id = k == 0 ? static_cast<int64_t>(0xFFFFFFFFu - static_cast<uint32_t>(key)) : -1;
      const float x = from_ordered(static_cast<uint32_t>(key >> 32));
      float lp = __fmaf_rn(x - M, p.inv_t, -row_log_s);
      if (M == neg_inf()) lp = neg_inf();
      if (k == 1) lp = __int_as_float(0x7FC00000);
      const uint64_t n = p.rows * static_cast<uint64_t>(p.top);
      if (p.top_logprobs) st_entry<float>(p.top_logprobs, at, n, lp, kSiteTop);
      if (p.top_tokens && p.top64) st_entry<int64_t>(p.top_tokens, at, n, id, kSiteTop);
      if (p.top_tokens && !p.top64) st_entry<int32_t>(p.top_tokens, at, n, static_cast<int32_t>(id), kSiteTop);
    }
  }
}

// ---------------------------------------------------------- the gradient ---
// What a row's gradient needs: log p_i = x_i / T - lse, rounded once, and
// d_i = p_i (nh log p_i + ngh), with g added at the token's column.
struct RowTerms {
  float inv_t, lse;
  float g;         // upstream gradient of the log probability, times 1/T
  float nh, ngh;   // -h / T and -(g + h H) / T
  uint32_t token;  // column of the token in this shard, ~0u if it is not here
};

// Pairs of elements share products and sums.  exp(-200) is 0 in binary32: the
// floor keeps 0 * -inf out.
template <int N>
__device__ __forceinline__ void grad_of(const RowTerms& t, float (&x)[N]) {
  const Two inv = two(t.inv_t, t.inv_t), nl = two(-t.lse, -t.lse), nh = two(t.nh, t.nh), ngh = two(t.ngh, t.ngh),
            l2e = two(kLog2E, kLog2E);
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    float a, b;
    apart(fma2(two(x[i], x[i + 1]), inv, nl), a, b);
    const Two logp = two(max_nan(a, -200.0f), max_nan(b, -200.0f));
    apart(mul2(logp, l2e), a, b);
    apart(mul2(two(ex2(a), ex2(b)), fma2(nh, logp, ngh)), x[i], x[i + 1]);
  }
}

template <int DT>
__global__ __launch_bounds__(kGradThreads) void dc_score_grad_kernel(const __grid_constant__ GradParams p) {
  constexpr int kPer = Elem<DT>::kPerVec;
  constexpr int kB = Elem<DT>::kBytes;
  pdl_enter();
  const uint64_t total = p.rows * p.chunks;
  for (uint64_t item = blockIdx.x; item < total; item += gridDim.x) {
    const uint64_t row = item / p.chunks;
    const uint32_t chunk = static_cast<uint32_t>(item - row * p.chunks);
    int q = 0;
    while (q + 1 < p.P && p.shard[q + 1].chunk0 <= chunk) ++q;
    const GradShard& sh = p.shard[q];
    const uint32_t k = chunk - sh.chunk0;
    const uint64_t in = sh.in + row * sh.in_stride, out = sh.out + row * sh.out_stride;
    const uint64_t ilo = hull_lo(in), ihi = hull_hi(in, static_cast<uint64_t>(sh.width) * kB);
    const uint64_t olo = out, ohi = out + static_cast<uint64_t>(sh.width) * kB;
    const uint32_t head = min(sh.width, static_cast<uint32_t>((-out) & 15u) / kB);
    const uint32_t nvec = (sh.width - head) / kPer;
    const uint32_t tail = head + nvec * kPer;
    // the logits first: the row's numbers arrive meanwhile
    uint4 raw[kGradVecs];
#pragma unroll
    for (int j = 0; j < kGradVecs; ++j) {
      const uint32_t v = k * kGradChunk + j * kGradThreads + threadIdx.x;
      if (v >= nvec) continue;
      const uint64_t a = in + static_cast<uint64_t>(head + v * kPer) * kB;
      const uint32_t s = static_cast<uint32_t>(a & 15u);
      const uint4* b = reinterpret_cast<const uint4*>(a - s);
      if (!in_bounds(b, s ? 32 : 16, ilo, ihi, kSiteGradIn)) continue;
      raw[j] = s == 0 ? ld_stream(b) : realign16_sel(ld_cached(b), ld_cached(b + 1), s);
    }
    RowTerms t;
    const int64_t token = ld_token(p.tokens, row, p.rows, p.tokens64 != 0);
    const float lse = ld_entry<float>(p.lse, row, p.rows, kSiteRow);
    t.g = p.grad_logprobs ? ld_entry<float>(p.grad_logprobs, row, p.rows, kSiteRow) * p.inv_t : 0.0f;
    if (token < 0) t.g = 0.0f;
    if (token >= static_cast<int64_t>(p.vocab)) t.g = __int_as_float(0x7FC00000);
    const float h = p.grad_entropy ? ld_entry<float>(p.grad_entropy, row, p.rows, kSiteRow) * p.inv_t : 0.0f;
    t.nh = -h;
    t.ngh = -(t.g + (p.grad_entropy ? h * ld_entry<float>(p.entropy, row, p.rows, kSiteRow) : 0.0f));
    t.inv_t = p.inv_t;
    // a row of nothing but -inf, or but the lowest of BF16 or FP32 beside which lse loses the row's
    // log of a count, has no gradient: p = 0 everywhere (FP16's lowest, -65504, is a number like others)
    const bool none = lse <= -1e30f;
    t.lse = none ? __int_as_float(0x7F800000) : lse;
    t.token = !none && token >= static_cast<int64_t>(sh.first) && token < static_cast<int64_t>(sh.first) + sh.width
                  ? static_cast<uint32_t>(token - static_cast<int64_t>(sh.first)) : ~0u;
    // columns of the vocabulary; the rest of the row is padding, whose gradient is 0
    const uint32_t real = p.vocab <= sh.first ? 0u : min(sh.width, p.vocab - sh.first);
    if (k == 0) {  // the elements outside the 16-byte vectors
      uint32_t col = threadIdx.x;
      if (col >= head) col = tail + (col - head);
      if (col < sh.width && threadIdx.x < head + kPer &&
          in_bounds(reinterpret_cast<const void*>(out + col * static_cast<uint64_t>(kB)), kB, olo, ohi, kSiteGradOut)) {
        float x[2] = {0.0f, 0.0f};
        if (col < real) {
          x[0] = load_elem<DT>(in + col * static_cast<uint64_t>(kB));
          grad_of(t, x);
          if (col == t.token) x[0] += t.g;
        }
        store_elem<DT>(out + col * static_cast<uint64_t>(kB), x[0]);
      }
    }
#pragma unroll
    for (int j = 0; j < kGradVecs; ++j) {
      const uint32_t v = k * kGradChunk + j * kGradThreads + threadIdx.x;
      if (v >= nvec) continue;
      const uint32_t col = head + v * kPer;
      float x[kPer];
      unpack<DT>(raw[j], x);
      grad_of(t, x);
      if (t.token - col < kPer) {  // (once a row)
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (col + i == t.token) x[i] += t.g;
      }
      if (col + kPer > real) {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
          if (col + i >= real) x[i] = 0.0f;
      }
      const uint64_t a = out + static_cast<uint64_t>(col) * kB;
      if (in_bounds(reinterpret_cast<const void*>(a), 16, olo, ohi, kSiteGradOut))
        st16(reinterpret_cast<uint4*>(a), repack<DT>(x));
    }
  }
}

template <int DT, bool TOP>
cudaError_t launch_score_t(const ScoreParams& p, int grid, bool pdl, cudaStream_t s) {
  const size_t smem = static_cast<size_t>(p.nseg) * (TOP ? 16 : 12);
  if (smem > 32 * 1024) {  // vocabularies of millions: more than a CTA may have unasked
    const cudaError_t e = cudaFuncSetAttribute(dc_score_kernel<DT, TOP>, cudaFuncAttributeMaxDynamicSharedMemorySize, 64 * 1024);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(p.warps) * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  int n = 0;
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
  cfg.numAttrs = static_cast<unsigned>(n);
  return cudaLaunchKernelEx(&cfg, dc_score_kernel<DT, TOP>, p);
}

}  // namespace

cudaError_t launch_score(const ScoreParams& p, int dtype, bool pdl, cudaStream_t s, int* grid) {
  *grid = static_cast<int>(p.rows * static_cast<uint64_t>(p.cluster));
  const bool top = p.top > 0;
  switch (dtype) {
    case kF16: return top ? launch_score_t<kF16, true>(p, *grid, pdl, s) : launch_score_t<kF16, false>(p, *grid, pdl, s);
    case kF32: return top ? launch_score_t<kF32, true>(p, *grid, pdl, s) : launch_score_t<kF32, false>(p, *grid, pdl, s);
    default: return top ? launch_score_t<kBF16, true>(p, *grid, pdl, s) : launch_score_t<kBF16, false>(p, *grid, pdl, s);
  }
}

cudaError_t launch_score_grad(const GradParams& p, int dtype, bool pdl, cudaStream_t s, int* grid) {
  const uint64_t total = p.rows * p.chunks;
  *grid = static_cast<int>(total < 0x7FFFFFFFull ? total : 0x7FFFFFFFull);
  switch (dtype) {
    case kF16: return launch_ex(dc_score_grad_kernel<kF16>, *grid, kGradThreads, pdl, s, p);
    case kF32: return launch_ex(dc_score_grad_kernel<kF32>, *grid, kGradThreads, pdl, s, p);
    default: return launch_ex(dc_score_grad_kernel<kBF16>, *grid, kGradThreads, pdl, s, p);
  }
}

DC_BOUNDS_READER(take_bounds_logprobs)

}  // namespace dc
