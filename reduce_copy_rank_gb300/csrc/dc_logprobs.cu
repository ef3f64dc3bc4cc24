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
// Bound: memory.  The logits are read once (and the gradient written once);
// an element costs about eight instructions and one exponential.
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
// The k-th largest of the lanes' values (k = 1..32).
__device__ __forceinline__ float kth_of_lanes(float v, int k, int lane) {
#pragma unroll
  for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
    for (int j = size >> 1; j > 0; j >>= 1) {
      const float o = __shfl_xor_sync(~0u, v, j);
      v = (((lane & j) == 0) == ((lane & size) == 0)) ? fmaxf(v, o) : fminf(v, o);
    }
  return __shfl_sync(~0u, v, k - 1);
}

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

// --------------------------------------------------------- one segment ---
template <int DT>
struct SegLoader {
  static constexpr int kPer = Elem<DT>::kPerVec;
  static constexpr int kVecs = kVocabSeg / kPer / 32;  // 16-byte vectors a lane holds

  // Lane `lane`'s vectors of segment `seg` of row `row`: vector j holds entries
  // (seg * kVocabSeg) + (j * 32 + lane) * kPer ...; entries past the vocabulary read -inf.
  // r: the shard of the previous segment of this warp (segments come in order).
  __device__ static __forceinline__ void load(const ScoreParams& p, uint64_t row, int seg, int lane, int& r,
                                              uint4 (&raw)[kVecs]) {
    const uint32_t e0 = static_cast<uint32_t>(seg) * kVocabSeg;
    while (p.shard[r].end <= e0) ++r;
    const LogitShard& sh = p.shard[r];
    const uint64_t lo = hull_lo(sh.base);
    const uint64_t hi =
        hull_hi(sh.base, (p.rows - 1) * sh.stride + static_cast<uint64_t>(sh.end - sh.first) * Elem<DT>::kBytes);
    if (e0 + kVocabSeg <= sh.end) {
      const uint64_t a = sh.base + row * sh.stride + static_cast<uint64_t>(e0 - sh.first) * Elem<DT>::kBytes +
                         static_cast<uint64_t>(lane) * 16;
      const uint32_t s = static_cast<uint32_t>(a & 15u);
      const uint4* b = reinterpret_cast<const uint4*>(a - s);
      if (s == 0) {
#pragma unroll
        for (int j = 0; j < kVecs; ++j)
          raw[j] = in_bounds(b + 32 * j, 16, lo, hi, kSiteLogit) ? ld_nc_stream(b + 32 * j) : uint4{};
      } else {
#pragma unroll
        for (int j = 0; j < kVecs; ++j) {
          const uint4 x = in_bounds(b + 32 * j, 16, lo, hi, kSiteLogit) ? ld_nc_cached(b + 32 * j) : uint4{};
          const uint4 y = in_bounds(b + 32 * j + 1, 16, lo, hi, kSiteLogit) ? ld_nc_cached(b + 32 * j + 1) : uint4{};
          raw[j] = realign16_sel(x, y, s);
        }
      }
      return;
    }
    // a segment that crosses shards or ends the vocabulary
#pragma unroll
    for (int j = 0; j < kVecs; ++j) {
      const uint32_t e = e0 + static_cast<uint32_t>(j * 32 + lane) * kPer;
      raw[j] = make_uint4(Elem<DT>::kNegInfWord, Elem<DT>::kNegInfWord, Elem<DT>::kNegInfWord, Elem<DT>::kNegInfWord);
      if (e >= p.vocab) continue;
      int q = r;
      while (p.shard[q].end <= e) ++q;
      uint64_t a = p.shard[q].base + row * p.shard[q].stride +
                   static_cast<uint64_t>(e - p.shard[q].first) * Elem<DT>::kBytes;
      if (e + kPer <= p.shard[q].end && (a & 15u) == 0) {
        const LogitShard& t = p.shard[q];
        if (in_bounds(reinterpret_cast<const void*>(a), 16, t.base,
                      t.base + (p.rows - 1) * t.stride + static_cast<uint64_t>(t.end - t.first) * Elem<DT>::kBytes,
                      kSiteLogit))
          raw[j] = ld_nc_stream(reinterpret_cast<const uint4*>(a));
        continue;
      }
      uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        if (e + i >= p.vocab) break;
        while (p.shard[q].end <= e + i) ++q;
        const LogitShard& t = p.shard[q];
        a = t.base + row * t.stride + static_cast<uint64_t>(e + i - t.first) * Elem<DT>::kBytes;
        if (!in_bounds(reinterpret_cast<const void*>(a), Elem<DT>::kBytes, t.base,
                       t.base + (p.rows - 1) * t.stride + static_cast<uint64_t>(t.end - t.first) * Elem<DT>::kBytes,
                       kSiteLogit))
          continue;
        if constexpr (DT == kF32) {
          w[i] = *reinterpret_cast<const uint32_t*>(a);
        } else {
          const uint32_t h = *reinterpret_cast<const uint16_t*>(a);
          w[i / 2] = (i & 1) ? (w[i / 2] & 0x0000FFFFu) | (h << 16) : (w[i / 2] & 0xFFFF0000u) | h;
        }
      }
      raw[j] = make_uint4(w[0], w[1], w[2], w[3]);
    }
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

template <int DT, bool TOP>
__global__ __launch_bounds__(kScoreWarps * 32) void dc_score_kernel(const __grid_constant__ ScoreParams p) {
  using L = SegLoader<DT>;
  extern __shared__ float part[];  // leader: m, s, t of every segment
  __shared__ uint64_t cand[TOP ? kScoreWarps : 1][64];
  __shared__ uint64_t lists[TOP ? kScoreWarps : 1][32];
  __shared__ uint64_t cta_lists[TOP ? kScoreMaxCluster : 1][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
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
  TopList top{0, 0, neg_inf()};
  int r_shard = 0;
  bool waited = cl == 1;
  const int step = kScoreWarps * static_cast<int>(cl);
  for (int seg = rank * kScoreWarps + warp; seg < p.nseg; seg += step) {
    uint4 raw[L::kVecs];
    L::load(p, row, seg, lane, r_shard, raw);
    uint32_t mw = vec_max<DT>(raw[0]);
#pragma unroll
    for (int j = 1; j < L::kVecs; ++j) mw = Elem<DT>::max2(mw, vec_max<DT>(raw[j]));
    const float lane_max = word_max<DT>(mw);
    float m = lane_max;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(~0u, m, o));
    const bool empty = m == neg_inf();
    const float r = empty ? 0.0f : m;
    float s0 = 0.0f, s1 = 0.0f, t0 = 0.0f, t1 = 0.0f;
#pragma unroll
    for (int j = 0; j < L::kVecs; ++j) {
      float x[L::kPer];
      unpack<DT>(raw[j], x);
#pragma unroll
      for (int i = 0; i < L::kPer; i += 2) {
        // 2^-400 is 0 in binary32; the floor keeps 0 * -inf out of t
        const float a0 = max_nan((x[i] - r) * c, -400.0f);
        const float a1 = max_nan((x[i + 1] - r) * c, -400.0f);
        const float e0 = ex2(a0), e1 = ex2(a1);
        s0 += e0;
        s1 += e1;
        t0 = __fmaf_rn(e0, a0, t0);
        t1 = __fmaf_rn(e1, a1, t1);
      }
    }
    float s = s0 + s1, t = t0 + t1;
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
    if constexpr (TOP) {
      // k lanes hold a value of at least the k-th largest lane maximum
      if (m == m) top.thr = fmaxf(top.thr, kth_of_lanes(lane_max, p.top, lane));
      const uint32_t e0 = static_cast<uint32_t>(seg) * kVocabSeg;
#pragma unroll
      for (int j = 0; j < L::kVecs; ++j) {
        const float vm = word_max<DT>(vec_max<DT>(raw[j]));
        if (!__any_sync(~0u, !(vm < top.thr))) continue;
        const uint32_t ev = e0 + static_cast<uint32_t>(j * 32 + lane) * L::kPer;
        float x[L::kPer];
        unpack<DT>(raw[j], x);
        uint32_t mask = 0;
#pragma unroll
        for (int i = 0; i < L::kPer; ++i)
          if (x[i] >= top.thr && ev + i < p.vocab) mask |= 1u << i;
        while (true) {
          const uint32_t who = __ballot_sync(~0u, mask != 0);
          if (who == 0) break;
          if (mask != 0) {
            const int i = __ffs(static_cast<int>(mask)) - 1;
            mask &= mask - 1;
            cand[warp][top.count + __popc(who & ((1u << lane) - 1u))] =
                (static_cast<uint64_t>(ordered(pick<DT>(raw[j], i))) << 32) | (0xFFFFFFFFu - (ev + i));
          }
          top.count += __popc(who);
          if (top.count >= 32) flush_candidates(top, cand[warp], p.top, lane);
        }
      }
    }
  }
  if (!waited) cluster_wait();

  if constexpr (TOP) {
    if (top.count) flush_candidates(top, cand[warp], p.top, lane);
    lists[warp][lane] = top.key;
    __syncthreads();
#pragma unroll
    for (int n = kScoreWarps / 2; n > 0; n >>= 1) {
      if (warp < n) {
        top.key = merge_desc(top.key, lists[warp + n][lane], lane);
        lists[warp][lane] = top.key;
      }
      __syncthreads();
    }
    if (warp == 0) st_cluster64(leader_addr(smem_addr(&cta_lists[rank][lane])), top.key);
  }
  if (cl > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  if (rank != 0 || warp != 0) return;

  // the row's segments: the largest logit, then lane l folds segments l,
  // l + 32, ... in order and the lanes join in a fixed exchange
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
    float lp;
    if (token < 0) lp = 0.0f;
    else if (token >= static_cast<int64_t>(p.vocab)) lp = __int_as_float(0x7FC00000);
    else if (none) lp = neg_inf();
    else lp = __fmaf_rn(x_token - M, p.inv_t, -log_s);
    st_entry<float>(p.logprobs, row, p.rows, lp, kSiteScore);
    if (p.lse) st_entry<float>(p.lse, row, p.rows, none ? neg_inf() : __fmaf_rn(M, p.inv_t, log_s), kSiteScore);
    if (p.entropy) st_entry<float>(p.entropy, row, p.rows, none ? 0.0f : log_s - U / S * kLn2, kSiteScore);
  }
  if constexpr (TOP) {
    uint64_t key = cta_lists[0][lane];
    for (int i = 1; i < static_cast<int>(cl); ++i) key = merge_desc(key, cta_lists[i][lane], lane);
    if (lane < p.top) {
      const uint64_t at = row * static_cast<uint64_t>(p.top) + lane;
      const int64_t id = key == 0 ? -1 : static_cast<int64_t>(0xFFFFFFFFu - static_cast<uint32_t>(key));
      const float x = from_ordered(static_cast<uint32_t>(key >> 32));
      float lp = __fmaf_rn(x - M, p.inv_t, -log_s);
      if (none) lp = neg_inf();
      if (key == 0) lp = __int_as_float(0x7FC00000);
      const uint64_t n = p.rows * static_cast<uint64_t>(p.top);
      if (p.top_logprobs) st_entry<float>(p.top_logprobs, at, n, lp, kSiteTop);
      if (p.top_tokens && p.top64) st_entry<int64_t>(p.top_tokens, at, n, id, kSiteTop);
      if (p.top_tokens && !p.top64) st_entry<int32_t>(p.top_tokens, at, n, static_cast<int32_t>(id), kSiteTop);
    }
  }
}

// ---------------------------------------------------------- the gradient ---
struct RowTerms {
  float inv_t, lse; // log p_i = x_i / T - lse, rounded once
  float g, h;       // upstream gradients, times 1/T
  float ghH;        // g + h H
  int64_t token;    // column of the token in this shard, or out of its range
  bool zero;        // a row of nothing but masks (-inf or the type's lowest): no gradient
};

// (1/T) [ g (1[i=y] - p) - h p (log p + H) ]
template <int DT>
__device__ __forceinline__ float grad_of(const RowTerms& t, float x, int64_t col) {
  // exp(-200) is 0 in binary32; the floor keeps 0 * -inf out
  const float logp = max_nan(__fmaf_rn(x, t.inv_t, -t.lse), -200.0f);
  const float p = ex2(logp * kLog2E);
  float d = -p * __fmaf_rn(t.h, logp, t.ghH);
  if (col == t.token) d += t.g;
  return t.zero ? 0.0f : d;
}

template <int DT>
__global__ __launch_bounds__(kGradThreads) void dc_score_grad_kernel(const __grid_constant__ GradParams p) {
  constexpr int kPer = Elem<DT>::kPerVec;
  constexpr int kB = Elem<DT>::kBytes;
  pdl_enter();
  const uint64_t total = p.rows * p.chunks;
  for (uint64_t item = blockIdx.x; item < total; item += gridDim.x) {
    const uint64_t row = item / p.chunks;
    const uint32_t chunk = static_cast<uint32_t>(item % p.chunks);
    int q = 0;
    while (q + 1 < p.P && p.shard[q + 1].chunk0 <= chunk) ++q;
    const GradShard& sh = p.shard[q];
    const uint32_t k = chunk - sh.chunk0;
    RowTerms t;
    const int64_t token = ld_token(p.tokens, row, p.rows, p.tokens64 != 0);
    const float lse = ld_entry<float>(p.lse, row, p.rows, kSiteRow);
    t.g = p.grad_logprobs ? ld_entry<float>(p.grad_logprobs, row, p.rows, kSiteRow) * p.inv_t : 0.0f;
    if (token < 0) t.g = 0.0f;
    if (token >= static_cast<int64_t>(p.vocab)) t.g = __int_as_float(0x7FC00000);
    t.h = p.grad_entropy ? ld_entry<float>(p.grad_entropy, row, p.rows, kSiteRow) * p.inv_t : 0.0f;
    t.ghH = t.g + (p.grad_entropy ? t.h * ld_entry<float>(p.entropy, row, p.rows, kSiteRow) : 0.0f);
    t.inv_t = p.inv_t;
    t.lse = lse;
    t.token = token < 0 ? -1 : token - static_cast<int64_t>(sh.first);
    t.zero = lse <= -1e30f;
    const uint64_t in = sh.in + row * sh.in_stride, out = sh.out + row * sh.out_stride;
    // columns of the vocabulary; the rest of the row is padding, whose gradient is 0
    const uint32_t real = p.vocab <= sh.first ? 0u : min(sh.width, p.vocab - sh.first);
    const uint64_t ilo = hull_lo(in), ihi = hull_hi(in, static_cast<uint64_t>(sh.width) * kB);
    const uint64_t olo = out, ohi = out + static_cast<uint64_t>(sh.width) * kB;
    const uint32_t head = min(sh.width, static_cast<uint32_t>((-out) & 15u) / kB);
    const uint32_t nvec = (sh.width - head) / kPer;
    const uint32_t tail = head + nvec * kPer;
    if (k == 0) {  // the elements outside the 16-byte vectors
      uint32_t col = threadIdx.x;
      if (col >= head) col = tail + (col - head);
      if (col < sh.width && threadIdx.x < head + kPer &&
          in_bounds(reinterpret_cast<const void*>(out + col * static_cast<uint64_t>(kB)), kB, olo, ohi, kSiteGradOut))
        store_elem<DT>(out + col * static_cast<uint64_t>(kB),
                       col < real ? grad_of<DT>(t, load_elem<DT>(in + col * static_cast<uint64_t>(kB)), col) : 0.0f);
    }
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
#pragma unroll
    for (int j = 0; j < kGradVecs; ++j) {
      const uint32_t v = k * kGradChunk + j * kGradThreads + threadIdx.x;
      if (v >= nvec) continue;
      const uint32_t col = head + v * kPer;
      float x[kPer];
      unpack<DT>(raw[j], x);
#pragma unroll
      for (int i = 0; i < kPer; ++i) x[i] = col + i < real ? grad_of<DT>(t, x[i], col + i) : 0.0f;
      const uint64_t a = out + static_cast<uint64_t>(col) * kB;
      if (in_bounds(reinterpret_cast<const void*>(a), 16, olo, ohi, kSiteGradOut))
        st16(reinterpret_cast<uint4*>(a), repack<DT>(x));
    }
  }
}

template <int DT, bool TOP>
cudaError_t launch_score_t(const ScoreParams& p, int grid, bool pdl, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kScoreWarps * 32);
  cfg.dynamicSmemBytes = static_cast<size_t>(p.nseg) * 12;
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
