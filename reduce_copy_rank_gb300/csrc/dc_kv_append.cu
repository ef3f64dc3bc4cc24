// Appending keys and values to a paged cache, the position rotation applied
// on the way (and to the queries of the same tokens).
//
// Mathematics.  A pair (a, b) of a head's first `rot` elements at position t
// becomes (a cos - b sin, b cos + a sin), with the pair's cos and sin from
// row t of a table; pairs are elements (i, i + rot/2), or (2i, 2i + 1) when
// interleaved.  Products and sums in binary32, one rounding to the element
// type.  Other elements and the values are copied.
//
// Bound: memory (every element is read and written once) for prompts, one
// launch's latency for single tokens.  A CTA takes one token (or a share of
// it when there are few): a thread owns one position in the head across query,
// key and value heads, so its cos and sin stay in registers; all its loads are
// issued before the token's place is looked up, which costs two dependent
// reads.  Measured on GB300 (copy rate 6.78 TB/s; launches replayed from a graph),
// 16 bits / binary32: 8191 tokens, 32 + 8 + 8 heads of 128: 37 / 69 us, 5.6 / 5.9
// TB/s; 32 + 32 + 32 heads of 80, neighbouring pairs: 43 / 82 us, 5.8 / 6.2 TB/s; 64
// tokens of 32 + 8 + 8 heads of 128: 2.2 / 2.2 us.
#include "dc_llm.h"
#include "dc_numeric.cuh"

namespace dc {
namespace {

enum : uint32_t { kSiteTokenInfo = 1, kSiteTable = 2, kSiteIn = 3, kSiteOut = 4, kSiteCache = 5, kSiteAngle = 6 };

// CTAs of 128 threads (binary32, whose heads of up to 1024 elements are 256
// vectors: 256, 4 an SM, not swept).  Measured on 16-bit heads, heads in flight a
// thread x CTAs per SM x threads: 8191 tokens, 32 + 8 + 8 heads of 128, by halves:
// 2 x 10 x 128 36.7 us, 4 x 8 x 128 39.9, 2 x 5 x 256 42.7, 4 x 4 x 256 48.8;
// 32 + 32 + 32 heads of 80, neighbouring pairs: 45.7, 43.3, 49.3, 53.6.
template <int DT, bool INTERLEAVED>
struct Shape {
  static constexpr int kThreads = DT == kF32 ? 256 : 128;
  static constexpr int kHeads = INTERLEAVED ? 4 : 2;  // whose loads a thread has in flight
  static constexpr int kCtas = DT == kF32 ? 4 : INTERLEAVED ? 8 : 10;
};

__device__ __forceinline__ int32_t ld_i32(uint64_t base, uint64_t i, uint64_t n) {
  const int32_t* a = reinterpret_cast<const int32_t*>(base) + i;
  return in_bounds(a, 4, base, base + n * 4, kSiteTokenInfo) ? *a : -1;
}

// One 16-byte vector of a [tokens, heads, dim] tensor's token row; `span` is
// the bytes of that row from its first head to its last.
struct Row {
  uint64_t base, head, span;
};
__device__ __forceinline__ uint4 ld_row(const Row& r, int h, uint32_t off) {
  const uint4* a = reinterpret_cast<const uint4*>(r.base + h * r.head + off);
  return in_bounds(a, 16, r.base, r.base + r.span, kSiteIn) ? ld_stream(a) : uint4{};
}
__device__ __forceinline__ void st_row(const Row& r, int h, uint32_t off, const uint4& v, uint32_t site) {
  uint4* a = reinterpret_cast<uint4*>(r.base + h * r.head + off);
  if (in_bounds(a, 16, r.base, r.base + r.span, site)) st16(a, v);
}

template <int DT, bool INTERLEAVED>
__global__ __launch_bounds__(Shape<DT, INTERLEAVED>::kThreads, Shape<DT, INTERLEAVED>::kCtas) void dc_append_kernel(
    const __grid_constant__ AppendParams p) {
  constexpr int kHeadsInFlight = Shape<DT, INTERLEAVED>::kHeads;
  constexpr int kThreads = Shape<DT, INTERLEAVED>::kThreads;
  constexpr uint32_t kB = Elem<DT>::kBytes;
  constexpr int kPer = Elem<DT>::kPerVec;
  constexpr int kAngles = INTERLEAVED ? kPer / 2 : kPer;  // of a thread's vector
  pdl_enter();
  const uint64_t token = blockIdx.x;
  const uint64_t row_bytes = static_cast<uint64_t>(p.dim) * kB;
  const Row q{p.q + token * p.q_token, p.q_head, (p.q_heads > 0 ? p.q_heads - 1 : 0) * p.q_head + row_bytes};
  const Row qo{p.qo + token * p.qo_token, p.qo_head, (p.q_heads > 0 ? p.q_heads - 1 : 0) * p.qo_head + row_bytes};
  const Row k{p.k + token * p.k_token, p.k_head, (p.kv_heads - 1) * p.k_head + row_bytes};
  const Row v{p.v + token * p.v_token, p.v_head, (p.kv_heads - 1) * p.v_head + row_bytes};

  // units of a head: pairs of vectors (INTERLEAVED: single vectors) that
  // rotate, then vectors that do not
  const int turning = INTERLEAVED ? p.rot / kPer : p.rot / (2 * kPer);
  const int units = turning + (p.dim - p.rot) / kPer;
  const int per = kThreads / units;  // heads a pass
  const int unit = static_cast<int>(threadIdx.x) % units, sub = static_cast<int>(threadIdx.x) / units;
  const int heads = p.q_heads + 2 * p.kv_heads;  // queries, keys, values
  const bool turns = unit < turning, pair = turns && !INTERLEAVED;
  const uint32_t off0 = turns ? static_cast<uint32_t>(unit) * 16
                              : static_cast<uint32_t>(p.rot * kB) + static_cast<uint32_t>(unit - turning) * 16;
  const uint32_t off1 = off0 + static_cast<uint32_t>(p.rot / 2) * kB;
  const int step = per * static_cast<int>(gridDim.y);
  const int first = sub < per ? static_cast<int>(blockIdx.y) * per + sub : heads;

  uint4 a[kHeadsInFlight], b[kHeadsInFlight];
  auto load = [&](int h0) {
#pragma unroll
    for (int i = 0; i < kHeadsInFlight; ++i) {
      const int h = h0 + i * step;
      if (h >= heads) break;
      const bool is_q = h < p.q_heads, is_k = h < p.q_heads + p.kv_heads;
      const Row src = is_q ? q : is_k ? k : v;
      const int hh = h - (is_q ? 0 : is_k ? p.q_heads : p.q_heads + p.kv_heads);
      a[i] = ld_row(src, hh, off0);
      if (pair) b[i] = ld_row(src, hh, off1);
    }
  };
  load(first);

  const int32_t pos = ld_i32(p.positions, token, p.tokens);
  const int32_t seq = ld_i32(p.seqs, token, p.tokens);
  if (pos < 0) return;  // padding: nothing is written for it
  // where the token goes; a place that does not exist is never touched
  bool ok = seq >= 0 && static_cast<uint32_t>(seq) < p.num_seqs;
  const uint32_t col = static_cast<uint32_t>(pos) / p.page_size, slot = static_cast<uint32_t>(pos) % p.page_size;
  ok = ok && col < p.table_width && (p.rot == 0 || static_cast<int64_t>(pos) < p.cos_rows);
  int32_t page = -1;
  if (ok) {
    const int32_t* t = reinterpret_cast<const int32_t*>(p.table) + seq * p.table_stride + col;
    const uint64_t hi = p.table + (static_cast<uint64_t>(p.num_seqs - 1) * p.table_stride + p.table_width) * 4;
    if (in_bounds(t, 4, p.table, hi, kSiteTable)) page = *t;
  }
  // the cosines and sines of this thread's elements (of its pairs)
  float cs[kAngles], sn[kAngles];
  if (turns && ok) {
    const uint64_t base = p.cos_sin + static_cast<uint64_t>(pos) * p.rot * 4;
    const float* c = reinterpret_cast<const float*>(base) + unit * kAngles;
#pragma unroll
    for (int i = 0; i < kAngles; ++i) {
      const bool read = in_bounds(c + i, 4, base, base + p.rot * 4ull, kSiteAngle);
      cs[i] = read ? __ldg(c + i) : 0.0f;
      sn[i] = read ? __ldg(c + i + p.rot / 2) : 0.0f;
    }
  }
  ok = ok && page >= 0 && page < p.num_pages;
  if (!ok) {  // the queries of a token that cannot be placed read NaN
    const int vecs = p.dim / kPer;
    const uint32_t w = DT == kF32 ? 0x7FC00000u : DT == kF16 ? 0x7E007E00u : 0x7FC07FC0u;
    for (int u = blockIdx.y * kThreads + threadIdx.x; u < p.q_heads * vecs; u += gridDim.y * kThreads)
      st_row(qo, u / vecs, static_cast<uint32_t>(u % vecs) * 16, make_uint4(w, w, w, w), kSiteOut);
    return;
  }
  const Row kc{p.kc.base + static_cast<uint64_t>(page) * p.kc.page + slot * p.kc.token, p.kc.head,
               (p.kv_heads - 1) * p.kc.head + row_bytes};
  const Row vc{p.vc.base + static_cast<uint64_t>(page) * p.vc.page + slot * p.vc.token, p.vc.head,
               (p.kv_heads - 1) * p.vc.head + row_bytes};
  for (int h0 = first; h0 < heads; h0 += step * kHeadsInFlight) {
    if (h0 != first) load(h0);
#pragma unroll
    for (int i = 0; i < kHeadsInFlight; ++i) {
      const int h = h0 + i * step;
      if (h >= heads) break;
      const bool is_q = h < p.q_heads, is_k = h < p.q_heads + p.kv_heads;
      const Row dst = is_q ? qo : is_k ? kc : vc;
      const int hh = h - (is_q ? 0 : is_k ? p.q_heads : p.q_heads + p.kv_heads);
      const uint32_t site = is_q ? kSiteOut : kSiteCache;
      if (turns && is_k) {
        float x[kPer];
        unpack<DT>(a[i], x);
        if constexpr (INTERLEAVED) {
#pragma unroll
          for (int e = 0; e < kPer; e += 2) {
            const float lo = x[e] * cs[e / 2] - x[e + 1] * sn[e / 2];
            x[e + 1] = x[e + 1] * cs[e / 2] + x[e] * sn[e / 2];
            x[e] = lo;
          }
        } else {
          float y[kPer];
          unpack<DT>(b[i], y);
#pragma unroll
          for (int e = 0; e < kPer; ++e) {
            const float lo = x[e] * cs[e] - y[e] * sn[e];
            y[e] = y[e] * cs[e] + x[e] * sn[e];
            x[e] = lo;
          }
          b[i] = repack<DT>(y);
        }
        a[i] = repack<DT>(x);
      }
      st_row(dst, hh, off0, a[i], site);
      if (pair) st_row(dst, hh, off1, b[i], site);
    }
  }
}

template <int DT, bool INTERLEAVED>
cudaError_t launch_t(const AppendParams& p, int sms, bool pdl, cudaStream_t s, int* grid) {
  constexpr int kPer = Elem<DT>::kPerVec, kThreads = Shape<DT, INTERLEAVED>::kThreads;
  // few tokens: several CTAs share one token's heads
  const int units = INTERLEAVED ? p.dim / kPer : p.rot / (2 * kPer) + (p.dim - p.rot) / kPer;
  const int per = kThreads / units, heads = p.q_heads + 2 * p.kv_heads;
  int y = 1;
  if (p.tokens < 2 * static_cast<uint64_t>(sms)) {
    const int most = (heads + per - 1) / per;
    const int room = static_cast<int>(4 * static_cast<uint64_t>(sms) / p.tokens);
    y = most < room ? most : room;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.tokens), static_cast<unsigned>(y));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = pdl ? attr : nullptr;
  cfg.numAttrs = pdl ? 1 : 0;
  *grid = static_cast<int>(p.tokens) * y;
  return cudaLaunchKernelEx(&cfg, dc_append_kernel<DT, INTERLEAVED>, p);
}

template <int DT>
cudaError_t launch_dt(const AppendParams& p, int sms, bool pdl, cudaStream_t s, int* grid) {
  return p.interleaved ? launch_t<DT, true>(p, sms, pdl, s, grid) : launch_t<DT, false>(p, sms, pdl, s, grid);
}

}  // namespace

cudaError_t launch_append(const AppendParams& p, int dtype, int sms, bool pdl, cudaStream_t s, int* grid) {
  switch (dtype) {
    case kF16: return launch_dt<kF16>(p, sms, pdl, s, grid);
    case kF32: return launch_dt<kF32>(p, sms, pdl, s, grid);
    default: return launch_dt<kBF16>(p, sms, pdl, s, grid);
  }
}

DC_BOUNDS_READER(take_bounds_append)

}  // namespace dc
