// Queries and keys normed per head and rotated to their positions, into tensors
// or (keys, with their values) into a paged cache; and the gradient of that.
//
// Mathematics.  For a head x of n elements, r = 1 / sqrt(mean x^2 + eps) and
// weights w: y = R(x r w), R the rotation of pairs (a, b) by a position's
// angles, (a c - b s, b c + a s).  With g = R^T dy (the rotation back):
// dx = r (g w - x r mean(g w x r)), dw = sum over tokens and heads of g x r.
// Everything in binary32, rounded once; a head's sums add a lane's elements in
// order, then the lanes in pairs, so they depend on nothing but the head.
//
// Bound: memory, every element read and written once.  A warp takes a token:
// its lanes hold the cosines and sines of their elements and go through the
// token's heads, as many at a time as 32 lanes hold, the next ones' loads in
// flight while they work; where there are few tokens several warps share one.  Queries,
// keys and values are CTAs of their own, so that the weights stay in registers
// and, for the gradient, the sums over a warp's tokens do too; the CTAs' sums
// are added up by a second kernel in one fixed order.
// Measured, 16384 tokens, 32/8 heads of 128, BF16: forward 67 us and gradient 102
// us, 5 TB/s of what has to move, issue slots 55 to 60 % busy; 8191 tokens of 96 heads
// of 80 into a cache 71 us, 3.5 TB/s (30 of 32 lanes, rows of 160 bytes).  With lanes
// in powers of two a head and more CTAs than fit the GPU at once 238 us (both
// directions) and 92.
#include <algorithm>

#include "dc_llm.h"
#include "dc_numeric.cuh"

namespace dc {
namespace {

enum : uint32_t { kSiteToken = 1, kSiteTable = 2, kSiteIn = 3, kSiteOut = 4, kSiteAngle = 5, kSiteWeight = 6, kSitePartial = 7 };

constexpr int kWarps = kNormThreads / 32;
constexpr int norm_ctas_per_sm(int units, bool gradient) { return units > 2 ? 1 : units == 2 ? 2 : gradient ? 4 : 6; }

__device__ __forceinline__ int32_t ld_i32(uint64_t base, uint64_t i, uint64_t n) {
  const int32_t* a = reinterpret_cast<const int32_t*>(base) + i;
  return in_bounds(a, 4, base, base + n * 4, kSiteToken) ? *a : -1;
}

// 1 / sqrt(x), within an ulp or so: the hardware's estimate and one step of
// Newton's iteration (0 and infinity as they are).
__device__ __forceinline__ float inverse_root(float x) {
  const float r = rsqrtf(x);
  const float s = __fmaf_rn(-0.5f * x * r, r, 1.5f) * r;
  return r > 0.0f && r < __int_as_float(0x7F800000) ? s : r;
}

// UNITS work units of a head for a lane: a pair of 16-byte vectors half the
// rotated part apart, or (INTERLEAVED, and what is not rotated) a single one.
template <int DT, bool INTERLEAVED, int UNITS, bool GRADIENT>
struct Kernel {
  static constexpr int kPer = Elem<DT>::kPerVec;
  static constexpr int kHalves = INTERLEAVED ? 1 : 2;
  static constexpr int kAngles = INTERLEAVED ? kPer / 2 : kPer;
  static constexpr int kAhead = INTERLEAVED && UNITS == 1 ? 2 : 1;  // heads whose loads are in flight

  struct Raw {
    uint4 v[UNITS][kHalves];
  };
  struct Values {
    float v[UNITS][kHalves][kPer];
  };

  const NormParams& p;
  uint32_t off[UNITS];       // bytes of a unit's first vector in a head
  bool there[UNITS], turns[UNITS];
  uint32_t half;             // bytes to its second one

  __device__ explicit Kernel(const NormParams& p_, int lane) : p(p_) {
    const int turning = INTERLEAVED ? p.rot / kPer : p.rot / (2 * kPer);
    half = static_cast<uint32_t>(p.rot / 2) * Elem<DT>::kBytes;
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      const int u = lane % p.lanes + i * p.lanes;
      there[i] = u < p.units && lane / p.lanes < 32 / p.lanes;
      turns[i] = u < turning;
      off[i] = turns[i] ? static_cast<uint32_t>(u) * 16
                        : static_cast<uint32_t>(p.rot * Elem<DT>::kBytes) + static_cast<uint32_t>(u - turning) * 16;
    }
  }
  // (a unit that is not rotated has one vector)
  __device__ bool has(int i, int h) const { return there[i] && (h == 0 || turns[i]); }

  __device__ void load(Raw& r, uint64_t head, bool read) const {
    const uint64_t hi = head + static_cast<uint64_t>(p.dim) * Elem<DT>::kBytes;
#pragma unroll
    for (int i = 0; i < UNITS; ++i)
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        const uint4* a = reinterpret_cast<const uint4*>(head + off[i] + (h ? half : 0));
        r.v[i][h] = read && has(i, h) && in_bounds(a, 16, head, hi, kSiteIn) ? ld_stream(a) : uint4{};
      }
  }
  __device__ void store(const Raw& r, uint64_t head, bool write, uint64_t lo, uint64_t hi) const {
#pragma unroll
    for (int i = 0; i < UNITS; ++i)
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        uint4* a = reinterpret_cast<uint4*>(head + off[i] + (h ? half : 0));
        if (write && has(i, h) && in_bounds(a, 16, lo, hi, kSiteOut)) st16(a, r.v[i][h]);
      }
  }
  __device__ void widen(const Raw& r, Values& x) const {
#pragma unroll
    for (int i = 0; i < UNITS; ++i)
#pragma unroll
      for (int h = 0; h < kHalves; ++h) unpack<DT>(r.v[i][h], x.v[i][h]);
  }
  __device__ void narrow(const Values& x, Raw& r) const {
#pragma unroll
    for (int i = 0; i < UNITS; ++i)
#pragma unroll
      for (int h = 0; h < kHalves; ++h) r.v[i][h] = repack<DT>(x.v[i][h]);
  }
  // The sum over a head of a product of two sets of values.
  __device__ float dot(const Values& a, const Values& b) const {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < UNITS; ++i)
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int e = 0; e < kPer; ++e) s = __fmaf_rn(a.v[i][h][e], b.v[i][h][e], s);
    if ((p.lanes & (p.lanes - 1)) == 0) {
#pragma unroll
      for (int d = 1; d < 32; d *= 2)
        if (d < p.lanes) s += __shfl_xor_sync(~0u, s, d);
      return s;
    }
    // neighbours in pairs, then pairs of pairs, ..., into a head's first lane
    const int lane = threadIdx.x & 31, u = lane % p.lanes;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      if (d >= p.lanes) break;
      const float t = __shfl_down_sync(~0u, s, d);
      if (u + d < p.lanes) s += t;
    }
    return __shfl_sync(~0u, s, lane - u);
  }
  // Rotates the units that turn, by the angles or (BACK) their negatives.
  template <bool BACK>
  __device__ void rotate(Values& x, const float (&cs)[UNITS][kAngles], const float (&sn)[UNITS][kAngles]) const {
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      if (!turns[i]) continue;
#pragma unroll
      for (int e = 0; e < kAngles; ++e) {
        float& a = INTERLEAVED ? x.v[i][0][2 * e] : x.v[i][0][e];
        float& b = INTERLEAVED ? x.v[i][0][2 * e + 1] : x.v[i][kHalves - 1][e];
        const float s = BACK ? -sn[i][e] : sn[i][e];
        const float lo = __fmaf_rn(a, cs[i][e], -(b * s));
        b = __fmaf_rn(b, cs[i][e], a * s);
        a = lo;
      }
    }
  }
  __device__ void weights(Values& w, uint64_t base) const {
#pragma unroll
    for (int i = 0; i < UNITS; ++i)
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          const uint32_t at = (off[i] + (h ? half : 0)) / Elem<DT>::kBytes + e;
          const uint64_t a = base + static_cast<uint64_t>(at) * (p.w32 ? 4 : Elem<DT>::kBytes);
          w.v[i][h][e] = !has(i, h) ? 0.0f : p.w32 ? *reinterpret_cast<const float*>(a) : load_elem<DT>(a);
        }
  }
};

template <int DT, bool INTERLEAVED, int UNITS, bool GRADIENT>
__global__ __launch_bounds__(kNormThreads, norm_ctas_per_sm(UNITS, GRADIENT)) void dc_norm_kernel(const __grid_constant__ NormParams p) {
  using K = Kernel<DT, INTERLEAVED, UNITS, GRADIENT>;
  constexpr int kB = Elem<DT>::kBytes;
  extern __shared__ float sums[];  // (gradient) [warps][heads at a time][dim]
  pdl_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int j = 0;
  while (j + 1 < p.jobs && blockIdx.x >= p.job[j + 1].cta0) ++j;
  const NormJob& job = p.job[j];
  const bool copy = job.w == 0;
  const K k(p, lane);
  const int heads_at_once = 32 / p.lanes, sub = lane / p.lanes;  // (lanes left over go with no head)
  const int step = heads_at_once * job.split;
  const uint64_t row_bytes = static_cast<uint64_t>(p.dim) * kB;
  typename K::Values w, dw;
  if (!copy) k.weights(w, job.w);
  if constexpr (GRADIENT) {
#pragma unroll
    for (int i = 0; i < UNITS; ++i)
#pragma unroll
      for (int h = 0; h < K::kHalves; ++h)
#pragma unroll
        for (int e = 0; e < K::kPer; ++e) dw.v[i][h][e] = 0.0f;
  }
  const uint64_t items = p.tokens * static_cast<uint64_t>(job.split);
  for (uint64_t item = static_cast<uint64_t>(blockIdx.x - job.cta0) * kWarps + warp; item < items;
       item += static_cast<uint64_t>(job.ctas) * kWarps) {
    const uint64_t token = job.split == 1 ? item : item / static_cast<uint32_t>(job.split);
    const int first = job.split == 1 ? 0 : static_cast<int>(item % static_cast<uint32_t>(job.split)) * heads_at_once;
    const uint64_t x_row = job.x.base + token * job.x.token;
    [[maybe_unused]] const uint64_t dy_row = job.dy.base + token * job.dy.token;
    typename K::Raw next[K::kAhead];
    [[maybe_unused]] typename K::Raw next_dy[K::kAhead];
    auto fetch = [&](int a, int h) {
      const bool read = h < job.heads && sub < heads_at_once;
      k.load(next[a], x_row + static_cast<uint64_t>(read ? h : 0) * job.x.head, read);
      if constexpr (GRADIENT) k.load(next_dy[a], dy_row + static_cast<uint64_t>(read ? h : 0) * job.dy.head, read);
    };
#pragma unroll
    for (int a = 0; a < K::kAhead; ++a) fetch(a, first + a * step + sub);

    const int32_t pos = ld_i32(p.positions, token, p.tokens);
    const bool padding = pos < 0;
    bool ok = !padding && (p.rot == 0 || static_cast<int64_t>(pos) < p.cos_rows);
    uint64_t y_row = job.y.base + token * job.y.token;
    // all of this warp's heads of the token become one number
    auto fill = [&](uint64_t row, float value) {
      typename K::Values v;
      typename K::Raw r;
#pragma unroll
      for (int i = 0; i < UNITS; ++i)
#pragma unroll
        for (int a = 0; a < K::kHalves; ++a)
#pragma unroll
          for (int e = 0; e < K::kPer; ++e) v.v[i][a][e] = value;
      k.narrow(v, r);
      for (int h = first + sub; h < job.heads; h += step)
        k.store(r, row + static_cast<uint64_t>(h) * job.y.head, sub < heads_at_once, row,
                row + static_cast<uint64_t>(job.heads - 1) * job.y.head + row_bytes);
    };
    if (p.cached) {
      if (padding) continue;  // nothing is written for it
      // where the token goes; a place that does not exist is never touched
      const int32_t seq = ld_i32(p.seqs, token, p.tokens);
      const uint32_t col = static_cast<uint32_t>(pos) / p.page_size, slot = static_cast<uint32_t>(pos) % p.page_size;
      ok = ok && seq >= 0 && static_cast<uint32_t>(seq) < p.num_seqs && col < p.table_width;
      int32_t page = -1;
      if (ok) {
        const int32_t* t = reinterpret_cast<const int32_t*>(p.table) + seq * p.table_stride + col;
        const uint64_t hi = p.table + (static_cast<uint64_t>(p.num_seqs - 1) * p.table_stride + p.table_width) * 4;
        if (in_bounds(t, 4, p.table, hi, kSiteTable)) page = *t;
      }
      ok = ok && page >= 0 && page < p.num_pages;
      if (j > 0) {
        if (!ok) continue;
        const PagedView& c = j == 1 ? p.kc : p.vc;
        y_row = c.base + static_cast<uint64_t>(page) * c.page + slot * c.token;
      }
    }
    if (!ok) {  // padding: zeros; a place that does not exist: NaN
      const float value = padding ? 0.0f : __int_as_float(0x7FC00000);
      fill(y_row, value);
      if constexpr (GRADIENT) {
#pragma unroll
        for (int i = 0; i < UNITS; ++i)
#pragma unroll
          for (int a = 0; a < K::kHalves; ++a)
#pragma unroll
            for (int e = 0; e < K::kPer; ++e) dw.v[i][a][e] += value;
      }
      continue;
    }
    const uint64_t y_hi = y_row + static_cast<uint64_t>(job.heads - 1) * job.y.head + row_bytes;
    float cs[UNITS][K::kAngles], sn[UNITS][K::kAngles];
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
      const uint64_t base = p.cos_sin + static_cast<uint64_t>(pos) * p.rot * 4;
      const float* c = reinterpret_cast<const float*>(base) + k.off[i] / 16 * K::kAngles;
      const bool read = !copy && k.turns[i] && in_bounds(c, K::kAngles * 4, base, base + p.rot * 4ull, kSiteAngle) &&
                        in_bounds(c + p.rot / 2, K::kAngles * 4, base, base + p.rot * 4ull, kSiteAngle);
      constexpr int kWide = K::kAngles < 4 ? 2 : 4;  // floats of a load, where the table is aligned for it
      if (read && p.angles_aligned) {
#pragma unroll
        for (int e = 0; e < K::kAngles; e += kWide) {
          if constexpr (kWide == 4) {
            const float4 x = __ldg(reinterpret_cast<const float4*>(c + e)), y = __ldg(reinterpret_cast<const float4*>(c + e + p.rot / 2));
            cs[i][e] = x.x, cs[i][e + 1] = x.y, cs[i][e + 2] = x.z, cs[i][e + 3] = x.w;
            sn[i][e] = y.x, sn[i][e + 1] = y.y, sn[i][e + 2] = y.z, sn[i][e + 3] = y.w;
          } else {
            const float2 x = __ldg(reinterpret_cast<const float2*>(c + e)), y = __ldg(reinterpret_cast<const float2*>(c + e + p.rot / 2));
            cs[i][e] = x.x, cs[i][e + 1] = x.y;
            sn[i][e] = y.x, sn[i][e + 1] = y.y;
          }
        }
      } else {
#pragma unroll
        for (int e = 0; e < K::kAngles; ++e) {
          cs[i][e] = read ? __ldg(c + e) : 0.0f;
          sn[i][e] = read ? __ldg(c + e + p.rot / 2) : 0.0f;
        }
      }
    }
    // (the lanes of a warp go through the loop together: they share sums)
    for (int hb = first; hb < job.heads; hb += K::kAhead * step) {
#pragma unroll
     for (int ahead = 0; ahead < K::kAhead; ++ahead) {
      const int h0 = hb + ahead * step, h = h0 + sub;
      if (h0 >= job.heads) break;
      const bool mine = h < job.heads && sub < heads_at_once;
      typename K::Raw now = next[ahead];
      [[maybe_unused]] typename K::Raw now_dy;
      if constexpr (GRADIENT) now_dy = next_dy[ahead];
      if (h0 + K::kAhead * step < job.heads) fetch(ahead, h + K::kAhead * step);
      const uint64_t out = y_row + static_cast<uint64_t>(mine ? h : 0) * job.y.head;
      if (!copy) {
        typename K::Values x;
        k.widen(now, x);
        const float r = inverse_root(__fmaf_rn(k.dot(x, x), p.inv_dim, p.eps));
#pragma unroll
        for (int i = 0; i < UNITS; ++i)
#pragma unroll
          for (int a = 0; a < K::kHalves; ++a)
#pragma unroll
            for (int e = 0; e < K::kPer; ++e) x.v[i][a][e] *= r;
        if constexpr (!GRADIENT) {
#pragma unroll
          for (int i = 0; i < UNITS; ++i)
#pragma unroll
            for (int a = 0; a < K::kHalves; ++a)
#pragma unroll
              for (int e = 0; e < K::kPer; ++e) x.v[i][a][e] *= w.v[i][a][e];
          k.template rotate<false>(x, cs, sn);
        } else {
          typename K::Values g;
          k.widen(now_dy, g);
          k.template rotate<true>(g, cs, sn);
#pragma unroll
          for (int i = 0; i < UNITS; ++i)
#pragma unroll
            for (int a = 0; a < K::kHalves; ++a)
#pragma unroll
              for (int e = 0; e < K::kPer; ++e) {
                // (where there is no head, g is 0 and x is 0 or NaN, of eps 0)
                if (mine) dw.v[i][a][e] = __fmaf_rn(g.v[i][a][e], x.v[i][a][e], dw.v[i][a][e]);
                g.v[i][a][e] *= w.v[i][a][e];
              }
          const float c = k.dot(g, x) * p.inv_dim;
#pragma unroll
          for (int i = 0; i < UNITS; ++i)
#pragma unroll
            for (int a = 0; a < K::kHalves; ++a)
#pragma unroll
              for (int e = 0; e < K::kPer; ++e)
                x.v[i][a][e] = r * __fmaf_rn(-c, x.v[i][a][e], g.v[i][a][e]);
        }
        k.narrow(x, now);
      }
      k.store(now, out, mine, y_row, y_hi);
     }
    }
  }
  if constexpr (GRADIENT) {
    if (!job.partial) return;
    // the CTA's sum: its warps' groups of lanes in order
    float* to = sums + (warp * heads_at_once + sub) * p.dim;
#pragma unroll
    for (int i = 0; i < UNITS; ++i)
#pragma unroll
      for (int h = 0; h < K::kHalves; ++h)
        if (k.has(i, h) && sub < heads_at_once) {
#pragma unroll
          for (int e = 0; e < K::kPer; ++e) to[(k.off[i] + (h ? k.half : 0)) / kB + e] = dw.v[i][h][e];
        }
    __syncthreads();
    for (int d = threadIdx.x; d < p.dim; d += kNormThreads) {
      float s = sums[d];
      for (int i = 1; i < kWarps * heads_at_once; ++i) s += sums[i * p.dim + d];
      float* a = reinterpret_cast<float*>(job.partial) + static_cast<uint64_t>(blockIdx.x - job.cta0) * p.dim + d;
      if (in_bounds(a, 4, job.partial, job.partial + 4ull * job.ctas * p.dim, kSitePartial)) *a = s;
    }
  }
}

// 32 columns a CTA: 32 threads a column, each every 32nd CTA's sum, then a tree.
template <int DT>
__global__ __launch_bounds__(1024) void dc_norm_finish_kernel(const __grid_constant__ NormFinishParams p) {
  pdl_enter();
  __shared__ float part[32][33];
  const int d = static_cast<int>(blockIdx.x) * 32 + static_cast<int>(threadIdx.x & 31), y = threadIdx.x >> 5, j = blockIdx.y;
  if (!p.out[j]) return;
  float s = 0.0f;
  const uint64_t base = p.partial[j], hi = base + 4ull * p.ctas[j] * p.dim;
  if (d < p.dim)
    for (uint32_t c = y; c < p.ctas[j]; c += 32) {
      const float* a = reinterpret_cast<const float*>(base) + static_cast<uint64_t>(c) * p.dim + d;
      if (in_bounds(a, 4, base, hi, kSitePartial)) s += *a;
    }
  part[y][threadIdx.x & 31] = s;
  __syncthreads();
  s = part[threadIdx.x & 31][y];  // lane: one of the 32 sums of column y
#pragma unroll
  for (int k = 1; k < 32; k *= 2) s += __shfl_xor_sync(~0u, s, k);
  const int column = static_cast<int>(blockIdx.x) * 32 + y;
  if ((threadIdx.x & 31) == 0 && column < p.dim) {
    const int es = p.out32 ? 4 : Elem<DT>::kBytes;
    const uint64_t a = p.out[j] + static_cast<uint64_t>(column) * es;
    if (!in_bounds(reinterpret_cast<const void*>(a), es, p.out[j], p.out[j] + static_cast<uint64_t>(p.dim) * es, kSiteOut)) return;
    if (p.out32) *reinterpret_cast<float*>(a) = s;
    else store_elem<DT>(a, s);
  }
}

int units_per_lane(const NormParams& p) {
  const int n = (p.units + p.lanes - 1) / p.lanes;
  return n <= 1 ? 1 : n <= 2 ? 2 : 4;
}

template <int DT, bool INTERLEAVED, bool GRADIENT>
cudaError_t launch_units(const NormParams& p, bool pdl, cudaStream_t s, int grid) {
  const size_t smem = GRADIENT ? static_cast<size_t>(kWarps) * (32 / p.lanes) * p.dim * 4 : 0;
  switch (units_per_lane(p)) {
    case 1: return launch_ex(dc_norm_kernel<DT, INTERLEAVED, 1, GRADIENT>, grid, kNormThreads, pdl, s, p, smem);
    case 2: return launch_ex(dc_norm_kernel<DT, INTERLEAVED, 2, GRADIENT>, grid, kNormThreads, pdl, s, p, smem);
    default:
      // (16-bit heads of 512 have at most 64 units)
      if constexpr (DT == kF32) return launch_ex(dc_norm_kernel<DT, INTERLEAVED, 4, GRADIENT>, grid, kNormThreads, pdl, s, p, smem);
      return cudaErrorInvalidValue;
  }
}

template <int DT>
cudaError_t launch_dt(const NormParams& p, bool interleaved, bool gradient, bool pdl, cudaStream_t s, int grid) {
  if (gradient) return interleaved ? launch_units<DT, true, true>(p, pdl, s, grid) : launch_units<DT, false, true>(p, pdl, s, grid);
  return interleaved ? launch_units<DT, true, false>(p, pdl, s, grid) : launch_units<DT, false, false>(p, pdl, s, grid);
}

}  // namespace

void plan_norm(NormParams* p, int dtype, bool interleaved, bool gradient) {
  const int per = dtype == kF32 ? 4 : 8;
  p->units = interleaved ? p->dim / per : p->rot / (2 * per) + (p->dim - p->rot) / per;
  // a head's lanes: as many as it has units, or a power of two where as many heads
  // fit a warp so (their sums take fewer steps)
  p->lanes = 1;
  while (p->lanes < 32 && p->lanes < p->units) p->lanes *= 2;
  if (p->units < 32 && 32 / p->units > 32 / p->lanes) p->lanes = p->units;
  p->angles_aligned = p->cos_sin % 16 == 0;
  p->inv_dim = 1.0f / static_cast<float>(p->dim);
  const int at_once = 32 / p->lanes;
  const int cap = gradient ? kNormGradCtas : kNormCtas;
  int heads = 0;
  for (int j = 0; j < p->jobs; ++j) heads += p->job[j].heads;
  uint32_t cta = 0;
  for (int j = 0; j < p->jobs; ++j) {
    NormJob& o = p->job[j];
    o.cta0 = cta;
    o.ctas = 0;
    o.split = 1;
    if (o.heads == 0) continue;  // (an append without queries)
    // few tokens: several warps share one, as long as the GPU has room for them
    const int most = (o.heads + at_once - 1) / at_once;
    const uint64_t share = std::max<uint64_t>(1, static_cast<uint64_t>(cap) * o.heads / heads);
    const uint64_t room = std::max<uint64_t>(1, share * kWarps / std::max<uint64_t>(1, p->tokens));
    o.split = static_cast<int32_t>(std::min<uint64_t>(static_cast<uint64_t>(most), room));
    const uint64_t ctas = (p->tokens * static_cast<uint64_t>(o.split) + kWarps - 1) / kWarps;
    o.ctas = static_cast<uint32_t>(std::max<uint64_t>(1, std::min<uint64_t>(ctas, share)));
    cta += o.ctas;
  }
}

cudaError_t launch_norm(const NormParams& p, int dtype, bool interleaved, bool gradient, bool pdl, cudaStream_t s, int* grid) {
  *grid = static_cast<int>(p.job[p.jobs - 1].cta0 + p.job[p.jobs - 1].ctas);
  switch (dtype) {
    case kF16: return launch_dt<kF16>(p, interleaved, gradient, pdl, s, *grid);
    case kF32: return launch_dt<kF32>(p, interleaved, gradient, pdl, s, *grid);
    default: return launch_dt<kBF16>(p, interleaved, gradient, pdl, s, *grid);
  }
}

cudaError_t launch_norm_finish(const NormFinishParams& p, int dtype, bool pdl, cudaStream_t s, int* grid) {
  const dim3 g(static_cast<unsigned>((p.dim + 31) / 32), 2);
  *grid = static_cast<int>(g.x * g.y);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = g;
  cfg.blockDim = dim3(1024);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = pdl ? attr : nullptr;
  cfg.numAttrs = pdl ? 1 : 0;
  switch (dtype) {
    case kF16: return cudaLaunchKernelEx(&cfg, dc_norm_finish_kernel<kF16>, p);
    case kF32: return cudaLaunchKernelEx(&cfg, dc_norm_finish_kernel<kF32>, p);
    default: return cudaLaunchKernelEx(&cfg, dc_norm_finish_kernel<kBF16>, p);
  }
}

DC_BOUNDS_READER(take_bounds_norm)

}  // namespace dc
