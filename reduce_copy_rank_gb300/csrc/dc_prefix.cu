// Attention of one new token per sequence where groups of sequences share a
// long prefix in the paged cache: the prefix's keys and values are read once for
// all of a group's queries.
//
// Mathematics.  A softmax over the prefix's and the sequence's own tokens is
// joined from its parts: each keeps a reference r (in units of log2, a whole
// number), l = sum 2^(s_t - r) and u = sum 2^(s_t - r) v_t, and parts add up
// after a change of reference, which multiplies by a power of two.  The own
// tokens' part comes from the kernel of paged attention; the prefix's is
// computed here in chunks of tokens; a last kernel adds the parts up in order.
//
// The rows of one product are the queries of all heads of a key head and of all
// sequences of the group, 128 at a time; a tile of 64 tokens is S = Q K^T on the
// tensor cores, its weights in registers and back into tensor memory as the left
// operand of U += P V.  Two warps copy keys and values through page numbers into
// the swizzled rows that the tensor cores read (TMA boxes of the tokens that divide
// a page and a tile; cp.async where those are fewer than 8), one issues the
// products, four hold a row a thread.  Two buffers of scores let the next tile's
// product run under this one's exponentials; with heads up to 128 two CTAs share
// an SM, whose chains of waits fill each other's gaps.
//
// Bound: memory while a group has up to about 128 rows; above that the chain of a
// tile (scores, read from tensor memory, exponentials, weights written back, product).
// Measured, 128 sequences behind 65536 tokens, 32/8 heads of 128, BF16: the prefix
// 144 us, 0.95 PFLOP/s; tiles of 128 tokens and one buffer of scores 206 us; 256 rows
// a CTA 186 to 198 us.  64 sequences in four groups of 7001 tokens, 12/12 heads of
// 64, FP16: 24 us.
//
// Rounding: the weights enter the second product in 16 bits (half a step each at
// most, 2^-8 or 2^-11 of it, of either sign); their sum l takes them unrounded.  In
// binary16 they are held times 2^7, a row's largest between 2^6 and 2^15, so that what is
// 2^-20 of that is still a normal number.  (The own tokens' weights enter as two numbers
// each, so that the last rounding is theirs alone: 2 products for 1, which their kernel has
// to spare and this one's chain has not.  Error of the outputs, BF16 / FP16: 2.4e-3 /
// 2.9e-4, with weights in 32 bits 1.7e-3 / 2.1e-4.)
#include <atomic>

#include "dc_llm.h"
#include "dc_numeric.cuh"
#include "dc_tc.cuh"

namespace dc {
namespace {

using namespace tc;

enum : uint32_t { kSiteLength = 1, kSiteTable = 2, kSiteQuery = 3, kSiteKey = 4, kSiteValue = 5, kSitePartial = 6, kSiteOut = 7 };

__device__ unsigned int g_prefix_fault_bits;

template <int D>
struct Shape {
  static constexpr int kTile = kPrefixTile;
  static constexpr int kBlocks = (D + 63) / 64;          // of 64 columns: swizzled rows of 128 bytes
  static constexpr int kStages = D > 64 ? 2 : 4;         // of keys, and of values
  static constexpr int kScores = 2;                      // buffers of scores: the next tile's are under way
  static constexpr int kCtas = D > 128 ? 1 : 2;
  static constexpr int kQ = kBlocks * kPrefixRows * 128, kKV = kBlocks * kTile * 128;
  static constexpr int kSmem = kQ + 2 * kStages * kKV + 1024;
  static constexpr uint32_t kOut = kScores * kTile;      // the output's first column of tensor memory
  static constexpr uint32_t kColumns = kOut + D <= 256 ? 256 : 512;
  static constexpr int kVecs = D / 8;                    // 16-byte parts of a row
};
// Four warps hold a row a thread, one issues products, one copies keys, one
// values, and the last helps with the queries (a ninth warp would take a quarter
// of the registers from all).
constexpr int kThreads = 256;
constexpr int kQueryLoaders = 96;

// A row's reference is at most kSlack behind its largest score: moving it takes
// a pass over the output so far, which almost every tile would need for one of a
// warp's rows.  The weights' unit is 2^7 in binary16, where they stay below 2^16.
constexpr float kSlack = 8.0f;
template <int DT>
constexpr float kShift = DT == kF16 ? 7.0f : 0.0f;

__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, uint64_t src, bool read) {
  const uint32_t n = read ? 16u : 0u;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}

// 2^(x - M) for whole numbers x <= M; 0 below 2^-126, and for x = -inf.
__device__ __forceinline__ float pow2_diff(float x, float M) {
  const int k = static_cast<int>(fmaxf(x - M, -127.0f));
  return __int_as_float((k + 127) << 23);
}

// A prefix's tokens; `bad`: a length past the table.
__device__ __forceinline__ uint32_t prefix_length(const PrefixParams& p, int prefix, bool* bad) {
  const int32_t* a = reinterpret_cast<const int32_t*>(p.lengths) + prefix;
  const int32_t n = in_bounds(a, 4, p.lengths, p.lengths + 4ull * p.prefixes, kSiteLength) ? *a : 0;
  *bad = n > 0 && static_cast<uint64_t>(n) > static_cast<uint64_t>(p.table_width) * p.page_size;
  return n < 0 ? 0u : *bad ? 1u : static_cast<uint32_t>(n);
}

// One warp copies its rows of keys or values, tile by tile.
template <int D>
struct Copier {
  using S = Shape<D>;
  static constexpr int kLooks = S::kTile / 32;
  const PrefixParams& p;
  const PagedView& view;
  uint64_t table_row, head;  // head: bytes of the key head in a token
  uint32_t end;              // the chunk's last token + 1
  uint32_t site;
  uint64_t at[kLooks];       // where this lane's rows of the next tile are (0: nowhere)
  bool missing = false;
  int32_t page = -1, slot = 0;  // (TMA) of this lane's box, -1: none

  __device__ int32_t id_of(uint32_t pg) {
    const int32_t* a = reinterpret_cast<const int32_t*>(table_row) + pg;
    const int32_t id = in_bounds(a, 4, table_row, table_row + 4ull * p.table_width, kSiteTable) ? *a : -1;
    if (id >= 0 && id < p.num_pages) return id;
    missing = true;
    return -1;
  }
  __device__ void look_up_box(uint32_t tile0, uint32_t boxes) {
    const uint32_t lane = threadIdx.x & 31, t = tile0 + lane * static_cast<uint32_t>(p.slots);
    page = -1;
    if (lane >= boxes || t >= end) return;
    const uint32_t pg = p.page_shift >= 0 ? t >> p.page_shift : t / p.page_size;
    page = id_of(pg);
    slot = static_cast<int32_t>(t - pg * p.page_size);
  }
  __device__ void look_up(uint32_t tile0) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < kLooks; ++i) {
      const uint32_t t = tile0 + i * 32 + lane;
      at[i] = 0;
      if (t >= end) continue;
      const uint32_t pg = p.page_shift >= 0 ? t >> p.page_shift : t / p.page_size;
      const int32_t id = id_of(pg);
      if (id < 0) continue;
      at[i] = view.base + static_cast<uint64_t>(id) * view.page + static_cast<uint64_t>(t - pg * p.page_size) * view.token + head;
    }
  }
  __device__ void copy(uint32_t to) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < kLooks; ++i)
#pragma unroll
      for (int j = 0; j < S::kVecs; ++j) {
        const int item = j * 32 + lane, row = item / S::kVecs, c = item % S::kVecs;
        const uint64_t from = __shfl_sync(~0u, at[i], row);
        const uint64_t x = from + c * 16;
        const bool read = from != 0 && in_bounds(reinterpret_cast<const void*>(x), 16, view.lo, view.hi, site);
        const uint32_t r = i * 32 + row;
        cp_async16_or_zero(to + (c / 8) * (S::kTile * 128) + r * 128 + ((c % 8) ^ (r & 7)) * 16, read ? x : view.base, read);
      }
  }
};

struct PrefixArgs {
  CUtensorMap k, v;  // (TMA)
  PrefixParams p;
};

// TMA: keys and values come in boxes of p.slots tokens of a page.
template <int DT, int D, bool TMA>
__global__ __launch_bounds__(kThreads, Shape<D>::kCtas) void dc_prefix_kernel(const __grid_constant__ PrefixArgs args) {
  using S = Shape<D>;
  const PrefixParams& p = args.p;
  extern __shared__ uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[4 * S::kStages + 3 * S::kScores + 2];
  __shared__ uint32_t tmem_at;
  __shared__ volatile uint32_t stop, lost;
  __shared__ uint32_t filled[2];  // (TMA) tiles whose copies were issued, of keys and of values
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // unit: (prefix, key head, chunk, rows)
  const int tile_rows = static_cast<int>(blockIdx.x % static_cast<uint32_t>(p.row_tiles)) * kPrefixRows;
  const uint32_t unit = blockIdx.x / static_cast<uint32_t>(p.row_tiles);
  const uint32_t chunk = unit % static_cast<uint32_t>(p.chunks);
  const int kh = static_cast<int>(unit / static_cast<uint32_t>(p.chunks) % static_cast<uint32_t>(p.kv_heads));
  const int prefix = static_cast<int>(unit / static_cast<uint32_t>(p.chunks) / static_cast<uint32_t>(p.kv_heads));

  // The kernel before, over the own tokens, has waited for all work before it in
  // every CTA by the time this one starts, and nothing here reads what it writes:
  // the two run side by side, and this one ends after it.  That what the work before
  // wrote is seen here too follows from the word that the other has released after its
  // wait; where it is not there yet, this kernel waits for all of the other.  Measured,
  // one after the other / side by side: 8 sequences of a group with 1025 tokens 20.6 /
  // 14.7 us, 4 groups of 16 with 7001 tokens each 49.7 / 45.2 us.
  pdl_launch_dependents();
  if (ld_acquire(p.ready) != 1) pdl_wait();
  bool bad;
  const uint32_t length = prefix_length(p, prefix, &bad);
  const uint32_t per = length ? prefix_chunk(length, p.kv_heads) : 1;
  const uint32_t first = chunk * per;
  if (first >= length) {
    pdl_wait();
    return;
  }
  const uint32_t end = min(length, first + per);
  const uint32_t tiles = (end - first + S::kTile - 1) / S::kTile;

  const uint32_t q_at = (smem_addr(smem) + 1023u) & ~1023u;
  const uint32_t k_at = q_at + S::kQ, v_at = k_at + S::kStages * S::kKV;
  const uint32_t k_full = smem_addr(bars), k_empty = k_full + 8 * S::kStages, v_full = k_empty + 8 * S::kStages,
                 v_empty = v_full + 8 * S::kStages, s_full = v_empty + 8 * S::kStages, p_full = s_full + 8 * S::kScores,
                 summed = p_full + 8 * S::kScores, q_full = summed + 8 * S::kScores, over = q_full + 8;
  if (threadIdx.x == 0) {
    for (int i = 0; i < S::kStages; ++i) {
      tma::mbar_init(k_full + 8 * i, TMA ? 1 : 32);
      tma::mbar_init(v_full + 8 * i, TMA ? 1 : 32);
      tma::mbar_init(k_empty + 8 * i, 1);
      tma::mbar_init(v_empty + 8 * i, 1);
    }
    for (int i = 0; i < S::kScores; ++i) {
      tma::mbar_init(s_full + 8 * i, 1);
      tma::mbar_init(p_full + 8 * i, 128);
      tma::mbar_init(summed + 8 * i, 1);
    }
    tma::mbar_init(q_full, kQueryLoaders);
    tma::mbar_init(over, 1);
    tma::mbar_init_fence();
    stop = 0;
    lost = bad ? 1u : 0u;
    filled[0] = filled[1] = 0;
  }
  if (warp == 4) tmem_alloc(smem_addr(&tmem_at), S::kColumns);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_at;
  const Waits waits{&stop, p.wait_ns};

  if (warp < 4) {
    // ---- a row a thread
    const int row = tile_rows + static_cast<int>(threadIdx.x);
    const bool used = tile_rows + warp * 32 < p.rows;  // (a warp without rows only keeps step)
    const uint32_t lanes = static_cast<uint32_t>(warp) * 32 << 16;
    const float sc = p.scale * kLog2E;
    float ref = neg_inf(), sum = 0.0f;
    bool ok = true;
    // Tile i's sum is done.  (A barrier for each buffer: its next phase needs this
    // thread's weights, so that it never runs two phases ahead.)
    auto wait_sum = [&](uint32_t i) { return ok = ok && wait(waits, summed + 8 * (i % S::kScores), (i / S::kScores) & 1); };
    for (uint32_t i = 0; i < tiles; ++i) {
      const uint32_t buf = i % S::kScores, at = tmem + lanes + buf * S::kTile;
      ok = wait(waits, s_full + 8 * buf, (i / S::kScores) & 1);
      if (i >= S::kScores) wait_sum(i - S::kScores);  // (done already: the scores waited for it)
      if (!__all_sync(~0u, ok)) break;
      fence_after();
      const uint32_t left = end - first - i * S::kTile;  // tokens of this tile, if it is the last
      if (used) {
        uint32_t r[2][32];
        tmem_ld32(at, r[0]);
        tmem_ld32(at + 32, r[1]);
        tmem_wait_ld(r[0]);
        tmem_wait_ld(r[1]);
        // the score that scale makes the largest: the largest, or (scale < 0) the smallest
        const float none = sc < 0.0f ? -neg_inf() : neg_inf();
        if (left < S::kTile) {
#pragma unroll
          for (int j = 0; j < S::kTile; ++j)
            if (static_cast<uint32_t>(j) >= left) r[j / 32][j % 32] = __float_as_uint(none);
        }
        float m[4] = {none, none, none, none};
        if (sc < 0.0f) {
#pragma unroll
          for (int j = 0; j < S::kTile; j += 2)
            m[j / 2 & 3] = min3(m[j / 2 & 3], __uint_as_float(r[j / 32][j % 32]), __uint_as_float(r[j / 32][j % 32 + 1]));
        } else {
#pragma unroll
          for (int j = 0; j < S::kTile; j += 2)
            m[j / 2 & 3] = max3(m[j / 2 & 3], __uint_as_float(r[j / 32][j % 32]), __uint_as_float(r[j / 32][j % 32 + 1]));
        }
        const float most = sc < 0.0f ? fminf(min3(m[0], m[1], m[2]), m[3]) : fmaxf(max3(m[0], m[1], m[2]), m[3]);
        // (of scale 0 the largest is 0, whatever the scores: NaN here moves nothing)
        const float up = ceilf(most * sc);
        // the reference follows once it is kSlack behind: until then weights are up to 2^kSlack
        const bool move = up > ref + kSlack;
        if (__any_sync(~0u, move)) {
          const float now = move ? up : ref, f = pow2_diff(ref, now);
          if (i > 0) {
            if (!__all_sync(~0u, wait_sum(i - 1))) break;
            fence_after();
#pragma unroll 1
            for (uint32_t d = 0; d < D; d += 32) {
              float v[32];
              tmem_ld32(tmem + lanes + S::kOut + d, v);
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] *= f;
              tmem_st32(tmem + lanes + S::kOut + d, v);
            }
          }
          sum *= f;
          ref = now;
        }
        float off = kShift<DT> - (ref == neg_inf() ? 0.0f : ref), by = sc;
        uint64_t l[2] = {0, 0};  // two sums each
        // A fused multiply-add takes the reference from a product that is not rounded, as the
        // own tokens' and the reference's are: beyond 2^14 that would show in the weights, and
        // far beyond in nothing else.
        if (fabsf(ref) >= 16384.0f && ref != neg_inf()) {
#pragma unroll
          for (int j = 0; j < S::kTile; ++j) r[j / 32][j % 32] = __float_as_uint(__uint_as_float(r[j / 32][j % 32]) * sc - ref);
          off = kShift<DT>;
          by = 1.0f;
        }
        __syncwarp();  // (tensor memory is a warp's to read and write)
        const uint64_t sc2 = pack2(by, by), off2 = pack2(off, off);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t w[16];
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            float x, y;
            unpack2(fma2(pack2(__uint_as_float(r[h][j]), __uint_as_float(r[h][j + 1])), sc2, off2), x, y);
            x = ex2(x);
            y = ex2(y);
            if (sc == 0.0f && left < S::kTile) {  // (what is behind the last token has no score to be told by)
              x = static_cast<uint32_t>(h * 32 + j) < left ? x : 0.0f;
              y = static_cast<uint32_t>(h * 32 + j + 1) < left ? y : 0.0f;
            }
            l[j / 2 & 1] = add2(l[j / 2 & 1], pack2(x, y));
            w[j / 2] = Elem<DT>::pack(x, y);
          }
          tmem_st16(at + h * 16, w);  // over scores that have been read
        }
        float l0, l1;
        unpack2(add2(l[0], l[1]), l0, l1);
        sum += l0 + l1;
        tmem_wait_st();
      }
      if (TMA && left < S::kTile) {
        // a copy brings whole boxes: values behind the last token have weight 0, but must be numbers
        const uint32_t st = i % S::kStages;
        ok = wait(waits, v_full + 8 * st, (i / S::kStages) & 1);
        if (!__all_sync(~0u, ok)) break;
        for (uint32_t c = threadIdx.x; c < (S::kTile - left) * S::kBlocks * 8; c += 128) {
          const uint32_t r = left + c / (S::kBlocks * 8), b = c / 8 % S::kBlocks;
          asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(v_at + st * S::kKV + b * (S::kTile * 128) + r * 128 + c % 8 * 16),
                       "r"(0u) : "memory");
        }
        tma::fence_proxy_async_smem();
      }
      fence_before();
      if (i == 0 && p.late == 1) come_late(p.wait_ns);
      mbar_arrive(p_full + 8 * buf);
    }
    if (tiles > 1) wait_sum(tiles - 2);
    wait_sum(tiles - 1);
    fence_after();
    asm volatile("bar.sync 1, 224;" ::: "memory");  // the copying warps have said what they missed
    if (used && __all_sync(~0u, ok)) {
      constexpr float kUnit = DT == kF16 ? 1.0f / 128.0f : 1.0f;
      const uint64_t at = (static_cast<uint64_t>(prefix) * p.kv_heads + kh) * p.chunks + chunk;
      const uint64_t all = static_cast<uint64_t>(p.prefixes) * p.kv_heads * p.chunks * p.rows;
      const uint64_t mine = at * p.rows + row;
#pragma unroll 1
      for (uint32_t d = 0; d < D; d += 32) {
        float v[32];
        __syncwarp();
        tmem_ld32(tmem + lanes + S::kOut + d, v);
        if (row >= p.rows) continue;
        float4* a = reinterpret_cast<float4*>(p.partial + (mine * D + d) * 4);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (in_bounds(a + j, 16, p.partial, p.partial + all * D * 4, kSitePartial))
            a[j] = make_float4(v[4 * j] * kUnit, v[4 * j + 1] * kUnit, v[4 * j + 2] * kUnit, v[4 * j + 3] * kUnit);
      }
      float2* b = reinterpret_cast<float2*>(p.partial_rl) + mine;
      if (row < p.rows && in_bounds(b, 8, p.partial_rl, p.partial_rl + all * 8, kSitePartial))
        *b = make_float2(ref, lost ? __int_as_float(0x7FC00000) : sum * kUnit);
    }
  } else if (warp == 4) {
    // ---- the products
    if (lane == 0) {
      constexpr uint32_t score = instruction<DT>(kPrefixRows, S::kTile, 0u), value = instruction<DT>(kPrefixRows, D, kMajorB);
      auto scores = [&](uint32_t i) {
        // they take the place of the weights kScores tiles before, which that tile's sum has to have read
        if (i >= S::kScores && !wait(waits, summed + 8 * (i % S::kScores), (i / S::kScores - 1) & 1)) return false;
        const uint32_t st = i % S::kStages, buf = i % S::kScores, k0 = k_at + st * S::kKV;
        if (!wait(waits, k_full + 8 * st, (i / S::kStages) & 1)) return false;
        fence_after();
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma(tmem + buf * S::kTile, desc_k(q_at + k / 4 * (kPrefixRows * 128) + k % 4 * 32),
              desc_k(k0 + k / 4 * (S::kTile * 128) + k % 4 * 32), score, k > 0);
        commit(s_full + 8 * buf);
        commit(k_empty + 8 * st);
        return true;
      };
      bool go = wait(waits, q_full, 0) && scores(0);
      for (uint32_t i = 0; i < tiles && go; ++i) {
        if (i + 1 < tiles) go = scores(i + 1);
        const uint32_t st = i % S::kStages, buf = i % S::kScores, v0 = v_at + st * S::kKV;
        go = go && wait(waits, v_full + 8 * st, (i / S::kStages) & 1) && wait(waits, p_full + 8 * buf, (i / S::kScores) & 1);
        if (!go) break;
        fence_after();
#pragma unroll
        for (int k = 0; k < S::kTile / 16; ++k)
          mma_tmem(tmem + S::kOut, tmem + buf * S::kTile + k * 8, desc_mn(v0 + k * 2048, S::kTile * 128), value, (i | k) != 0);
        commit(v_empty + 8 * st);
        commit(summed + 8 * buf);
      }
    }
    __syncwarp();
  } else {
    // ---- copies: queries first, then one warp the keys and one the values
    const bool values = warp == 6;
    const int id = static_cast<int>(threadIdx.x) - 160;
    for (int item = id; item < kPrefixRows * S::kVecs; item += kQueryLoaders) {
      const int r = item / S::kVecs, c = item % S::kVecs, row = tile_rows + r;
      const int seq = prefix * p.each + row / p.group, head = kh * p.group + row % p.group;
      const uint64_t from = p.q + static_cast<uint64_t>(seq) * p.q_seq + static_cast<uint64_t>(head) * p.q_head;
      const uint64_t x = from + c * 16;
      const bool read = row < p.rows && in_bounds(reinterpret_cast<const void*>(x), 16, from, from + D * 2, kSiteQuery);
      cp_async16_or_zero(q_at + (c / 8) * (kPrefixRows * 128) + r * 128 + ((c % 8) ^ (r & 7)) * 16, read ? x : p.q, read);
    }
    cp_async_commit();
    tma::fence_proxy_async_global();  // (keys and values may be an earlier kernel's stores)
    const PagedView& view = values ? p.vc : p.kc;
    Copier<D> copier{p, view, p.table + static_cast<uint64_t>(prefix) * static_cast<uint64_t>(p.table_stride) * 4,
                     static_cast<uint64_t>(kh) * view.head, end, values ? kSiteValue : kSiteKey, {}};
    const uint32_t full = values ? v_full : k_full, empty = values ? v_empty : k_empty, to = values ? v_at : k_at;
    bool q_told = false, go = true;
    if (warp != 7 && !bad) {
      if (TMA) copier.look_up_box(first, S::kTile / static_cast<uint32_t>(p.slots));
      else copier.look_up(first);
    }
    if (TMA && warp != 7) {
      // each lane copies a box of the tile
      const uint32_t boxes = S::kTile / static_cast<uint32_t>(p.slots);
      const CUtensorMap* map = values ? &args.v : &args.k;
      uint32_t i = 0;
      for (; i < tiles; ++i) {
        const uint32_t st = i % S::kStages, bar = full + 8 * st;
        if (i >= S::kStages && !__all_sync(~0u, wait(waits, empty + 8 * st, (i / S::kStages - 1) & 1))) break;
        if (i == 1 && values && p.late == 2) come_late(p.wait_ns);
        const int32_t page = copier.page, slot = copier.slot;
        const uint32_t there = __popc(__ballot_sync(~0u, page >= 0));
        if (lane == 0) tma::mbar_arrive_expect_tx(bar, there * static_cast<uint32_t>(p.slots) * 128 * S::kBlocks);
        __syncwarp();
        if (page >= 0) {
          const uint32_t dst = to + st * S::kKV + static_cast<uint32_t>(lane * p.slots) * 128;
#pragma unroll
          for (int b = 0; b < S::kBlocks; ++b) load_paged(dst + b * (S::kTile * 128), map, bar, b * 64, kh, slot, page);
        }
        if (i + 1 < tiles && !bad) copier.look_up_box(first + (i + 1) * S::kTile, boxes);
        if (i == 0) {
          cp_async_wait<0>();
          tma::fence_proxy_async_smem();
          mbar_arrive(q_full);
        }
      }
      if (lane == 0) filled[values] = i;
      go = false;
    }
    if (warp == 7) {
      cp_async_wait<0>();
      tma::fence_proxy_async_smem();
      mbar_arrive(q_full);
      go = false;
    }
    constexpr uint32_t kAhead = 2;  // tiles under way
    uint32_t issued = 0, told = 0;
    while (told < tiles && go) {
      const uint32_t st = issued % S::kStages;
      bool room = issued < tiles && issued - told < kAhead;
      if (room && issued >= S::kStages) {
        // wait for the place where nothing else is left to do
        const uint32_t parity = (issued / S::kStages - 1) & 1;
        if (issued == told) go = room = __all_sync(~0u, wait(waits, empty + 8 * st, parity));
        else room = __all_sync(~0u, tma::mbar_try_wait(empty + 8 * st, parity));
      }
      if (room) {
        if (issued == 1 && values && p.late == 2) come_late(p.wait_ns);
        copier.copy(to + st * S::kKV);
        cp_async_commit();
        ++issued;
        if (issued < tiles && !bad) copier.look_up(first + issued * S::kTile);
        if (issued < tiles && issued < kAhead) continue;
      }
      if (issued == told) continue;
      // the oldest copies are there: their place is the tensor cores'
      if (!q_told) {
        if (issued - told == 1) cp_async_wait<1>();
        else cp_async_wait<2>();
        tma::fence_proxy_async_smem();
        mbar_arrive(q_full);
        q_told = true;
      }
      if (issued - told == 1) cp_async_wait<0>();
      else cp_async_wait<1>();
      tma::fence_proxy_async_smem();
      mbar_arrive(full + 8 * (told % S::kStages));
      ++told;
    }
    cp_async_wait<0>();
    if (copier.missing) lost = 1;
    asm volatile("bar.sync 1, 224;" ::: "memory");
  }
  __syncthreads();
  pdl_wait();
  if (stop) {
    // Every thread has stopped: the copies and products in flight are waited for, which
    // read and write this CTA's shared and tensor memory.
    if (threadIdx.x == 0) atomicOr(&g_prefix_fault_bits, kFaultTensorWait);
    bool ended = true;
    if (threadIdx.x == 128) {  // (the thread that issued the products)
      commit(over);
      ended = tma::mbar_wait_bounded(over, 0, kDrainNs);
    }
    if (TMA && threadIdx.x < 2) {
      const uint32_t full = threadIdx.x ? v_full : k_full, end = filled[threadIdx.x];
      for (uint32_t k = end > S::kStages ? end - S::kStages : 0; k < end; ++k)
        ended = tma::mbar_wait_bounded(full + 8 * (k % S::kStages), (k / S::kStages) & 1, kDrainNs) && ended;
    }
    if (!ended) atomicOr(&g_prefix_fault_bits, kFaultTensorDrain);
    __syncthreads();
  }
  if (warp == 4) {
    fence_after();
    tmem_free(tmem, S::kColumns);
  }
}

// The prefix's chunks in order, then the own tokens: a warp a row, a lane every
// 32nd four columns.
constexpr int kJoinThreads = 128;
template <int DT, int D>
__global__ __launch_bounds__(kJoinThreads) void dc_prefix_join_kernel(const __grid_constant__ PrefixParams p) {
  pdl_enter();
  constexpr int kVecs = (D / 4 + 31) / 32;
  const int lane = threadIdx.x & 31;
  const uint64_t row = static_cast<uint64_t>(blockIdx.x) * (kJoinThreads / 32) + (threadIdx.x >> 5);
  const uint64_t n = static_cast<uint64_t>(p.seqs) * p.q_heads;
  if (blockIdx.x == 0 && threadIdx.x == 0) *reinterpret_cast<uint32_t*>(p.ready) = 0;  // (for the next call)
  if (row >= n) return;
  const int seq = static_cast<int>(row / static_cast<uint32_t>(p.q_heads)), head = static_cast<int>(row % static_cast<uint32_t>(p.q_heads));
  const int prefix = seq / p.each;
  bool bad;
  const uint32_t length = prefix_length(p, prefix, &bad), chunks = prefix_chunks(length, p.kv_heads);
  const uint64_t all = static_cast<uint64_t>(p.prefixes) * p.kv_heads * p.chunks * p.rows;
  const uint64_t at = (static_cast<uint64_t>(prefix) * p.kv_heads + head / p.group) * p.chunks * p.rows +
                      static_cast<uint64_t>(seq % p.each) * p.group + head % p.group;  // of chunk 0; the next is p.rows on
  const float2 own = reinterpret_cast<const float2*>(p.raw_rl)[row];
  auto chunk = [&](uint32_t c) {  // its reference and sum
    const float2* a = reinterpret_cast<const float2*>(p.partial_rl) + at + static_cast<uint64_t>(c) * p.rows;
    return c < chunks && in_bounds(a, 8, p.partial_rl, p.partial_rl + all * 8, kSitePartial) ? *a : make_float2(neg_inf(), 0.0f);
  };
  float2 held = chunk(lane);  // lane l's: of 32 chunks the l-th
  float most = fmaxf(own.x, held.x);
  for (uint32_t c = lane + 32; c < chunks; c += 32) most = fmaxf(most, chunk(c).x);
#pragma unroll
  for (int d = 16; d > 0; d /= 2) most = fmaxf(most, __shfl_xor_sync(~0u, most, d));
  float4 u[kVecs];
#pragma unroll
  for (int v = 0; v < kVecs; ++v) u[v] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float l = 0.0f;
  auto add = [&](const float4 (&x)[kVecs], float f, float part) {
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      u[v].x = __fmaf_rn(x[v].x, f, u[v].x);
      u[v].y = __fmaf_rn(x[v].y, f, u[v].y);
      u[v].z = __fmaf_rn(x[v].z, f, u[v].z);
      u[v].w = __fmaf_rn(x[v].w, f, u[v].w);
    }
    l = __fmaf_rn(part, f, l);
  };
  auto load = [&](float4 (&x)[kVecs], uint64_t from, uint64_t lo, uint64_t hi) {
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
      const float4* a = reinterpret_cast<const float4*>(from) + v * 32 + lane;
      x[v] = (v * 32 + lane) * 4 < D && in_bounds(a, 16, lo, hi, kSitePartial) ? *a : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
  };
  constexpr int kAtOnce = kVecs > 1 ? 4 : 8;
  for (uint32_t k = 0; k < chunks; k += 32) {
    if (k) held = chunk(k + lane);
    for (uint32_t c0 = k; c0 < min(chunks, k + 32); c0 += kAtOnce) {
      float4 x[kAtOnce][kVecs];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
        if (c0 + j < chunks)
          load(x[j], p.partial + (at + static_cast<uint64_t>(c0 + j) * p.rows) * D * 4, p.partial, p.partial + all * D * 4);
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
        if (c0 + j < chunks) {
          const float r = __shfl_sync(~0u, held.x, (c0 + j) % 32), s = __shfl_sync(~0u, held.y, (c0 + j) % 32);
          add(x[j], pow2_diff(r, most), s);
        }
    }
  }
  float4 x[kVecs];
  load(x, p.raw + row * D * 4, p.raw, p.raw + n * D * 4);
  add(x, pow2_diff(own.x, most), own.y);
  const bool none = l == 0.0f && most == neg_inf();  // nothing to attend to: zeros
  const float inv = none ? 0.0f : 1.0f / l;
  const uint64_t out = p.out + static_cast<uint64_t>(seq) * p.out_seq + static_cast<uint64_t>(head) * p.out_head;
#pragma unroll
  for (int v = 0; v < kVecs; ++v) {
    uint2* a = reinterpret_cast<uint2*>(out) + v * 32 + lane;
    if ((v * 32 + lane) * 4 < D && in_bounds(a, 8, out, out + D * 2, kSiteOut))
      *a = make_uint2(Elem<DT>::pack(u[v].x * inv, u[v].y * inv), Elem<DT>::pack(u[v].z * inv, u[v].w * inv));
  }
  if (lane == 0 && p.lse) {
    float* b = reinterpret_cast<float*>(p.lse) + row;
    if (in_bounds(b, 4, p.lse, p.lse + n * 4, kSiteOut)) *b = none ? neg_inf() : (most + log2f(l)) * kLn2;
  }
}

template <int DT, int D, bool TMA>
cudaError_t launch_one(const PrefixParams& p, bool pdl, cudaStream_t s, int grid) {
  static std::atomic<uint64_t> allowed{0};  // devices whose limit is set
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(allowed.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(dc_prefix_kernel<DT, D, TMA>, cudaFuncAttributeMaxDynamicSharedMemorySize, Shape<D>::kSmem);
    if (e != cudaSuccess) return e;
    allowed.fetch_or(bit, std::memory_order_relaxed);
  }
  PrefixArgs args{};
  args.p = p;
  if (TMA) {
    const uint32_t slots = static_cast<uint32_t>(p.slots);
    e = make_paged_map(&args.k, DT, p.kc, D, p.kv_heads, p.page_size, p.num_pages, slots);
    if (e == cudaSuccess) e = make_paged_map(&args.v, DT, p.vc, D, p.kv_heads, p.page_size, p.num_pages, slots);
    if (e != cudaSuccess) return e;
  }
  return launch_ex(dc_prefix_kernel<DT, D, TMA>, grid, kThreads, pdl, s, args, Shape<D>::kSmem);
}

template <int DT, int D>
cudaError_t launch_loads(const PrefixParams& p, bool pdl, cudaStream_t s, int grid) {
  return p.slots ? launch_one<DT, D, true>(p, pdl, s, grid) : launch_one<DT, D, false>(p, pdl, s, grid);
}

template <int DT>
cudaError_t launch_dim(const PrefixParams& p, int dim, bool join, bool pdl, cudaStream_t s, int grid) {
  switch (dim) {
    case 64: return join ? launch_ex(dc_prefix_join_kernel<DT, 64>, grid, kJoinThreads, pdl, s, p) : launch_loads<DT, 64>(p, pdl, s, grid);
    case 96: return join ? launch_ex(dc_prefix_join_kernel<DT, 96>, grid, kJoinThreads, pdl, s, p) : launch_loads<DT, 96>(p, pdl, s, grid);
    case 128: return join ? launch_ex(dc_prefix_join_kernel<DT, 128>, grid, kJoinThreads, pdl, s, p) : launch_loads<DT, 128>(p, pdl, s, grid);
    case 192: return join ? launch_ex(dc_prefix_join_kernel<DT, 192>, grid, kJoinThreads, pdl, s, p) : launch_loads<DT, 192>(p, pdl, s, grid);
    default: return join ? launch_ex(dc_prefix_join_kernel<DT, 256>, grid, kJoinThreads, pdl, s, p) : launch_loads<DT, 256>(p, pdl, s, grid);
  }
}

}  // namespace

cudaError_t launch_prefix(const PrefixParams& p, int dtype, int dim, bool pdl, cudaStream_t s, int* grid) {
  *grid = p.prefixes * p.kv_heads * p.chunks * p.row_tiles;
  return dtype == kF16 ? launch_dim<kF16>(p, dim, false, pdl, s, *grid) : launch_dim<kBF16>(p, dim, false, pdl, s, *grid);
}

cudaError_t launch_prefix_join(const PrefixParams& p, int dtype, int dim, bool pdl, cudaStream_t s, int* grid) {
  const uint64_t rows = static_cast<uint64_t>(p.seqs) * static_cast<uint64_t>(p.q_heads);
  *grid = static_cast<int>((rows + kJoinThreads / 32 - 1) / (kJoinThreads / 32));
  return dtype == kF16 ? launch_dim<kF16>(p, dim, true, pdl, s, *grid) : launch_dim<kBF16>(p, dim, true, pdl, s, *grid);
}

DC_BOUNDS_READER(take_bounds_prefix)

DC_FAULT_READER(take_prefix_faults, g_prefix_fault_bits)

}  // namespace dc
