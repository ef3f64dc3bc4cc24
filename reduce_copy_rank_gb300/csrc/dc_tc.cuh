// dc_tc.cuh -- the fifth-generation tensor cores and the TMA engine's tiled
// copies, as the language-model kernels use them: tcgen05.mma on shared-memory
// operands with accumulators in tensor memory, and 2-D tiled loads with a
// 128-byte swizzle.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include "dc_llm.h"
#include "dc_tma.cuh"

namespace dc {
namespace tc {

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// ---------------------------------------------------------- operand tiles ---
// Tiles lie in shared memory as rows of 128 bytes (64 elements of 16 bits)
// whose 16-byte parts are permuted by the row's number modulo 8 (the 128-byte
// swizzle): 8 rows are 1024 bytes, aligned to that.  A tile whose rows run
// along the product's inner dimension (K-major: a row is 64 of k for one m or
// n) and one whose rows run across it (MN-major: a row is 64 of m or n for one
// k) have the same bytes; the descriptor tells the tensor core which.

// The shared-memory descriptor: start / 16 in bits 0..13, leading and stride
// byte offsets / 16 in bits 16..29 and 32..45, 1 in bits 46..48 (this
// generation's format), the swizzle in bits 61..63 (2: 128 bytes).
__device__ __forceinline__ uint64_t desc(uint32_t addr, uint32_t leading, uint32_t stride) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | static_cast<uint64_t>(leading >> 4) << 16 |
         static_cast<uint64_t>(stride >> 4) << 32 | 1ull << 46 | 2ull << 61;
}
// K-major: groups of 8 rows are 1024 bytes apart (the leading offset is not
// used); 16 elements of k are 32 bytes on.
__device__ __forceinline__ uint64_t desc_k(uint32_t addr) { return desc(addr, 16, 1024); }
// MN-major: groups of 8 k are 1024 bytes apart, blocks of 64 m or n `block`
// bytes; 16 of k are 2048 bytes on.
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr, uint32_t block) { return desc(addr, block, 1024); }

// The instruction descriptor of kind::f16 with binary32 accumulators.
constexpr uint32_t kMajorA = 1u << 15, kMajorB = 1u << 16;  // MN-major operands
template <int DT>
__host__ __device__ constexpr uint32_t instruction(int m, int n, uint32_t flags) {
  return 1u << 4 | (DT == kBF16 ? 1u << 7 | 1u << 10 : 0u) | flags | static_cast<uint32_t>(n / 8) << 17 |
         static_cast<uint32_t>(m / 16) << 24;
}

// D (tensor memory) = A B, or += where `add`; one thread issues it.
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add))
      : "memory");
}

// The same with A in tensor memory: lane m, 2 elements of k a column.
__device__ __forceinline__ void mma_tmem(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add))
      : "memory");
}

// The mbarrier at `bar` gets one arrival when all tcgen05 work that this
// thread has issued is done.
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}

// ------------------------------------------------------------- CTA pairs ---
// Two CTAs of a cluster, on two SMs, multiply as one: a product of 256 rows, of
// which each CTA holds 128 (in its shared memory and, of the result, its tensor
// memory), and half of B's columns.  The even CTA issues; what it commits is told
// to both CTAs' barriers at the same address.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Shared memory at this CTA's address `a` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t a, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {  // (of cluster_addr)
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void st_cluster(uint32_t at, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_cluster(uint32_t at) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add))
      : "memory");
}
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
               "h"(static_cast<uint16_t>(3))
               : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(columns) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free_pair(uint32_t at, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns) : "memory");
}

__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// ---------------------------------------------------------- tensor memory ---
// One whole warp allocates and frees; the address lands in shared memory.
__device__ __forceinline__ void tmem_alloc(uint32_t dst, uint32_t columns) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst), "r"(columns) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t at, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(columns) : "memory");
}

// 32 columns of this warp's 32 lanes: thread l gets lane l's (the address's
// lane is the warp's first: 32 * (warp % 4)).
// (The values may be used after tmem_wait_ld, which names them: loads of other
// columns can be under way while one's values are worked on.)
__device__ __forceinline__ void tmem_ld32(uint32_t at, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at)
      : "memory");
}
// Waits for every load of this thread; `r` is what one of them has brought.
__device__ __forceinline__ void tmem_wait_ld(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                 "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
// 16 columns, waited for.
__device__ __forceinline__ void tmem_ld16(uint32_t at, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at)
      : "memory");
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
// Both: 32 columns as numbers.
__device__ __forceinline__ void tmem_ld32(uint32_t at, float (&v)[32]) {
  uint32_t r[32];
  tmem_ld32(at, r);
  tmem_wait_ld(r);
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}
// The other way: 32 or 16 columns from each thread's words.
__device__ __forceinline__ void tmem_st32(uint32_t at, const float (&v)[32]) {
  uint32_t r[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(v[i]);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
      "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]),
      "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(at)
      : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ------------------------------------------------------------ packed numbers ---
// Two binary32 numbers an instruction, each rounded as alone.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// The largest or smallest of three numbers.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// --------------------------------------------------------------- mbarriers ---
__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

// What the waits of a CTA share: once one has run out all give up at once.
struct Waits {
  volatile uint32_t* stop;  // in shared memory, 0 at first
  uint64_t limit_ns;
};
// (Each try suspends the thread for a while; the clock, which is slow to read,
// is looked at now and then.)
__device__ __forceinline__ bool wait(const Waits& w, uint32_t bar, uint32_t parity) {
  uint32_t done;  // (a look that does not suspend is quicker where the phase has completed)
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  if (done) return true;
  uint64_t t0 = 0;
  for (uint32_t i = 0; i < tma::kMaxPolls; ++i) {
    if (tma::mbar_try_wait(bar, parity)) return true;
    if (*w.stop) return false;
    if ((i & 31) == 31) {
      const uint64_t now = tma::global_ns();
      if (t0 == 0) t0 = now;
      else if (now - t0 >= w.limit_ns) break;
    }
  }
  *w.stop = 1;
  return false;
}

// Once a CTA has given up, its copies and products in flight still read and write
// shared and tensor memory: it leaves when they are done, however short the limit
// was that ran out.
constexpr uint64_t kDrainNs = 10000000000ull;

// Test kernels' lateness: twice the limit (bounded also where the clock stands still).
__device__ __forceinline__ void come_late(uint64_t limit_ns) {
  const uint64_t t0 = tma::global_ns();
  for (uint32_t i = 0; i < 1u << 22 && tma::global_ns() - t0 < 2 * limit_ns; ++i) __nanosleep(1000);
}

// ------------------------------------------------------------- tiled loads ---
// The box of `map` at column x (a multiple of 16 bytes) of a paged cache: key head, slot
// and page; places outside the tensor read 0.
__device__ __forceinline__ void load_paged(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t head,
                                           int32_t slot, int32_t page) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(x), "r"(head), "r"(slot), "r"(page)
      : "memory");
}
// The tile at column x and row y of a matrix, into this CTA's shared memory, counted by
// a barrier of either CTA of the pair (a cluster_addr).
__device__ __forceinline__ void load_tile_pair(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t x, int32_t y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// A map over rows x columns of 16-bit elements (row stride in bytes, a multiple
// of 16), in tiles of 64 columns x tile_rows rows, swizzled by 128 bytes.
cudaError_t make_map(CUtensorMap* map, int dtype, uint64_t base, uint64_t rows, uint64_t columns, uint64_t row_stride,
                     uint32_t tile_rows);
// ... over a paged cache (strides in bytes), in boxes of 64 columns of one head
// and `slots` neighbouring tokens of a page.
cudaError_t make_paged_map(CUtensorMap* map, int dtype, const PagedView& v, int dim, int heads, uint32_t page_size,
                           int64_t pages, uint32_t slots);

// cudaError_t NAME(uint32_t* bits): reads and clears a file's fault word WORD.
#define DC_FAULT_READER(NAME, WORD)                              \
  cudaError_t NAME(uint32_t* bits) {                             \
    *bits = 0;                                                   \
    cudaError_t e = cudaDeviceSynchronize();                     \
    if (e != cudaSuccess) return e;                              \
    unsigned int v = 0;                                          \
    e = cudaMemcpyFromSymbol(&v, WORD, sizeof v);                \
    if (e == cudaSuccess && v) {                                 \
      const unsigned int zero = 0;                               \
      e = cudaMemcpyToSymbol(WORD, &zero, sizeof zero);          \
    }                                                            \
    *bits = v;                                                   \
    return e;                                                    \
  }

}  // namespace tc
}  // namespace dc
