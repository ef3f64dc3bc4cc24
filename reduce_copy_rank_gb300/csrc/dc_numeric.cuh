// dc_numeric.cuh -- element types, base-2 exponentials and the order of
// floating-point keys, shared by the language-model operators.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "dc_device.cuh"
#include "dc_internal.h"

namespace dc {

constexpr float kLog2E = 1.44269504088896340736f;
constexpr float kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float neg_inf() { return __int_as_float(static_cast<int>(0xFF800000u)); }

// 2^x in one instruction (ex2.approx: at most 2 ulp off; results below 2^-126 are 0).
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The larger of two numbers, NaN if either is (fmaxf drops NaN).
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// The 16-bit number next below the one with bits h, twice in a word; -inf
// (bits 0x8000 | inf) stays, and so do NaN and +inf, whose sums are NaN anyway.
__device__ __forceinline__ uint32_t detail_below2(uint32_t h, uint32_t inf) {
  const uint32_t mag = h & 0x7FFFu;
  if (mag < inf) h = (h & 0x8000u) ? h + 1 : mag ? h - 1 : 0x8001u;
  return h | (h << 16);
}

// Element types: DT is kBF16, kF16 or kF32.
template <int DT>
struct Elem;

template <>
struct Elem<kBF16> {
  static constexpr int kBytes = 2;
  static constexpr int kPerVec = 8;                        // elements in 16 bytes
  static constexpr uint32_t kNegInfWord = 0xFF80FF80u;     // 4 bytes of -inf
  __device__ static __forceinline__ float lo(uint32_t w) { return bf16lo_to_f32(w); }
  __device__ static __forceinline__ float hi(uint32_t w) { return bf16hi_to_f32(w); }
  __device__ static __forceinline__ uint32_t pack(float a, float b) { return pack_bf16x2_rn(a, b); }
  __device__ static __forceinline__ uint16_t bits(float a) { return f32_to_bf16_rn(a); }
  __device__ static __forceinline__ float one(uint16_t h) { return __uint_as_float(static_cast<uint32_t>(h) << 16); }
  // both halves' larger values, NaN if either is
  __device__ static __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  // two copies of a number below x (at most two steps of the type below), -inf if there is none
  __device__ static __forceinline__ uint32_t below2(float x) { return detail_below2(bits(x), 0x7F80u); }
};

template <>
struct Elem<kF16> {
  static constexpr int kBytes = 2;
  static constexpr int kPerVec = 8;
  static constexpr uint32_t kNegInfWord = 0xFC00FC00u;
  __device__ static __forceinline__ float lo(uint32_t w) { return f16_to_f32(static_cast<uint16_t>(w)); }
  __device__ static __forceinline__ float hi(uint32_t w) { return f16_to_f32(static_cast<uint16_t>(w >> 16)); }
  __device__ static __forceinline__ uint32_t pack(float a, float b) { return pack_f16x2_rn(a, b); }
  __device__ static __forceinline__ uint16_t bits(float a) { return f32_to_f16_rn(a); }
  __device__ static __forceinline__ float one(uint16_t h) { return f16_to_f32(h); }
  __device__ static __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
  }
  __device__ static __forceinline__ uint32_t below2(float x) { return detail_below2(bits(x), 0x7C00u); }
};

template <>
struct Elem<kF32> {
  static constexpr int kBytes = 4;
  static constexpr int kPerVec = 4;
  static constexpr uint32_t kNegInfWord = 0xFF800000u;
  __device__ static __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    return __float_as_uint(max_nan(__uint_as_float(a), __uint_as_float(b)));
  }
};

// The larger element of a word.
template <int DT>
__device__ __forceinline__ float word_max(uint32_t w) {
  if constexpr (DT == kF32) return __uint_as_float(w);
  else return max_nan(Elem<DT>::lo(w), Elem<DT>::hi(w));
}

// The elements of a 16-byte vector as binary32 (exact).
template <int DT>
__device__ __forceinline__ void unpack(const uint4& v, float (&x)[Elem<DT>::kPerVec]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == kF32) {
      x[i] = __uint_as_float(w[i]);
    } else {
      x[2 * i] = Elem<DT>::lo(w[i]);
      x[2 * i + 1] = Elem<DT>::hi(w[i]);
    }
  }
}

// ... and back, each rounded once to nearest even.
template <int DT>
__device__ __forceinline__ uint4 repack(const float (&x)[Elem<DT>::kPerVec]) {
  uint4 v;
  if constexpr (DT == kF32) {
    v = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  } else {
    v = make_uint4(Elem<DT>::pack(x[0], x[1]), Elem<DT>::pack(x[2], x[3]), Elem<DT>::pack(x[4], x[5]),
                   Elem<DT>::pack(x[6], x[7]));
  }
  return v;
}

// One element at a byte address (coherent).
template <int DT>
__device__ __forceinline__ float load_elem(uint64_t addr) {
  if constexpr (DT == kF32) return *reinterpret_cast<const float*>(addr);
  else return Elem<DT>::one(*reinterpret_cast<const uint16_t*>(addr));
}

template <int DT>
__device__ __forceinline__ void store_elem(uint64_t addr, float x) {
  if constexpr (DT == kF32) *reinterpret_cast<float*>(addr) = x;
  else *reinterpret_cast<uint16_t*>(addr) = Elem<DT>::bits(x);
}

// An unsigned integer that orders as the number does; +0 and -0 are equal,
// NaN comes before -inf.
__device__ __forceinline__ uint32_t ordered(float x) {
  if (x != x) return 0;
  const uint32_t b = __float_as_uint(x + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
  return __uint_as_float((u & 0x80000000u) ? (u & 0x7FFFFFFFu) : ~u);
}

}  // namespace dc
