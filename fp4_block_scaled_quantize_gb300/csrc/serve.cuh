// serve.cuh -- what the serving kernels (matvec.cu, append.cu, attention16.cuh)
// share: 16-bit element types, conversions and launch geometry.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "common.cuh"
#include "formats.cuh"

namespace fp4 {

__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) {
  return __float2half_rn(v);
}
template <>
__device__ __forceinline__ float from_f32<float>(float v) {
  return v;
}

// Two values as a pair of T, the first low, and back.
template <typename T>
__device__ __forceinline__ uint32_t pack(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
template <>
__device__ __forceinline__ uint32_t pack<__half>(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
template <typename T>
__device__ __forceinline__ float2 unpack(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack<__nv_bfloat16>(uint32_t w) {
  return make_float2(bf16_lo(w), bf16_hi(w));
}
template <>
__device__ __forceinline__ float2 unpack<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2 *>(&w));
}

// Four E4M3 codes as two pairs of f16.
__device__ __forceinline__ void e4m3_halves(uint32_t w, uint32_t &lo, uint32_t &hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// i / d for 0 <= i < 2^31 by a multiplication: with 2^(l - 1) < d <= 2^l and m =
// ceil(2^(31 + l) / d), which is below 2^32 for d > 1, m d exceeds 2^(31 + l)
// by less than d <= 2^l, so i m / 2^(31 + l) exceeds i / d by less than 1 / d.
struct Divisor {
  uint32_t m;
  int shift;  // l - 1; -1: d = 1
};
inline Divisor divisor(int d) {
  int l = 0;
  while (((int64_t)1 << l) < d) ++l;
  if (l == 0) return {0, -1};
  return {(uint32_t)((((uint64_t)1 << (31 + l)) + d - 1) / d), l - 1};
}
__device__ __forceinline__ int over(int i, const Divisor &d) {
  return d.shift < 0 ? i : (int)(__umulhi((uint32_t)i, d.m) >> d.shift);
}

// log2 of a power of two, else `other`.
inline int log2_or(int v, int other) {
  if (v < 1 || (v & (v - 1)) != 0) return other;
  int e = 0;
  while (1 << e < v) ++e;
  return e;
}

// Multiprocessors of the current device (asked once per device).
inline int sm_count() {
  constexpr int kMaxDev = 64;
  static std::atomic<int> cache[kMaxDev];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  if (dev >= 0 && dev < kMaxDev) {
    const int c = cache[dev].load(std::memory_order_relaxed);
    if (c > 0) return c;
  }
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 1;
  if (dev >= 0 && dev < kMaxDev) cache[dev].store(n, std::memory_order_relaxed);
  return n;
}

}  // namespace fp4
