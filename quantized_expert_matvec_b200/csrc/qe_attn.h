// qe_attn.h -- what the cache append and the attention over the cache share:
// limits, the division by the page size and 16-bit packing.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "qe_internal.h"

namespace qe {

constexpr int kMaxPageSize = 65536;
constexpr int kMaxHeads = 1024;

// n / d for n < 2^31: with 2^s >= d and m = ceil(2^(31+s) / d), m d exceeds
// 2^(31+s) by less than d <= 2^s, so n m / 2^(31+s) exceeds n / d by less than
// 1 / d and floors to the quotient.  m <= 2^32 - 1 unless d = 1 gives 2^31.
struct FastDiv {
  uint32_t d, m, s;
  __host__ __device__ __forceinline__ uint32_t div(uint32_t n) const { return (uint32_t)(((uint64_t)n * m) >> (31 + s)); }
};
inline FastDiv fast_div(uint32_t d) {
  FastDiv f{d, 0, 0};
  while ((1u << f.s) < d) ++f.s;
  f.m = (uint32_t)(((1ull << (31 + f.s)) + d - 1) / d);
  return f;
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

int check_kv_cache(const qe_kv_cache* c);
// n rows of `row` bytes, `stride` bytes apart
struct Rows {
  const void* p;
  size_t row, stride;
  int n;
};
bool rows_overlap(const Rows& a, const Rows& b);  // a.n == b.n

}  // namespace qe
