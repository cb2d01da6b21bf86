// Vectors of float elements in memory of any alignment (gfx950's vector
// memory instructions take byte-aligned addresses), converted to and from fp32.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxq {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
// the same with the alignment of the element that they are loaded over
typedef u32x4 u32x4_any __attribute__((aligned(1)));
typedef u32x2 u32x2_any __attribute__((aligned(1)));

__device__ __forceinline__ float load_f(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float load_f(const uint16_t* p, int64_t i) { return __uint_as_float((uint32_t)p[i] << 16); }

__device__ __forceinline__ uint16_t bf16_of(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }  // to nearest even
__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  b2 v = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ void store_f(float* p, int64_t i, float v) { p[i] = v; }
__device__ __forceinline__ void store_f(uint16_t* p, int64_t i, float v) { p[i] = bf16_of(v); }

// W consecutive elements as they lie in memory, one instruction's worth: fp32
// one or four at a time, bf16 one, four or eight.
template <typename T, int W>
struct Raw;
template <typename T>
struct Raw<T, 1> {
  T a;
};
template <>
struct Raw<float, 4> {
  u32x4 a;
};
template <>
struct Raw<uint16_t, 4> {
  u32x2 a;
};
template <>
struct Raw<uint16_t, 8> {
  u32x4 a;
};
template <typename T, int W>
struct RawPtr;
template <typename T>
struct RawPtr<T, 1> {
  typedef T type;
};
template <>
struct RawPtr<float, 4> {
  typedef u32x4_any type;
};
template <>
struct RawPtr<uint16_t, 4> {
  typedef u32x2_any type;
};
template <>
struct RawPtr<uint16_t, 8> {
  typedef u32x4_any type;
};

// NT: past the caches' retention, for data that is touched once
template <int W, bool NT, typename T>
__device__ __forceinline__ Raw<T, W> load_raw(const T* p) {
  const typename RawPtr<T, W>::type* q = reinterpret_cast<const typename RawPtr<T, W>::type*>(p);
  if (NT) return {__builtin_nontemporal_load(q)};
  return {*q};
}

__device__ __forceinline__ void unpack(const Raw<float, 4>& r, float* f) {
#pragma unroll
  for (int j = 0; j < 4; j++) f[j] = __uint_as_float(r.a[j]);
}
__device__ __forceinline__ void unpack(const Raw<float, 1>& r, float* f) { f[0] = r.a; }
__device__ __forceinline__ void unpack(const Raw<uint16_t, 1>& r, float* f) { f[0] = __uint_as_float((uint32_t)r.a << 16); }
template <int W>
__device__ __forceinline__ void unpack(const Raw<uint16_t, W>& r, float* f) {
#pragma unroll
  for (int j = 0; j < W / 2; j++) {
    f[2 * j] = __uint_as_float(r.a[j] << 16);
    f[2 * j + 1] = __uint_as_float(r.a[j] & 0xFFFF0000u);
  }
}

template <int W, bool NT>
__device__ __forceinline__ void store_vec(float* p, const float* f) {
  if constexpr (W == 1) {
    *p = f[0];
    return;
  }
#pragma unroll
  for (int k = 0; k < W / 4; k++) {
    u32x4 a;
#pragma unroll
    for (int j = 0; j < 4; j++) a[j] = __float_as_uint(f[4 * k + j]);
    u32x4_any* q = reinterpret_cast<u32x4_any*>(p) + k;
    if (NT)
      __builtin_nontemporal_store(a, q);
    else
      *q = a;
  }
}
template <int W, bool NT>
__device__ __forceinline__ void store_vec(uint16_t* p, const float* f) {
  if constexpr (W == 1) {
    *p = bf16_of(f[0]);
  } else {
    Raw<uint16_t, W> r;
#pragma unroll
    for (int j = 0; j < W / 2; j++) r.a[j] = bf16x2_of(f[2 * j], f[2 * j + 1]);
    typename RawPtr<uint16_t, W>::type* q = reinterpret_cast<typename RawPtr<uint16_t, W>::type*>(p);
    if (NT)
      __builtin_nontemporal_store(r.a, q);
    else
      *q = r.a;
  }
}

}  // namespace mxq
