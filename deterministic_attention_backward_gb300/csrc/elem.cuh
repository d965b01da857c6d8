// elem.cuh -- element types of the memory-bound operators (bf16, fp16, fp32): vectors of V
// elements (16 bytes, or one element where sizes or addresses do not allow more), converted
// to and from fp32.  Conversions to a narrower type round to nearest even.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <type_traits>

#include "f32x2.cuh"

namespace dash {

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) {
  return __bfloat162float(x);
}
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// V elements as they lie in memory: one 16-byte access for V = 16 / sizeof(T), an element
// access for V = 1.
template <typename T, int V>
struct alignas(V * sizeof(T)) Pack {
  T e[V];
};
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_pack(const T *p) {
  static_assert(V == 1 || V * sizeof(T) == 16, "16-byte vectors or single elements");
  Pack<T, V> r;
  if constexpr (V == 1)
    r.e[0] = *p;
  else
    *reinterpret_cast<uint4 *>(&r) = *reinterpret_cast<const uint4 *>(p);
  return r;
}
template <typename T, int V>
__device__ __forceinline__ void store_pack(T *p, const Pack<T, V> &r) {
  if constexpr (V == 1)
    *p = r.e[0];
  else
    *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(&r);
}
template <typename T, int V>
__device__ __forceinline__ void unpack(const Pack<T, V> &r, float (&f)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = to_f32<T>(r.e[i]);
}
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> pack(const float (&f)[V]) {
  Pack<T, V> r;
#pragma unroll
  for (int i = 0; i < V; ++i) r.e[i] = from_f32<T>(f[i]);
  return r;
}

// A 16-byte vector as pairs of fp32 values, and back.
template <typename T>
__device__ __forceinline__ void unpack2(const uint4 &v, f2 (&f)[8 / sizeof(T)]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  if constexpr (sizeof(T) == 4) {
    f[0] = f2_of(w[0], w[1]);
    f[1] = f2_of(w[2], w[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const T *e = reinterpret_cast<const T *>(&w[i]);
      f[i] = f2_of(to_f32<T>(e[0]), to_f32<T>(e[1]));
    }
  }
}
template <>
__device__ __forceinline__ void unpack2<__nv_bfloat16>(const uint4 &v, f2 (&f)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = f2_of(w[i] << 16, w[i] & 0xffff0000u);
}
template <typename T>
__device__ __forceinline__ uint4 pack2(const f2 (&f)[8 / sizeof(T)]) {
  uint32_t w[4];
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float a, b;
      f2_to(f[i], a, b);
      w[2 * i] = __float_as_uint(a), w[2 * i + 1] = __float_as_uint(b);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      f2_to(f[i], a, b);
      if constexpr (std::is_same<T, __half>::value) {
        const __half2 h = __floats2half2_rn(a, b);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
      }
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace dash
