// elem.cuh -- element types of the memory-bound operators (bf16, fp16, fp32): vectors of V
// elements (16 bytes, or one element where sizes or addresses do not allow more), converted
// to and from fp32.  Conversions to a narrower type round to nearest even.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

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

}  // namespace dash
