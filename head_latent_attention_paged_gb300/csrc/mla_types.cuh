// Element types of the layer operators: loads to and stores from 32 bits.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace mla {

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }

// Rounded once, to nearest even.
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// A 32-bit word's values (one of f32, two of the 16-bit types, the first in
// the low half) and back, rounded once.
template <typename T>
struct Word;
template <>
struct Word<float> {
  static constexpr int kElems = 1;
  static __device__ __forceinline__ void get(uint32_t w, float* v) { v[0] = __uint_as_float(w); }
  static __device__ __forceinline__ uint32_t put(const float* v) { return __float_as_uint(v[0]); }
};
template <>
struct Word<__nv_bfloat16> {
  static constexpr int kElems = 2;
  static __device__ __forceinline__ void get(uint32_t w, float* v) {
    v[0] = __uint_as_float(w << 16);
    v[1] = __uint_as_float(w & 0xFFFF0000u);
  }
  static __device__ __forceinline__ uint32_t put(const float* v) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[0], v[1]);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};
template <>
struct Word<__half> {
  static constexpr int kElems = 2;
  static __device__ __forceinline__ void get(uint32_t w, float* v) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
    v[0] = f.x;
    v[1] = f.y;
  }
  static __device__ __forceinline__ uint32_t put(const float* v) {
    const __half2 h = __floats2half2_rn(v[0], v[1]);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
};

// 16 bytes of elements as f32 and back.
template <typename T>
__device__ __forceinline__ void unpack16(const uint4& w, float* v) {
  Word<T>::get(w.x, v);
  Word<T>::get(w.y, v + Word<T>::kElems);
  Word<T>::get(w.z, v + 2 * Word<T>::kElems);
  Word<T>::get(w.w, v + 3 * Word<T>::kElems);
}
template <typename T>
__device__ __forceinline__ uint4 pack16(const float* v) {
  return make_uint4(Word<T>::put(v), Word<T>::put(v + Word<T>::kElems), Word<T>::put(v + 2 * Word<T>::kElems),
                    Word<T>::put(v + 3 * Word<T>::kElems));
}

}  // namespace mla
