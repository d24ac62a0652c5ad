// Row access of the embedding, loss and optimizer kernels: 16-byte vectors of
// a row whose start need only be aligned to its elements (rows of an odd
// width start anywhere), float32 values of them, and workgroup reductions.
#pragma once

#include "lora_device.hpp"

namespace lora {

// 16 bytes at any address that is a multiple of the element size (gfx950
// loads and stores them in one instruction at any byte address).
template <class E>
struct Vec;
template <>
struct Vec<uint16_t> {
  static constexpr int N = 8;
  typedef unsigned int type __attribute__((ext_vector_type(4), aligned(2)));
  static __device__ __forceinline__ void unpack(type w, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ type pack(const float* f) {
    type w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = bf16_bits(f[2 * i]) | (bf16_bits(f[2 * i + 1]) << 16);
    return w;
  }
  static __device__ __forceinline__ float value(uint16_t v) { return bf16_value(v); }
  static __device__ __forceinline__ uint16_t round(float v) { return static_cast<uint16_t>(bf16_bits(v)); }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  typedef unsigned int type __attribute__((ext_vector_type(4), aligned(4)));
  static __device__ __forceinline__ void unpack(type w, float* f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(w[i]);
  }
  static __device__ __forceinline__ type pack(const float* f) {
    type w;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(f[i]);
    return w;
  }
  static __device__ __forceinline__ float value(float v) { return v; }
  static __device__ __forceinline__ float round(float v) { return v; }
};

template <class E>
__device__ __forceinline__ typename Vec<E>::type vload(const E* p) {
  return *reinterpret_cast<const typename Vec<E>::type*>(p);
}
template <class E>
__device__ __forceinline__ typename Vec<E>::type vload_nt(const E* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const typename Vec<E>::type*>(p));
}
template <class E>
__device__ __forceinline__ void vstore_nt(E* p, typename Vec<E>::type v) {
  __builtin_nontemporal_store(v, reinterpret_cast<typename Vec<E>::type*>(p));
}
template <class E>
__device__ __forceinline__ void vstore(E* p, typename Vec<E>::type v) {
  *reinterpret_cast<typename Vec<E>::type*>(p) = v;
}

// N consecutive elements of a row as float32 and back; N is a multiple of the vector's.
template <int N, class E>
__device__ __forceinline__ void load_row(const E* p, float* f) {
#pragma unroll
  for (int i = 0; i < N; i += Vec<E>::N) Vec<E>::unpack(vload_nt(p + i), f + i);
}
template <int N, class E>
__device__ __forceinline__ void store_row(E* p, const float* f) {
#pragma unroll
  for (int i = 0; i < N; i += Vec<E>::N) vstore_nt(p + i, Vec<E>::pack(f + i));
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}

}  // namespace lora
