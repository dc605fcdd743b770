// Element types of the operators around the layer: loads to binary32 and
// stores rounded to nearest even, one element or eight at a time.
#pragma once

#include "common.hpp"

namespace nvfp4 {

// Word, value(): an element's bits and its binary32 value.
struct Bf16 {
  static constexpr int kBytes = 2;
  using Word = uint16_t;
  __device__ static float value(Word w) { return __uint_as_float(static_cast<uint32_t>(w) << 16); }
  __device__ static float get(const void* p, int64_t i) {
    return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16);
  }
  __device__ static uint32_t bits(float f) {
    return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));  // the converter keeps NaN a NaN
  }
  __device__ static void put(void* p, int64_t i, float f) {
    static_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(bits(f));
  }
  __device__ static void unpack(uint32_t w, float& lo, float& hi) {
    lo = bf16_lo(w);
    hi = bf16_hi(w);
  }
};

struct F16 {
  static constexpr int kBytes = 2;
  using Word = _Float16;
  __device__ static float value(Word w) { return static_cast<float>(w); }
  __device__ static float get(const void* p, int64_t i) {
    return static_cast<float>(static_cast<const _Float16*>(p)[i]);
  }
  __device__ static uint32_t bits(float f) { return __builtin_bit_cast(uint16_t, static_cast<_Float16>(f)); }
  __device__ static void put(void* p, int64_t i, float f) {
    static_cast<_Float16*>(p)[i] = static_cast<_Float16>(f);
  }
  __device__ static void unpack(uint32_t w, float& lo, float& hi) {
    const half2v h = __builtin_bit_cast(half2v, w);
    lo = static_cast<float>(h[0]);
    hi = static_cast<float>(h[1]);
  }
};

struct F32 {
  static constexpr int kBytes = 4;
  using Word = float;
  __device__ static float value(Word w) { return w; }
  __device__ static float get(const void* p, int64_t i) { return static_cast<const float*>(p)[i]; }
  __device__ static void put(void* p, int64_t i, float f) { static_cast<float*>(p)[i] = f; }
};

// The raw bits of eight consecutive elements (16-byte aligned).
template <typename T>
struct Raw8 {
  u32x4 v[T::kBytes / 2];
};

template <typename T>
__device__ __forceinline__ void load8(Raw8<T>& r, const void* p, int64_t i) {
  const u32x4* s = reinterpret_cast<const u32x4*>(static_cast<const char*>(p) + i * T::kBytes);
#pragma unroll
  for (int j = 0; j < T::kBytes / 2; ++j) r.v[j] = s[j];
}

// The same where a row starts anywhere (its elements are aligned): global
// memory is read in 16-byte pieces at any address.
template <typename T>
__device__ __forceinline__ void load8_any(Raw8<T>& r, const void* p, int64_t i) {
  __builtin_memcpy(&r, static_cast<const char*>(p) + i * T::kBytes, sizeof(r));
}

template <typename T>
__device__ __forceinline__ void to_f32(const Raw8<T>& r, float (&f)[8]) {
  if constexpr (T::kBytes == 4) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(r.v[j / 4][j % 4]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) T::unpack(r.v[0][j], f[2 * j], f[2 * j + 1]);
  }
}

template <typename T>
__device__ __forceinline__ void from_f32(Raw8<T>& r, const float (&f)[8]) {
  if constexpr (T::kBytes == 4) {
#pragma unroll
    for (int j = 0; j < 8; ++j) r.v[j / 4][j % 4] = __float_as_uint(f[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) r.v[0][j] = T::bits(f[2 * j]) | (T::bits(f[2 * j + 1]) << 16);
  }
}
template <typename T>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&f)[8]) {
  Raw8<T> r;
  from_f32<T>(r, f);
  u32x4* d = reinterpret_cast<u32x4*>(static_cast<char*>(p) + i * T::kBytes);
#pragma unroll
  for (int j = 0; j < T::kBytes / 2; ++j) d[j] = r.v[j];
}
template <typename T>
__device__ __forceinline__ void store8_any(void* p, int64_t i, const float (&f)[8]) {
  Raw8<T> r;
  from_f32<T>(r, f);
  __builtin_memcpy(static_cast<char*>(p) + i * T::kBytes, &r, sizeof(r));
}

// Four elements at any address.
template <typename T>
__device__ __forceinline__ void store4_any(void* p, int64_t i, const float (&f)[4]) {
  char* d = static_cast<char*>(p) + i * T::kBytes;
  if constexpr (T::kBytes == 4) {
    __builtin_memcpy(d, f, sizeof(f));
  } else {
    const u32x2 w = {T::bits(f[0]) | (T::bits(f[1]) << 16), T::bits(f[2]) | (T::bits(f[3]) << 16)};
    __builtin_memcpy(d, &w, sizeof(w));
  }
}

}  // namespace nvfp4
