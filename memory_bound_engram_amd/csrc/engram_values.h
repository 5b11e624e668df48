// engram_values.h -- eight neighbouring values of a row, bf16, fp16 or fp32, as
// they lie in memory and as fp32 (gfx950, internal).
#pragma once

#include "engram_device.h"

namespace engram {

struct bf16_t { uint16_t v; };

// Eight values as they lie in memory.
template <typename T>
struct Raw {
  u32x4 w[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw<T> load_raw(const T* p) {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = load16(reinterpret_cast<const u32x4*>(p) + i);
  return r;
}
template <typename T>
__device__ __forceinline__ Raw<T> zero_raw() {
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = u32x4{0, 0, 0, 0};
  return r;
}
__device__ __forceinline__ void unpack8(const Raw<bf16_t>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf_lo(r.w[0][i]);
    v[2 * i + 1] = bf_hi(r.w[0][i]);
  }
}
__device__ __forceinline__ void unpack8(const Raw<_Float16>& r, float (&v)[8]) {
  typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
  const f16x8 h = __builtin_bit_cast(f16x8, r.w[0]);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (float)h[i];
}
__device__ __forceinline__ void unpack8(const Raw<float>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r.w[i / 4][i % 4]);
}
// kStream: the line is not kept in the caches.
template <bool kStream>
__device__ __forceinline__ void put16(void* p, u32x4 v) {
  if (kStream) store16_stream(p, v);
  else store16(p, v);
}
template <bool kStream>
__device__ __forceinline__ void store8(bf16_t* p, const float (&v)[8]) {
  u32x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
  put16<kStream>(p, r);
}
template <bool kStream>
__device__ __forceinline__ void store8(_Float16* p, const float (&v)[8]) {
  typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
  f16x8 r;
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = (_Float16)v[i];
  put16<kStream>(p, __builtin_bit_cast(u32x4, r));
}
template <bool kStream>
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  u32x4 a, b;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[i] = __float_as_uint(v[i]);
    b[i] = __float_as_uint(v[i + 4]);
  }
  put16<kStream>(p, a);
  put16<kStream>(p + 4, b);
}

// Four neighbouring values, likewise.
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
template <typename T>
struct Raw4 {
  u32x2 w[sizeof(T) / 2];
};
template <bool kStream = false, typename T>
__device__ __forceinline__ Raw4<T> load_raw4(const T* p) {
  if constexpr (sizeof(T) == 4) return __builtin_bit_cast(Raw4<T>, kStream ? load16_stream(p) : load16(p));
  else if constexpr (kStream) return Raw4<T>{{__builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p))}};
  else return Raw4<T>{{*reinterpret_cast<const u32x2*>(p)}};
}
template <typename T>
__device__ __forceinline__ Raw4<T> zero_raw4() {
  Raw4<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.w[i] = u32x2{0, 0};
  return r;
}
__device__ __forceinline__ void unpack4(const Raw4<bf16_t>& r, float (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v[2 * i] = bf_lo(r.w[0][i]);
    v[2 * i + 1] = bf_hi(r.w[0][i]);
  }
}
__device__ __forceinline__ void unpack4(const Raw4<_Float16>& r, float (&v)[4]) {
  typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
  const f16x4 h = __builtin_bit_cast(f16x4, r.w[0]);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = (float)h[i];
}
__device__ __forceinline__ void unpack4(const Raw4<float>& r, float (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r.w[i / 2][i % 2]);
}
template <bool kStream>
__device__ __forceinline__ void put8(void* p, u32x2 v) {
  if (kStream) __builtin_nontemporal_store(v, reinterpret_cast<u32x2*>(p));
  else *reinterpret_cast<u32x2*>(p) = v;
}
template <bool kStream>
__device__ __forceinline__ void store4(bf16_t* p, const float (&v)[4]) {
  put8<kStream>(p, u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])});
}
template <bool kStream>
__device__ __forceinline__ void store4(_Float16* p, const float (&v)[4]) {
  typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
  f16x4 r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = (_Float16)v[i];
  put8<kStream>(p, __builtin_bit_cast(u32x2, r));
}
template <bool kStream>
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
  put16<kStream>(p, u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])});
}

}  // namespace engram
