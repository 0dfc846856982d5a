// Device-side helpers of the linear-layer operators: element types, 8-bit
// packing and the block scale.
#pragma once

#include <hip/hip_runtime.h>

#include "linear.hpp"

namespace mr {

typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
typedef float f4 __attribute__((ext_vector_type(4)));
// The same at any address: one load or store instruction all the same (the
// hardware takes unaligned vector accesses), so rows of odd widths move like
// the others.
typedef v4u v4u_any __attribute__((aligned(1)));
typedef v2u v2u_any __attribute__((aligned(1)));

struct bf16_t {
  uint16_t bits;
};

// float32 of a stored value, and the stored type's nearest value (ties to even).
__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(_Float16 v) { return (float)v; }
__device__ __forceinline__ float widen(bf16_t v) { return __uint_as_float((uint32_t)v.bits << 16); }
template <typename T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ float narrow<float>(float v) {
  return v;
}
template <>
__device__ __forceinline__ _Float16 narrow<_Float16>(float v) {
  return (_Float16)v;
}
template <>
__device__ __forceinline__ bf16_t narrow<bf16_t>(float v) {
  const __bf16 b = (__bf16)v;
  bf16_t r;
  __builtin_memcpy(&r, &b, 2);
  return r;
}

// Eight consecutive values as they are stored, at any address: 16 bytes (twice that for float32).
template <typename T>
struct Raw8 {
  v4u u[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw8<T> load8(const T* p) {
  Raw8<T> r;
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) r.u[i] = reinterpret_cast<const v4u_any*>(p)[i];
  return r;
}
__device__ __forceinline__ void widen8(const Raw8<float>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r.u[i >> 2][i & 3]);
}
__device__ __forceinline__ void widen8(const Raw8<bf16_t>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(r.u[0][i] << 16);
    v[2 * i + 1] = __uint_as_float(r.u[0][i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void widen8(const Raw8<_Float16>& r, float (&v)[8]) {
  _Float16 h[8];
  __builtin_memcpy(h, &r, 16);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = (float)h[i];
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
  T t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = narrow<T>(v[i]);
  Raw8<T> r;
  __builtin_memcpy(&r, t, sizeof r);
#pragma unroll
  for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<v4u_any*>(p)[i] = r.u[i];
}

// Four values in 8 bits (ties to even; the callers' scale keeps them in range).
__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d, bool e5m2) {
  int r = 0;
  if (e5m2) {
    r = __builtin_amdgcn_cvt_pk_bf8_f32(a, b, r, false);
    r = __builtin_amdgcn_cvt_pk_bf8_f32(c, d, r, true);
  } else {
    r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, r, false);
    r = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
  }
  return (uint32_t)r;
}

// Magnitudes are compared as their bits: ordered like the values, with NaN
// above infinity, so that a block that holds a NaN gets a NaN scale.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Largest of the 16 lanes of a DPP row, in every one of them.
__device__ __forceinline__ uint32_t max16(uint32_t v) {
  v = umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xf, 0xf, false));  // row_ror:8
  v = umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xf, 0xf, false));
  v = umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xf, 0xf, false));
  v = umax(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xf, 0xf, false));
  return v;
}
__device__ __forceinline__ uint32_t max64(uint32_t v) {
  v = max16(v);
  v = umax(v, (uint32_t)__shfl_xor((int)v, 16));
  return umax(v, (uint32_t)__shfl_xor((int)v, 32));
}
__device__ __forceinline__ float sum64(float v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

// Scale of a block from its largest magnitude; 0 magnitudes give 2^-100 / top.
__device__ __forceinline__ float block_scale(uint32_t amax, bool e5m2) {
  const float a = __uint_as_float(umax(amax, __float_as_uint(kSmallestAmax)));
  return a / (e5m2 ? kE5m2Max : kE4m3Max);
}

// Values of a block over its scale, the float32 quotient (nearest, ties to even):
// the product with the rounded reciprocal is at most a place off, and the
// remainder v - q s, which one fused operation gives exactly, says by how much
// (Markstein's method).  The product alone turns ties of the 8-bit rounding,
// which 16-bit inputs meet often.  8191 x 1024 bf16 in both orders: 13.2 us, with
// the product alone 12.9, with the full division 16.4.  (Values below 2^-102 lose
// places of the remainder, which ties can stand down to 2^-124.)
struct Quotient {
  float inv, s;  // an infinite scale: 0 for finite values, NaN for infinite ones, without its remainder
  __device__ __forceinline__ explicit Quotient(float scale)
      : inv(1.f / scale), s(__builtin_isinf(scale) ? 0.f : scale) {}
  __device__ __forceinline__ float operator()(float v) const {
    const float q = v * inv;
    return fmaf(fmaf(-q, s, v), inv, q);
  }
};

}  // namespace mr
