// Device-side helpers of the norms: how a row lies among threads, and its sums.
#pragma once

#include "linear_common.hpp"

namespace mr {

// A thread's chunk k of a row: the 8 columns from 8 (t + TPR k), t its place among
// the row's threads; 16 lanes make a scale block.  The last chunk of a row may
// be a part of one.
template <int TPR>
__device__ __forceinline__ int chunk_col(int t, int k) {
  return 8 * (t + TPR * k);
}
template <typename T>
__device__ __forceinline__ void load_chunk(const T* row, int c, int width, float (&v)[8]) {
  if (c + 8 <= width) {
    widen8(load8<T>(row + c), v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.f;
  if (c < width) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (c + i < width) v[i] = widen(row[c + i]);
  }
}
template <typename T>
__device__ __forceinline__ void store_chunk(T* row, int c, int width, const float (&v)[8]) {
  if (c + 8 <= width) {
    store8<T>(row + c, v);
  } else if (c < width) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (c + i < width) row[c + i] = narrow<T>(v[i]);
  }
}
// Columns c .. c + 7 of a parameter vector, float32 or of the rows' type.
template <typename T>
__device__ __forceinline__ void load_param(const void* p, int f32, int c, int width, float (&v)[8]) {
  if (f32)
    load_chunk<float>(reinterpret_cast<const float*>(p), c, width, v);
  else
    load_chunk<T>(reinterpret_cast<const T*>(p), c, width, v);
}
// The chunk in 8 bits with its block's scale; q and s are the row's.  All 64 lanes take part.
__device__ __forceinline__ void store_eight(unsigned char* q, float* s, int c, int width, const float (&v)[8], bool e5m2) {
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) amax = umax(amax, magnitude(v[i]));
  amax = max16(amax);
  const float sb = block_scale(amax, e5m2);
  const Quotient over(sb);
  if (c < width && (threadIdx.x & 15) == 0) s[c / kBlock] = sb;
  v2u p;
  p[0] = pack4(over(v[0]), over(v[1]), over(v[2]), over(v[3]), e5m2);
  p[1] = pack4(over(v[4]), over(v[5]), over(v[6]), over(v[7]), e5m2);
  if (c + 8 <= width) {
    *reinterpret_cast<v2u_any*>(q + c) = p;
  } else if (c < width) {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (c + i < width) q[c + i] = (unsigned char)(p[i >> 2] >> (8 * (i & 3)));
  }
}

// Sum over the row's threads, in each of them.
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = sum64(v);
  if constexpr (TPR == 64) return v;
  const int wave = threadIdx.x >> 6;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[wave] = v;
  __syncthreads();
  float s = red[0];
#pragma unroll
  for (int w = 1; w < TPR / 64; ++w) s += red[w];
  return s;
}

// CH chunks per thread; workgroups of 256 threads (256 / TPR rows at a time) or
// of TPR.
template <int TPR>
constexpr int kNormThreads = TPR < 256 ? 256 : TPR;

}  // namespace mr
