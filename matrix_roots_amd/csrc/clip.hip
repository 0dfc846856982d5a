// Clipping of many gradients by their common norm:
//
//   n_i = ||G_i||, n = (sum_i n_i^2)^(1/2),  G_i <- G_i c,
//   c = max_norm / n where n is finite and larger than max_norm, else 1.
//
// Squares, their sums and the factor are float64: a float32 square overflows or
// vanishes from 2^64 and 2^-64 on, and the sums of a billion terms keep their
// places.  A scaled value is the float64 product, rounded to the output's type
// through float32.
#include <math.h>

#include "clip.hpp"
#include "linear_common.hpp"
#include "mr_common.hpp"

namespace mr {

namespace {

__device__ __forceinline__ double sum64d(double v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}

__device__ __forceinline__ int job_of(const ClipBatch& B, int b) {
  int j = 0;
  while (j + 1 < B.njobs && b >= B.job[j + 1].block_begin) ++j;
  return j;
}

// f(place in the input, place in the output, how many values are left of the row)
// for the workgroup's units of a job: eight values of a row, or what is left of it.
template <typename F>
__device__ __forceinline__ void for_units(const ClipJob& J, int64_t blk, int64_t per, F&& f) {
  const int64_t in_row = (J.cols + 7) / 8, all = J.rows * in_row;
  const int64_t begin = blk * per, end = begin + per < all ? begin + per : all;
  if (J.rows == 1) {
#pragma unroll 4
    for (int64_t u = begin + threadIdx.x; u < end; u += 256) f(8 * u, 8 * u, J.cols - 8 * u);
  } else {
    for (int64_t u = begin + threadIdx.x; u < end; u += 256) {
      const int64_t r = u / in_row, c = 8 * (u - r * in_row);
      f(r * J.ldg + c, r * J.ldo + c, J.cols - c);
    }
  }
}

template <typename T>
__device__ __forceinline__ void load_some(const T* p, int64_t n, float (&v)[8]) {
  if (n >= 8) {
    widen8(load8<T>(p), v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.f;
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < n) v[i] = widen(p[i]);
}
template <typename T>
__device__ __forceinline__ void store_some(T* p, int64_t n, const float (&v)[8]) {
  if (n >= 8) {
    store8<T>(p, v);
    return;
  }
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < n) p[i] = narrow<T>(v[i]);
}

template <typename T>
__device__ __forceinline__ double squares_of(const ClipJob& J, int64_t blk, int64_t per) {
  const T* g = reinterpret_cast<const T*>(J.g);
  double s = 0.0, t = 0.0;
  for_units(J, blk, per, [&](int64_t in, int64_t, int64_t n) {
    float v[8];
    load_some<T>(g + in, n, v);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      s = fma((double)v[i], (double)v[i], s);
      t = fma((double)v[i + 1], (double)v[i + 1], t);
    }
  });
  return s + t;
}

template <typename T, typename O>
__device__ __forceinline__ void scale_to(const ClipJob& J, int64_t blk, int64_t per, double by) {
  const T* g = reinterpret_cast<const T*>(J.g);
  O* o = reinterpret_cast<O*>(J.out);
  for_units(J, blk, per, [&](int64_t in, int64_t out, int64_t n) {
    float v[8];
    load_some<T>(g + in, n, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)((double)v[i] * by);
    store_some<O>(o + out, n, v);
  });
}

}  // namespace

__global__ __launch_bounds__(256) void clip_squares_kernel(const ClipBatch B) {
  __shared__ double red[4];
  const int j = job_of(B, blockIdx.x);
  const ClipJob& J = B.job[j];
  const int blk = (int)blockIdx.x - J.block_begin;
  double s = J.dtype == MR_F32   ? squares_of<float>(J, blk, B.per_block)
             : J.dtype == MR_F16 ? squares_of<_Float16>(J, blk, B.per_block)
                                 : squares_of<bf16_t>(J, blk, B.per_block);
  s = sum64d(s);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    B.partial[J.slot + blk] = red[0] + red[1] + red[2] + red[3];
    if (blk == 0) B.first[B.first_problem + j] = J.slot;
  }
}

// Each gradient's partial sums by a wave, then all gradients' squares by the first.
__global__ __launch_bounds__(1024) void clip_norms_kernel(const double* partial, const int32_t* first, int count,
                                                          int slots, double max_norm, double* norms, double* by) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int i = wave; i < count; i += 16) {
    double s = 0.0;
    const int end = i + 1 < count ? first[i + 1] : slots;
    for (int b = first[i] + lane; b < end; b += 64) s += partial[b];
    s = sum64d(s);
    if (lane == 0) norms[1 + i] = s;
  }
  __threadfence_block();
  __syncthreads();
  if (wave == 0) {
    double s = 0.0;
    for (int i = lane; i < count; i += 64) s += norms[1 + i];
    s = sum64d(s);
    if (lane == 0) {
      const double n = sqrt(s);
      norms[0] = n;
      if (by) *by = n > max_norm && !isinf(n) ? max_norm / n : 1.0;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < count; i += 1024) norms[1 + i] = sqrt(norms[1 + i]);
}

__global__ __launch_bounds__(256) void clip_scale_kernel(const ClipBatch B) {
  const ClipJob& J = B.job[job_of(B, blockIdx.x)];
  const double by = *B.by;
  if (by == 1.0 && J.out == J.g) return;
  const int blk = (int)blockIdx.x - J.block_begin;
  if (J.dtype == MR_F32)
    scale_to<float, float>(J, blk, B.per_block, by);
  else if (J.dtype == MR_F16)
    J.out_dtype == MR_F32 ? scale_to<_Float16, float>(J, blk, B.per_block, by)
                          : scale_to<_Float16, _Float16>(J, blk, B.per_block, by);
  else
    J.out_dtype == MR_F32 ? scale_to<bf16_t, float>(J, blk, B.per_block, by)
                          : scale_to<bf16_t, bf16_t>(J, blk, B.per_block, by);
}

// ------------------------------------------------------------ launchers
hipError_t launch_clip_squares(const ClipBatch& b, hipStream_t s) {
  hipLaunchKernelGGL(clip_squares_kernel, dim3(b.total_blocks), dim3(256), 0, s, b);
  return hipGetLastError();
}
hipError_t launch_clip_norms(const double* partial, const int32_t* first, int count, int slots, double max_norm,
                             double* norms, double* by, hipStream_t s) {
  hipLaunchKernelGGL(clip_norms_kernel, dim3(1), dim3(1024), 0, s, partial, first, count, slots, max_norm, norms, by);
  return hipGetLastError();
}
hipError_t launch_clip_scale(const ClipBatch& b, hipStream_t s) {
  hipLaunchKernelGGL(clip_scale_kernel, dim3(b.total_blocks), dim3(256), 0, s, b);
  return hipGetLastError();
}

}  // namespace mr
