// Clipping of many gradients by their common norm:
//
//   n_i = ||G_i||, n = (sum_i n_i^2)^(1/2),  G_i <- G_i c,
//   c = max_norm / n where n is finite and larger than max_norm, else 1.
//
// Squares, their sums and the factor are float64: a float32 square overflows or
// vanishes from 2^64 and 2^-64 on, and the sums of a billion terms keep their
// places.  A scaled value is the float64 product, rounded to the output's type
// through float32.
//
// HBM-bound, in two launches: squares (one sum for each workgroup), then the
// scaling, each of whose workgroups adds all sums up by itself in one order.
#include <math.h>

#include "clip.hpp"
#include "linear_common.hpp"
#include "mr_common.hpp"

namespace mr {

namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;  // units of eight values that a thread loads before it works on them

__device__ __forceinline__ double sum64d(double v) {
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) v += __shfl_xor(v, m);
  return v;
}
__device__ __forceinline__ double block_sum(double v, double* red) {
  v = sum64d(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = red[0];
  for (int w = 1; w < (int)blockDim.x / 64; ++w) s += red[w];
  return s;
}

// The launch's gradient that workgroup b belongs to: every lane looks at two.
template <typename Jobs>
__device__ __forceinline__ int job_of(const ClipBatch<Jobs>& B, int b) {
  const int lane = threadIdx.x & 63;
  int n = __popcll(__ballot(lane < B.njobs && B.job.begin[lane < B.njobs ? lane : 0] <= b));
  if constexpr (Jobs::kJobs > 64) n += __popcll(__ballot(lane + 64 < B.njobs && B.job.begin[lane + 64 < B.njobs ? lane + 64 : 0] <= b));
  return __builtin_amdgcn_readfirstlane(n - 1);
}

template <typename T>
__device__ __forceinline__ Raw8<T> load_some(const T* p, int64_t n) {
  T t[8] = {};
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < n) t[i] = p[i];
  Raw8<T> r;
  __builtin_memcpy(&r, t, sizeof r);
  return r;
}
template <typename T>
__device__ __forceinline__ void store_some(T* p, int64_t n, const float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < n) p[i] = narrow<T>(v[i]);
}

// use(eight values as they are stored, their place in the output, how many of them
// are there) for the units [begin, end) of gradient j.
template <typename T, typename Jobs, typename F>
__device__ __forceinline__ void for_units(const ClipBatch<Jobs>& B, int j, int64_t begin, int64_t end, F&& use) {
  const T* g = reinterpret_cast<const T*>(B.job.g[j]);
  const int64_t cols = B.job.cols[j];
  if constexpr (Jobs::kRows) {
    const int64_t in_row = (cols + 7) / 8, all = B.job.rows[j] * in_row, ldg = B.job.ldg[j], ldo = B.job.ldo[j];
    if (end > all) end = all;
    for (int64_t u = begin + threadIdx.x; u < end; u += kThreads) {
      const int64_t r = u / in_row, c = 8 * (u - r * in_row), n = cols - c;
      const T* p = g + r * ldg + c;
      use(n >= 8 ? load8<T>(p) : load_some<T>(p, n), r * ldo + c, n);
    }
  } else {
    const int64_t whole = cols / 8;
    const int64_t to = end < whole ? end : whole;
    int64_t u = begin + threadIdx.x;
    for (; u + (kAhead - 1) * kThreads < to; u += kAhead * kThreads) {
      Raw8<T> r[kAhead];
#pragma unroll
      for (int q = 0; q < kAhead; ++q) r[q] = load8<T>(g + 8 * (u + q * kThreads));
#pragma unroll
      for (int q = 0; q < kAhead; ++q) use(r[q], 8 * (u + q * kThreads), 8);
    }
    for (; u < to; u += kThreads) use(load8<T>(g + 8 * u), 8 * u, 8);
    if (whole >= begin && whole < end && threadIdx.x == 0 && cols > 8 * whole)
      use(load_some<T>(g + 8 * whole, cols - 8 * whole), 8 * whole, cols - 8 * whole);
  }
}

template <typename T, typename Jobs>
__device__ __forceinline__ double squares_of(const ClipBatch<Jobs>& B, int j, int64_t begin, int64_t end) {
  double s = 0.0, t = 0.0;
  for_units<T>(B, j, begin, end, [&](const Raw8<T>& r, int64_t, int64_t) {
    float v[8];
    widen8(r, v);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      s = fma((double)v[i], (double)v[i], s);
      t = fma((double)v[i + 1], (double)v[i + 1], t);
    }
  });
  return s + t;
}

template <typename T, typename O, typename Jobs>
__device__ __forceinline__ void scale_to(const ClipBatch<Jobs>& B, int j, int64_t begin, int64_t end, double by) {
  O* o = reinterpret_cast<O*>(B.job.out[j]);
  for_units<T>(B, j, begin, end, [&](const Raw8<T>& r, int64_t at, int64_t n) {
    float v[8];
    widen8(r, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)((double)v[i] * by);
    if (n >= 8)
      store8<O>(o + at, v);
    else
      store_some<O>(o + at, n, v);
  });
}

}  // namespace

template <typename Jobs>
__global__ __launch_bounds__(kThreads) void clip_squares_kernel(const ClipBatch<Jobs> B) {
  __shared__ double red[4];
  const int j = job_of(B, blockIdx.x);
  const int64_t begin = ((int64_t)blockIdx.x - B.job.begin[j]) * B.per;
  const int type = B.job.type[j] & 15;
  double s = type == MR_F32   ? squares_of<float>(B, j, begin, begin + B.per)
             : type == MR_F16 ? squares_of<_Float16>(B, j, begin, begin + B.per)
                              : squares_of<bf16_t>(B, j, begin, begin + B.per);
  s = block_sum(s, red);
  if (threadIdx.x == 0) B.partial[B.slot + blockIdx.x] = s;
}

// One sum of all partial sums, where they are many.
__global__ __launch_bounds__(1024) void clip_fold_kernel(const double* partial, int slots, double* sum) {
  __shared__ double red[16];
  double s = 0.0;
#pragma unroll 4
  for (int i = threadIdx.x; i < slots; i += 1024) s += partial[i];
  s = block_sum(s, red);
  if (threadIdx.x == 0) *sum = s;
}

// Workgroups in the opposite order: what the squares read last is still in the last-level cache.
template <typename Jobs>
__global__ __launch_bounds__(kThreads) void clip_scale_kernel(const ClipBatch<Jobs> B) {
  __shared__ double red[4];
  const int b = B.blocks - 1 - (int)blockIdx.x;
  double s = 0.0;
#pragma unroll 8
  for (int i = threadIdx.x; i < B.nsums; i += kThreads) s += B.sums[i];
  s = block_sum(s, red);
  const double n = sqrt(s);
  if (B.slot == 0 && b == 0 && threadIdx.x == 0) B.norms[0] = n;
  const int j = job_of(B, b);
  const int first = B.job.begin[j];
  if (b == first) {  // the gradient's own norm
    const int last = j + 1 < B.njobs ? B.job.begin[j + 1] : B.blocks;
    double own = 0.0;
    for (int i = first + threadIdx.x; i < last; i += kThreads) own += B.partial[B.slot + i];
    own = block_sum(own, red);
    if (threadIdx.x == 0) B.norms[1 + B.job.problem[j]] = sqrt(own);
  }
  const double by = n > B.max_norm && !isinf(n) ? B.max_norm / n : 1.0;
  if (by == 1.0 && B.job.out[j] == B.job.g[j]) return;
  const int64_t begin = ((int64_t)b - first) * B.per, end = begin + B.per;
  const int type = B.job.type[j] & 15;
  const bool wide = B.job.type[j] >> 4 == MR_F32;
  if (type == MR_F32)
    scale_to<float, float>(B, j, begin, end, by);
  else if (type == MR_F16)
    wide ? scale_to<_Float16, float>(B, j, begin, end, by) : scale_to<_Float16, _Float16>(B, j, begin, end, by);
  else
    wide ? scale_to<bf16_t, float>(B, j, begin, end, by) : scale_to<bf16_t, bf16_t>(B, j, begin, end, by);
}

// ------------------------------------------------------------ launchers
template <typename Jobs>
hipError_t launch_clip_squares(const ClipBatch<Jobs>& b, hipStream_t s) {
  hipLaunchKernelGGL((clip_squares_kernel<Jobs>), dim3(b.blocks), dim3(kThreads), 0, s, b);
  return hipGetLastError();
}
template <typename Jobs>
hipError_t launch_clip_scale(const ClipBatch<Jobs>& b, hipStream_t s) {
  hipLaunchKernelGGL((clip_scale_kernel<Jobs>), dim3(b.blocks), dim3(kThreads), 0, s, b);
  return hipGetLastError();
}
template hipError_t launch_clip_squares(const ClipBatch<ClipFlat>&, hipStream_t);
template hipError_t launch_clip_squares(const ClipBatch<ClipRows>&, hipStream_t);
template hipError_t launch_clip_scale(const ClipBatch<ClipFlat>&, hipStream_t);
template hipError_t launch_clip_scale(const ClipBatch<ClipRows>&, hipStream_t);

hipError_t launch_clip_fold(const double* partial, int slots, double* sum, hipStream_t s) {
  hipLaunchKernelGGL(clip_fold_kernel, dim3(1), dim3(1024), 0, s, partial, slots, sum);
  return hipGetLastError();
}

}  // namespace mr
