// Clipping of many gradients by their common norm:
//
//   n_i = ||G_i||, n = (sum_i n_i^2)^(1/2),  G_i <- G_i c,
//   c = max_norm / n where n is finite and larger than max_norm, else 1.
//
// Squares, their sums and the factor are float64: a float32 square overflows from
// 2^64 on and loses places below 2^-63, and sums of a billion terms keep theirs.
// A scaled value is the float64 product, rounded to the output's type through
// float32 (twice at most for 16-bit outputs: half a step and 2^-24 of it).
//
// HBM-bound, in two launches: squares (one sum for each workgroup), then the
// scaling, each of whose workgroups adds all sums up by itself in one order.  58
// float32 gradients of 100.7 M values: 69 us for the squares (403 MB, 5.8 TB/s) and
// 8.6 for a scaling that changes nothing (246 for both where all are scaled in place,
// 1.2 GB, 4.9 TB/s, passes one after another); 17 bf16 gradients of 103.8 M values into
// float32: 40 and 101 us from a clean cache, 175 for both in passes one after another
// (831 MB).  A lane's load or store is 16 bytes wherever the wider type allows, so
// that an instruction covers whole lines: 177 us, with 32-byte lanes 187.
#include <math.h>

#include "clip.hpp"
#include "linear_common.hpp"
#include "mr_common.hpp"

namespace mr {

namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 8;  // loads of a thread before it works on their values (175 us; 4: 181, 12: 180)

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

// V values as they are stored, at any address: 8 or 16 bytes in one load.
template <typename T, int V>
struct Values {
  typedef uint32_t u __attribute__((ext_vector_type(sizeof(T) * V / 4)));
  typedef u any __attribute__((aligned(1)));
};
template <int V, typename T>
__device__ __forceinline__ void load_values(const T* p, T (&v)[V]) {
  const typename Values<T, V>::u r = *reinterpret_cast<const typename Values<T, V>::any*>(p);
  __builtin_memcpy(v, &r, sizeof r);
}
template <int V, typename T>
__device__ __forceinline__ void store_values(T* p, const T (&v)[V]) {
  typename Values<T, V>::u r;
  __builtin_memcpy(&r, v, sizeof r);
  *reinterpret_cast<typename Values<T, V>::any*>(p) = r;
}

// use(V values as they are stored, their place in the output, how many of them are
// there; zeros behind) for the units [begin, end) of gradient j.  Lanes take
// neighbouring V, so that V of 16 bytes makes whole lines of each instruction.
template <typename T, int V, typename Jobs, typename F>
__device__ __forceinline__ void for_values(const ClipBatch<Jobs>& B, int j, int64_t begin, int64_t end, F&& use) {
  const T* g = reinterpret_cast<const T*>(B.job.g[j]);
  const int64_t cols = B.job.cols[j];
  auto some = [&](const T* p, int64_t n, int64_t at) {
    T v[V] = {};
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (i < n) v[i] = p[i];
    use(v, at, n);
  };
  if constexpr (Jobs::kRows) {
    const int64_t in_row = (cols + 7) / 8, all = B.job.rows[j] * in_row, ldg = B.job.ldg[j], ldo = B.job.ldo[j];
    if (end > all) end = all;
    for (int64_t u = begin + threadIdx.x; u < end; u += kThreads) {
      const int64_t r = u / in_row, c0 = 8 * (u - r * in_row);
#pragma unroll
      for (int64_t c = c0; c < c0 + 8; c += V) {
        const T* p = g + r * ldg + c;
        T v[V];
        if (c + V <= cols) {
          load_values<V>(p, v);
          use(v, r * ldo + c, V);
        } else if (c < cols) {
          some(p, cols - c, r * ldo + c);
        }
      }
    }
  } else {
    const int64_t whole = cols / V * V, to = 8 * end < whole ? 8 * end : whole;
    constexpr int64_t step = V * kThreads;
    int64_t i = 8 * begin + V * (int64_t)threadIdx.x;
    for (; i + (kAhead - 1) * step < to; i += kAhead * step) {
      T v[kAhead][V];
#pragma unroll
      for (int q = 0; q < kAhead; ++q) load_values<V>(g + i + q * step, v[q]);
#pragma unroll
      for (int q = 0; q < kAhead; ++q) use(v[q], i + q * step, V);
    }
    for (; i < to; i += step) {
      T v[V];
      load_values<V>(g + i, v);
      use(v, i, V);
    }
    if (threadIdx.x == 0 && whole < cols && whole >= 8 * begin && whole < 8 * end) some(g + whole, cols - whole, whole);
  }
}

template <typename T, typename Jobs>
__device__ __forceinline__ double squares_of(const ClipBatch<Jobs>& B, int j, int64_t begin, int64_t end) {
  constexpr int V = 16 / sizeof(T);
  double s = 0.0, t = 0.0;
  for_values<T, V>(B, j, begin, end, [&](const T (&v)[V], int64_t, int64_t) {
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const double a = (double)widen(v[i]), b = (double)widen(v[i + 1]);
      s = fma(a, a, s);
      t = fma(b, b, t);
    }
  });
  return s + t;
}

template <typename T, typename O, typename Jobs>
__device__ __forceinline__ void scale_to(const ClipBatch<Jobs>& B, int j, int64_t begin, int64_t end, double by) {
  constexpr int V = 16 / sizeof(O);
  O* o = reinterpret_cast<O*>(B.job.out[j]);
  for_values<T, V>(B, j, begin, end, [&](const T (&v)[V], int64_t at, int64_t n) {
    O w[V];
#pragma unroll
    for (int i = 0; i < V; ++i) w[i] = narrow<O>((float)((double)widen(v[i]) * by));
    if (n >= V) {
      store_values<V>(o + at, w);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i < n) o[at + i] = w[i];
    }
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
