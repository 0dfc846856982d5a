// Root-mean-square norm of rows, with the residual's addition before it and an
// 8-bit output with a scale per 128 columns after it, and its gradient:
//
//   h = x + r (rounded to the stored type), rho = (mean_j h_j^2 + eps)^(-1/2),
//   y_j = h_j rho w_j,  s_b = max(max_{j in b} |y_j|, 2^-100) / F,
//   q_j = y_j / s_b rounded to 8 bits (F: the 8-bit type's largest value);
//
//   dx = dres + rho (g - hh mean_j(g_j hh_j)),  g = dy w,  hh = h rho,
//   dw_j = sum over rows of dy_j hh_j.
//
// All sums are float32 (a row's: at most 256 terms per lane, then a tree; a
// column's: one accumulator per lane over the workgroup's rows, the
// workgroups' sums added in a fixed order, so no result depends on timing).
//
// Both passes move a row once: it stays in registers between the reduction
// and the output.  A row belongs to one wave (up to 2048 columns) or to the
// waves of a workgroup (up to 16384).
#include "linear_common.hpp"
#include "mr_common.hpp"

namespace mr {

namespace {

// Where a thread's values lie.  VEC: chunks of 8 consecutive columns, 16
// lanes to a scale block.  Else (odd widths, rows that are not 16-byte
// aligned): pairs of columns 64 apart, one wave to a scale block.
template <int TPR, bool VEC>
struct Place {
  static constexpr int NV = VEC ? 8 : 2;
  int t;  // thread within the row's threads
  __device__ __forceinline__ int col(int chunk) const {
    if (VEC) return 8 * (t + TPR * chunk);
    return kBlock * ((t >> 6) + (TPR / 64) * chunk) + (t & 63);
  }
  static constexpr int STEP = VEC ? 1 : 64;
};

template <typename T, int NV>
struct Chunk {
  float v[NV];
};

template <typename T, int TPR, bool VEC>
__device__ __forceinline__ void load_chunk(const T* row, int c, int width, float (&v)[Place<TPR, VEC>::NV]) {
  if constexpr (VEC) {
    if (c < width) {
      widen8(load8<T>(row + c), v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) v[i] = c + 64 * i < width ? widen(row[c + 64 * i]) : 0.f;
  }
}

template <typename T, int TPR, bool VEC>
__device__ __forceinline__ void store_chunk(T* row, int c, int width, const float (&v)[Place<TPR, VEC>::NV]) {
  if constexpr (VEC) {
    if (c < width) store8<T>(row + c, v);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (c + 64 * i < width) row[c + 64 * i] = narrow<T>(v[i]);
  }
}

template <typename T, int TPR, bool VEC>
__device__ __forceinline__ void load_weight(const NormArgs& a, int c, float (&v)[Place<TPR, VEC>::NV]) {
  if (a.w_f32)
    load_chunk<float, TPR, VEC>(reinterpret_cast<const float*>(a.w), c, a.width, v);
  else
    load_chunk<T, TPR, VEC>(reinterpret_cast<const T*>(a.w), c, a.width, v);
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

}  // namespace

// CH chunks per thread; workgroups of 256 threads (256 / TPR rows at a time) or
// of TPR.
template <int TPR>
constexpr int kNormThreads = TPR < 256 ? 256 : TPR;

template <typename T, int TPR, int CH, bool VEC>
__global__ __launch_bounds__(kNormThreads<TPR>) void norm_forward_kernel(const NormArgs a) {
  __shared__ float red[16];
  constexpr int RPB = kNormThreads<TPR> / TPR, NV = Place<TPR, VEC>::NV;
  Place<TPR, VEC> pl{RPB == 1 ? (int)threadIdx.x : (int)threadIdx.x % TPR};
  const float inv_width = 1.f / (float)a.width;
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.rows; r0 += (int64_t)gridDim.x * RPB) {
    const int64_t r = RPB == 1 ? r0 : r0 + threadIdx.x / TPR;
    asm volatile("" : "+v"(pl.t));  // columns and addresses are worked out per row, not kept in registers over the loop
    if (TPR == 64 && r >= a.rows) break;  // whole waves: no barrier follows
    const T* x = reinterpret_cast<const T*>(a.x) + r * a.ldx;
    const T* res = a.res ? reinterpret_cast<const T*>(a.res) + r * a.ldres : nullptr;
    float v[CH][NV];
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k) load_chunk<T, TPR, VEC>(x, pl.col(k), a.width, v[k]);
    if (res) {
      T* h = reinterpret_cast<T*>(a.h) + r * a.ldh;
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        float u[NV];
        load_chunk<T, TPR, VEC>(res, pl.col(k), a.width, u);
        // the stored sum, rounded to T, is what the norm is of: the backward pass reads it
#pragma unroll
        for (int i = 0; i < NV; ++i) v[k][i] = widen(narrow<T>(v[k][i] + u[i]));
        store_chunk<T, TPR, VEC>(h, pl.col(k), a.width, v[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < CH; ++k)
#pragma unroll
      for (int i = 0; i < NV; ++i) ss = fmaf(v[k][i], v[k][i], ss);
    ss = row_sum<TPR>(ss, red);
    const float rho = 1.f / sqrtf(ss * inv_width + a.eps);
    if (a.rstd && pl.t == 0) a.rstd[r] = rho;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = pl.col(k);
      float w[NV];
      load_weight<T, TPR, VEC>(a, c, w);
      uint32_t amax = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        v[k][i] = v[k][i] * rho * w[i];
        amax = umax(amax, magnitude(v[k][i]));
      }
      if (a.y) store_chunk<T, TPR, VEC>(reinterpret_cast<T*>(a.y) + r * a.ldy, c, a.width, v[k]);
      if (a.q) {
        amax = VEC ? max16(amax) : max64(amax);
        const float s = block_scale(amax, a.e5m2);
        const float inv = 1.f / s;
        const int b = c / kBlock;
        if (c < a.width && (pl.t & (VEC ? 15 : 63)) == 0) a.s[r * a.lds + b] = s;
        unsigned char* q = a.q + r * a.ldq + c;
        if constexpr (VEC) {
          v2u p;
          p[0] = pack4(v[k][0] * inv, v[k][1] * inv, v[k][2] * inv, v[k][3] * inv, a.e5m2);
          p[1] = pack4(v[k][4] * inv, v[k][5] * inv, v[k][6] * inv, v[k][7] * inv, a.e5m2);
          if (c < a.width) *reinterpret_cast<v2u*>(q) = p;
        } else {
          const uint32_t p = pack4(v[k][0] * inv, v[k][1] * inv, 0.f, 0.f, a.e5m2);
          if (c < a.width) q[0] = (unsigned char)p;
          if (c + 64 < a.width) q[64] = (unsigned char)(p >> 8);
        }
      }
    }
  }
}

// Rows r0, r0 + gridDim RPB, ...: dx, and this workgroup's column sums of
// dy hh into a.partial[blockIdx.x].
template <typename T, int TPR, int CH, bool VEC>
__global__ __launch_bounds__(kNormThreads<TPR>) void norm_backward_kernel(const NormArgs a) {
  constexpr int RPB = kNormThreads<TPR> / TPR, NV = Place<TPR, VEC>::NV;
  __shared__ float red[16];
  __shared__ float cols[RPB > 1 ? TPR * CH * NV : 1];
  Place<TPR, VEC> pl{RPB == 1 ? (int)threadIdx.x : (int)threadIdx.x % TPR};
  const float inv_width = 1.f / (float)a.width;
  float dw[CH][NV];
#pragma unroll
  for (int k = 0; k < CH; ++k)
#pragma unroll
    for (int i = 0; i < NV; ++i) dw[k][i] = 0.f;
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.rows; r0 += (int64_t)gridDim.x * RPB) {
    const int64_t r = RPB == 1 ? r0 : r0 + threadIdx.x / TPR;
    asm volatile("" : "+v"(pl.t));  // columns and addresses are worked out per row, not kept in registers over the loop
    if (TPR == 64 && r >= a.rows) break;  // whole waves: the barriers below come after the loop
    const T* dy = reinterpret_cast<const T*>(a.dy) + r * a.lddy;
    const T* h = reinterpret_cast<const T*>(a.x) + r * a.ldx;
    const float rho = a.rstd_in[r];
    float g[CH][NV], hh[CH][NV];
    float dot = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      load_chunk<T, TPR, VEC>(dy, pl.col(k), a.width, g[k]);
      load_chunk<T, TPR, VEC>(h, pl.col(k), a.width, hh[k]);
    }
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      float w[NV];
      load_weight<T, TPR, VEC>(a, pl.col(k), w);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        hh[k][i] *= rho;
        dw[k][i] = fmaf(g[k][i], hh[k][i], dw[k][i]);
        g[k][i] *= w[i];
        dot = fmaf(g[k][i], hh[k][i], dot);
      }
    }
    const float c = row_sum<TPR>(dot, red) * inv_width;
    const T* res = a.res ? reinterpret_cast<const T*>(a.res) + r * a.ldres : nullptr;
    T* dx = reinterpret_cast<T*>(a.y) + r * a.ldy;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      float u[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) u[i] = 0.f;
      if (res) load_chunk<T, TPR, VEC>(res, pl.col(k), a.width, u);
#pragma unroll
      for (int i = 0; i < NV; ++i) u[i] += rho * (g[k][i] - hh[k][i] * c);
      store_chunk<T, TPR, VEC>(dx, pl.col(k), a.width, u);
    }
  }
  if (!a.partial) return;
  float* out = a.partial + (int64_t)blockIdx.x * a.width;
  if constexpr (RPB > 1) {
    for (int w = 1; w < RPB; ++w) {  // waves 1, 2, 3 add to wave 0's sums in turn
      if ((int)threadIdx.x / TPR == w) {
#pragma unroll
        for (int k = 0; k < CH; ++k)
#pragma unroll
          for (int i = 0; i < NV; ++i) cols[(k * NV + i) * TPR + pl.t] = dw[k][i];
      }
      __syncthreads();
      if ((int)threadIdx.x < TPR) {
#pragma unroll
        for (int k = 0; k < CH; ++k)
#pragma unroll
          for (int i = 0; i < NV; ++i) dw[k][i] += cols[(k * NV + i) * TPR + pl.t];
      }
      __syncthreads();
    }
    if ((int)threadIdx.x >= TPR) return;
  }
#pragma unroll
  for (int k = 0; k < CH; ++k)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = pl.col(k) + i * Place<TPR, VEC>::STEP;
      if (c < a.width) out[c] = dw[k][i];
    }
}

// dweight[c] = sum over workgroups of their column sums: 64 columns per
// workgroup, four waves over every fourth partial row.
__global__ __launch_bounds__(256) void norm_weight_grad_kernel(const float* partial, int blocks, int width,
                                                               float* dweight) {
  __shared__ float part[4][64];
  const int c = blockIdx.x * 64 + (threadIdx.x & 63);
  const int w = threadIdx.x >> 6;
  float s = 0.f;
  if (c < width)
    for (int b = w; b < blocks; b += 4) s += partial[(int64_t)b * width + c];
  part[w][threadIdx.x & 63] = s;
  __syncthreads();
  if (w == 0 && c < width)
    dweight[c] = (part[0][threadIdx.x] + part[1][threadIdx.x]) + (part[2][threadIdx.x] + part[3][threadIdx.x]);
}

// ------------------------------------------------------------ launchers
namespace {

constexpr int kNormMaxBlocks = 2048;  // 8 workgroups per CU

template <typename T, int TPR, int CH, bool VEC>
hipError_t go(const NormArgs& a, bool backward, int blocks, hipStream_t s) {
  if (backward)
    hipLaunchKernelGGL((norm_backward_kernel<T, TPR, CH, VEC>), dim3(blocks), dim3(kNormThreads<TPR>), 0, s, a);
  else
    hipLaunchKernelGGL((norm_forward_kernel<T, TPR, CH, VEC>), dim3(blocks), dim3(kNormThreads<TPR>), 0, s, a);
  return hipGetLastError();
}

template <typename T>
hipError_t pick(const NormArgs& a, bool vec, bool backward, int blocks, hipStream_t s) {
  const int w = a.width;
  if (vec) {
    if (w <= 512) return go<T, 64, 1, true>(a, backward, blocks, s);
    if (w <= 1024) return go<T, 64, 2, true>(a, backward, blocks, s);
    if (w <= 2048) return go<T, 64, 4, true>(a, backward, blocks, s);
    if (w <= 4096) return go<T, 256, 2, true>(a, backward, blocks, s);
    if (w <= 8192) return go<T, 256, 4, true>(a, backward, blocks, s);
    return go<T, 512, 4, true>(a, backward, blocks, s);
  }
  if (w <= 512) return go<T, 64, 4, false>(a, backward, blocks, s);
  if (w <= 2048) return go<T, 256, 4, false>(a, backward, blocks, s);
  if (w <= 4096) return go<T, 256, 8, false>(a, backward, blocks, s);
  return go<T, 1024, 8, false>(a, backward, blocks, s);
}

hipError_t pick_type(const NormArgs& a, mr_dtype dt, bool vec, bool backward, int blocks, hipStream_t s) {
  if (dt == MR_F32) return pick<float>(a, vec, backward, blocks, s);
  if (dt == MR_F16) return pick<_Float16>(a, vec, backward, blocks, s);
  return pick<bf16_t>(a, vec, backward, blocks, s);
}

}  // namespace

hipError_t launch_norm_forward(const NormArgs& a, mr_dtype dt, bool vec, hipStream_t s) {
  const int64_t g = a.width <= (vec ? 2048 : 512) ? (a.rows + 3) / 4 : a.rows;
  return pick_type(a, dt, vec, false, (int)(g < kNormMaxBlocks ? g : kNormMaxBlocks), s);
}

int norm_backward_blocks(int64_t rows, int64_t width) {
  const int64_t g = width <= 512 ? (rows + 3) / 4 : rows;
  return (int)(g < 512 ? g : 512);
}

hipError_t launch_norm_backward(const NormArgs& a, mr_dtype dt, bool vec, int blocks, hipStream_t s) {
  return pick_type(a, dt, vec, true, blocks, s);
}

hipError_t launch_norm_weight_grad(const float* partial, int blocks, int width, float* dweight, hipStream_t s) {
  hipLaunchKernelGGL(norm_weight_grad_kernel, dim3((width + 63) / 64), dim3(256), 0, s, partial, blocks, width, dweight);
  return hipGetLastError();
}

}  // namespace mr
