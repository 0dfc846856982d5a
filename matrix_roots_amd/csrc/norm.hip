// Root-mean-square norm of rows, with the residual's addition before it and an
// 8-bit output with a scale per 128 columns after it, and its gradient:
//
//   h = x + r (rounded to the stored type), rho = (mean_j h_j^2 + eps)^(-1/2),
//   y_j = h_j rho w_j,  s_b = max(max_{j in b} |y_j|, 2^-100) / F,
//   q_j = y_j / s_b (in float32) rounded to 8 bits (F: the 8-bit type's largest value);
//
//   dx = dres + rho (g - hh mean_j(g_j hh_j)),  g = dy w,  hh = h rho,
//   dw_j = sum over rows of dy_j hh_j.
//
// All sums are float32 (a row's: at most 32 terms per lane, then a tree; a
// column's: one accumulator per lane over the workgroup's rows, the
// workgroups' sums added in a fixed order, so no result depends on timing).
//
// HBM-bound.  Both passes move a row once: it stays in registers between the
// reduction and the output.  16384 x 2048 bf16, one MI355X: forward with
// residual, y and e4m3 62 us (304 MB, 4.9 TB/s, what a large copy reaches),
// gradient 52 us (268 MB, 5.2 TB/s) and 4.6 us for the columns' join; 1 x 1024:
// 3.3 us, a launch.  A row belongs to one wave (up to 2048 columns) or to the
// waves of a workgroup (up to 16384).
#include "mr_common.hpp"
#include "norm_common.hpp"

namespace mr {

template <typename T, int TPR, int CH>
__global__ __launch_bounds__(kNormThreads<TPR>) void norm_forward_kernel(const NormArgs a) {
  __shared__ float red[16];
  constexpr int RPB = kNormThreads<TPR> / TPR, NV = 8;
  int t = RPB == 1 ? (int)threadIdx.x : (int)threadIdx.x % TPR;  // place among the row's threads
  const float inv_width = 1.f / (float)a.width;
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.rows; r0 += (int64_t)gridDim.x * RPB) {
    const int64_t r = RPB == 1 ? r0 : r0 + threadIdx.x / TPR;
    asm volatile("" : "+v"(t));  // columns and addresses are worked out per row, not kept in registers over the loop
    if (TPR == 64 && r >= a.rows) break;  // whole waves: no barrier follows
    const T* x = reinterpret_cast<const T*>(a.x) + r * a.ldx;
    const T* res = a.res ? reinterpret_cast<const T*>(a.res) + r * a.ldres : nullptr;
    float v[CH][NV];
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k) load_chunk<T>(x, chunk_col<TPR>(t, k), a.width, v[k]);
    if (res) {
      T* h = reinterpret_cast<T*>(a.h) + r * a.ldh;
      float u[CH][NV];
#pragma unroll
      for (int k = 0; k < CH; ++k) load_chunk<T>(res, chunk_col<TPR>(t, k), a.width, u[k]);
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        // the stored sum, rounded to T, is what the norm is of: the backward pass reads it
#pragma unroll
        for (int i = 0; i < NV; ++i) v[k][i] = widen(narrow<T>(v[k][i] + u[k][i]));
        store_chunk<T>(h, chunk_col<TPR>(t, k), a.width, v[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < CH; ++k)
#pragma unroll
      for (int i = 0; i < NV; ++i) ss = fmaf(v[k][i], v[k][i], ss);
    ss = row_sum<TPR>(ss, red);
    const float rho = 1.f / sqrtf(ss * inv_width + a.eps);
    if (a.rstd && t == 0) a.rstd[r] = rho;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int c = chunk_col<TPR>(t, k);
      float w[NV];
      load_param<T>(a.w, a.w_f32, c, a.width, w);
#pragma unroll
      for (int i = 0; i < NV; ++i) v[k][i] = v[k][i] * rho * w[i];
      if (a.y) store_chunk<T>(reinterpret_cast<T*>(a.y) + r * a.ldy, c, a.width, v[k]);
      if (a.q) store_eight(a.q + r * a.ldq, a.s + r * a.lds, c, a.width, v[k], a.e5m2);
    }
  }
}

// Rows r0, r0 + gridDim RPB, ...: dx, and this workgroup's column sums of
// dy hh into a.partial[blockIdx.x].
template <typename T, int TPR, int CH>
__global__ __launch_bounds__(kNormThreads<TPR>) void norm_backward_kernel(const NormArgs a) {
  constexpr int RPB = kNormThreads<TPR> / TPR, NV = 8;
  __shared__ float red[16];
  __shared__ float cols[RPB > 1 ? TPR * CH * NV : 1];
  int t = RPB == 1 ? (int)threadIdx.x : (int)threadIdx.x % TPR;  // place among the row's threads
  const float inv_width = 1.f / (float)a.width;
  float dw[CH][NV];
#pragma unroll
  for (int k = 0; k < CH; ++k)
#pragma unroll
    for (int i = 0; i < NV; ++i) dw[k][i] = 0.f;
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.rows; r0 += (int64_t)gridDim.x * RPB) {
    const int64_t r = RPB == 1 ? r0 : r0 + threadIdx.x / TPR;
    asm volatile("" : "+v"(t));  // columns and addresses are worked out per row, not kept in registers over the loop
    if (TPR == 64 && r >= a.rows) break;  // whole waves: the barriers below come after the loop
    const T* dy = reinterpret_cast<const T*>(a.dy) + r * a.lddy;
    const T* h = reinterpret_cast<const T*>(a.x) + r * a.ldx;
    const float rho = a.rstd_in[r];
    float g[CH][NV], hh[CH][NV];
    float dot = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      load_chunk<T>(dy, chunk_col<TPR>(t, k), a.width, g[k]);
      load_chunk<T>(h, chunk_col<TPR>(t, k), a.width, hh[k]);
    }
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      float w[NV];
      load_param<T>(a.w, a.w_f32, chunk_col<TPR>(t, k), a.width, w);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        hh[k][i] *= rho;
        dw[k][i] = fmaf(g[k][i], hh[k][i], dw[k][i]);
        g[k][i] *= w[i];
        dot = fmaf(g[k][i], hh[k][i], dot);
      }
    }
    // under way during the reduction
    const T* res = a.res ? reinterpret_cast<const T*>(a.res) + r * a.ldres : nullptr;
    Raw8<T> rr[CH];
    if (res) {
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        const int col = chunk_col<TPR>(t, k);
        if (col + 8 <= a.width) rr[k] = load8<T>(res + col);
      }
    }
    const float c = row_sum<TPR>(dot, red) * inv_width;
    T* dx = reinterpret_cast<T*>(a.y) + r * a.ldy;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      float u[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) u[i] = 0.f;
      if (res) {
        const int col = chunk_col<TPR>(t, k);
        if (col + 8 <= a.width)
          widen8(rr[k], u);
        else
          load_chunk<T>(res, col, a.width, u);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) u[i] += rho * (g[k][i] - hh[k][i] * c);
      store_chunk<T>(dx, chunk_col<TPR>(t, k), a.width, u);
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
          for (int i = 0; i < NV; ++i) cols[(k * NV + i) * TPR + t] = dw[k][i];
      }
      __syncthreads();
      if ((int)threadIdx.x < TPR) {
#pragma unroll
        for (int k = 0; k < CH; ++k)
#pragma unroll
          for (int i = 0; i < NV; ++i) dw[k][i] += cols[(k * NV + i) * TPR + t];
      }
      __syncthreads();
    }
    if ((int)threadIdx.x >= TPR) return;
  }
#pragma unroll
  for (int k = 0; k < CH; ++k) store_chunk<float>(out, chunk_col<TPR>(t, k), a.width, dw[k]);
}

// dweight[c] = sum over workgroups of their column sums: 32 columns per
// workgroup, 32 groups of lanes over every 32nd partial row (16 rows each of
// 512, all loads in flight at once: 4.6 us for 512 x 2048 sums where one thread
// per column and four waves took 38), joined in a fixed order.
__global__ __launch_bounds__(1024) void norm_weight_grad_kernel(const float* partial, int blocks, int width,
                                                                float* dweight) {
  __shared__ float part[32][33];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), g = threadIdx.x >> 5;
  float s = 0.f;
  if (c < width) {
#pragma unroll 16
    for (int b = g; b < blocks; b += 32) s += partial[(int64_t)b * width + c];
  }
  part[g][threadIdx.x & 31] = s;
  __syncthreads();
  if (g == 0 && c < width) {
    float t = part[0][threadIdx.x];
#pragma unroll
    for (int i = 1; i < 32; ++i) t += part[i][threadIdx.x];
    dweight[c] = t;
  }
}

// ------------------------------------------------------------ launchers
namespace {

constexpr int kNormMaxBlocks = 2048;  // 8 workgroups per CU

template <typename T, int TPR, int CH>
hipError_t go(const NormArgs& a, bool backward, int blocks, hipStream_t s) {
  if (backward)
    hipLaunchKernelGGL((norm_backward_kernel<T, TPR, CH>), dim3(blocks), dim3(kNormThreads<TPR>), 0, s, a);
  else
    hipLaunchKernelGGL((norm_forward_kernel<T, TPR, CH>), dim3(blocks), dim3(kNormThreads<TPR>), 0, s, a);
  return hipGetLastError();
}

template <typename T>
hipError_t pick(const NormArgs& a, bool backward, int blocks, hipStream_t s) {
  const int w = a.width;
  if (w <= 512) return go<T, 64, 1>(a, backward, blocks, s);
  if (w <= 1024) return go<T, 64, 2>(a, backward, blocks, s);
  if (w <= 2048) return go<T, 64, 4>(a, backward, blocks, s);
  if (w <= 4096) return go<T, 256, 2>(a, backward, blocks, s);
  if (w <= 8192) return go<T, 256, 4>(a, backward, blocks, s);
  return go<T, 512, 4>(a, backward, blocks, s);
}

hipError_t pick_type(const NormArgs& a, mr_dtype dt, bool backward, int blocks, hipStream_t s) {
  if (dt == MR_F32) return pick<float>(a, backward, blocks, s);
  if (dt == MR_F16) return pick<_Float16>(a, backward, blocks, s);
  return pick<bf16_t>(a, backward, blocks, s);
}

int64_t row_groups(int64_t rows, int64_t width) { return width <= 2048 ? (rows + 3) / 4 : rows; }

}  // namespace

hipError_t launch_norm_forward(const NormArgs& a, mr_dtype dt, hipStream_t s) {
  const int64_t g = row_groups(a.rows, a.width);
  return pick_type(a, dt, false, (int)(g < kNormMaxBlocks ? g : kNormMaxBlocks), s);
}

int norm_backward_blocks(int64_t rows, int64_t width) {
  const int64_t g = row_groups(rows, width);
  return (int)(g < 512 ? g : 512);
}

hipError_t launch_norm_backward(const NormArgs& a, mr_dtype dt, int blocks, hipStream_t s) {
  return pick_type(a, dt, true, blocks, s);
}

hipError_t launch_norm_weight_grad(const float* partial, int blocks, int width, float* dweight, hipStream_t s) {
  hipLaunchKernelGGL(norm_weight_grad_kernel, dim3((width + 31) / 32), dim3(1024), 0, s, partial, blocks, width, dweight);
  return hipGetLastError();
}

}  // namespace mr
