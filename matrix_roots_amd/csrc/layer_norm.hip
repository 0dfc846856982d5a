// Layer norm of rows, with the residual's addition before it and an 8-bit
// output with a scale per 128 columns after it, and its gradient:
//
//   h = x + r (rounded to the stored type), mu = mean_j h_j,
//   rho = (mean_j (h_j - mu)^2 + eps)^(-1/2),  y_j = (h_j - mu) rho w_j + b_j,
//   and y in 8 bits as the root-mean-square norm's;
//
//   dx = dres + rho (g - mean_j g_j - hh mean_j(g_j hh_j)),  g = dy w,
//   hh = (h - mu) rho,  dw_j = sum over rows of dy_j hh_j,  db_j = of dy_j.
//
// A row stays in registers from its loads to its last output, so the mean is
// known before the squares are added: with m the mean rounded to the rows' type and
// d = h - m, mu = m + mean(d) and the variance is mean(d^2) - mean(d)^2.  mean(d) is
// what m was rounded by; without it a row of equal values far from zero would come
// out as that rounding over sqrt(eps).  Values of 16 bits less a number of their own
// type are exact but for a few; less a float32 m they would all be rounded alike, and
// the mean be off by that (1024 bf16 columns: 2.3e-8 of the deviation, so 5e-9).
// mean(d)^2 is no more than the variance there, as m is the nearest to the mean of the
// numbers that the row can hold.  Sums are float32 in an order that sizes alone
// decide; squares of differences beyond its range leave a rho of 0.
//
// HBM-bound.  16384 x 2048 bf16: forward with residual and y 49 us from a clean cache
// (268 MB, 5.4 TB/s), 58 in passes one after another; gradient with the residual's
// 54 us (278 MB, 5.2 TB/s) and 4.9 for the join of its columns' sums.  A row
// belongs to one wave (up to 2048 columns) or to the waves of a workgroup (up to
// 16384), in as few chunks of eight columns a thread as hold it.
#include "mr_common.hpp"
#include "norm_common.hpp"

namespace mr {

namespace {

// Sums of two values over the row's threads, in each of them; the rows of a workgroup take their turns together.
template <int TPR>
__device__ __forceinline__ void row_sum2(float& u, float& v, float (*red)[16]) {
  u = sum64(u);
  v = sum64(v);
  if constexpr (TPR == 64) return;
  const int wave = threadIdx.x >> 6, first = threadIdx.x / TPR * (TPR / 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[0][wave] = u, red[1][wave] = v;
  __syncthreads();
  u = red[0][first], v = red[1][first];
#pragma unroll
  for (int w = 1; w < TPR / 64; ++w) u += red[0][first + w], v += red[1][first + w];
}

// Threads of the gradient's workgroups: four rows of one wave, two of four waves that
// hold more than two chunks (7710 x 4352 bf16 74 us, one row at a time 82; 969 x 6503
// 26 and 33: half as many sums to join), else one.
template <int TPR, int CH>
constexpr int kBackThreads = TPR == 256 && CH > 2 ? 512 : kNormThreads<TPR>;

// The eight columns a thread holds of a row in chunk k of CH.  Chunks before the
// last are whole (`pick` takes the smallest CH).  In that one the thread at a ragged
// end takes the row's last eight, and threads behind it do too: all loads are
// whole and none depends on a branch.  The columns that a neighbour holds as well,
// the first `skip`, are left out of the row's sums; what is stored for them twice is
// the same.  Rows of less than eight (FEW) are the first thread's.
template <int TPR, int CH, bool FEW>
struct Span {
  int c, skip, width;
  __device__ __forceinline__ Span(int t, int k, int w) : width(w) {
    const int at = chunk_col<TPR>(t, k);
    c = FEW ? 0 : k < CH - 1 || at + 8 <= w ? at : w - 8;
    skip = FEW ? (t == 0 ? 0 : 8) : at - c;
  }
  __device__ __forceinline__ bool mine(int i) const { return i >= skip && (!FEW || i < width); }
  __device__ __forceinline__ bool any() const { return skip < 8; }
  template <typename T>
  __device__ __forceinline__ Raw8<T> load(const T* row) const {
    if constexpr (!FEW) return load8<T>(row + c);
    T v[8] = {};
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < width) v[i] = row[i];
    Raw8<T> r;
    __builtin_memcpy(&r, v, sizeof r);
    return r;
  }
  template <typename T>
  __device__ __forceinline__ void store(T* row, const float (&v)[8]) const {
    if (!any()) return;
    if constexpr (!FEW) {
      store8<T>(row + c, v);
    } else {
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (i < width) row[i] = narrow<T>(v[i]);
    }
  }
  template <typename T>
  __device__ __forceinline__ void param(const void* p, int f32, float (&v)[8]) const {
    if (f32)
      widen8(load<float>(reinterpret_cast<const float*>(p)), v);
    else
      widen8(load<T>(reinterpret_cast<const T*>(p)), v);
  }
  // v in 8 bits with its block's scale; q and s are the row's.  All 64 lanes take part.
  __device__ __forceinline__ void store_eight(unsigned char* q, float* s, const float (&v)[8], bool e5m2) const {
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = mine(i) ? umax(amax, magnitude(v[i])) : amax;
    amax = max16(amax);
    const float sb = block_scale(amax, e5m2);
    const Quotient over(sb);
    if (any() && (threadIdx.x & 15) == 0) s[(c + skip) / kBlock] = sb;
    v2u p;
    p[0] = pack4(over(v[0]), over(v[1]), over(v[2]), over(v[3]), e5m2);
    p[1] = pack4(over(v[4]), over(v[5]), over(v[6]), over(v[7]), e5m2);
    if (!FEW && skip == 0) {
      *reinterpret_cast<v2u_any*>(q + c) = p;
    } else if (any()) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (mine(i)) q[c + i] = (unsigned char)(p[i >> 2] >> (8 * (i & 3)));
    }
  }
};

}  // namespace

template <typename T, int TPR, int CH, bool FEW>
__global__ __launch_bounds__(kNormThreads<TPR>) void layer_norm_forward_kernel(const LayerNormArgs a) {
  __shared__ float red[2][16];
  constexpr int RPB = kNormThreads<TPR> / TPR, NV = 8;
  int t = RPB == 1 ? (int)threadIdx.x : (int)threadIdx.x % TPR;  // place among the row's threads
  const float inv_width = 1.f / (float)a.width;
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.rows; r0 += (int64_t)gridDim.x * RPB) {
    const int64_t r = RPB == 1 ? r0 : r0 + threadIdx.x / TPR;
    asm volatile("" : "+v"(t));  // columns and addresses are worked out per row, not kept in registers over the loop
    if (TPR == 64 && r >= a.rows) break;  // whole waves: no barrier follows
    const T* x = reinterpret_cast<const T*>(a.x) + r * a.ldx;
    const T* res = a.res ? reinterpret_cast<const T*>(a.res) + r * a.ldres : nullptr;
    auto span = [&](int k) { return Span<TPR, CH, FEW>(t, k, a.width); };
    Raw8<T> raw[CH];
    float v[CH][NV];
#pragma unroll
    for (int k = 0; k < CH; ++k) raw[k] = span(k).load(x);
    if (res) {
      T* h = reinterpret_cast<T*>(a.h) + r * a.ldh;
      Raw8<T> add[CH];
#pragma unroll
      for (int k = 0; k < CH; ++k) add[k] = span(k).load(res);
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        float u[NV];
        widen8(raw[k], v[k]);
        widen8(add[k], u);
        // the stored sum, rounded to T, is what the norm is of: the backward pass reads it
#pragma unroll
        for (int i = 0; i < NV; ++i) v[k][i] = widen(narrow<T>(v[k][i] + u[i]));
        span(k).store(h, v[k]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < CH; ++k) widen8(raw[k], v[k]);
    }
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      if (k == CH - 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i) s += span(k).mine(i) ? v[k][i] : 0.f;
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) s += v[k][i];
      }
    }
    float m = widen(narrow<T>(row_sum<TPR>(s, red[0]) * inv_width));
    asm volatile("" : "+v"(m));  // one rounded m for all differences: none takes the product in a fused operation
    float ds = 0.f, ss = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
#pragma unroll
      for (int i = 0; i < NV; ++i) v[k][i] -= m;
      if (k == CH - 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const float d = span(k).mine(i) ? v[k][i] : 0.f;
          ds += d;
          ss = fmaf(d, d, ss);
        }
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          ds += v[k][i];
          ss = fmaf(v[k][i], v[k][i], ss);
        }
      }
    }
    row_sum2<TPR>(ds, ss, red);
    const float e = ds * inv_width;
    const float var = fmaf(-e, e, ss * inv_width);
    const float rho = 1.f / sqrtf((var < 0.f ? 0.f : var) + a.eps);  // NaN stays NaN
    if (t == 0) {
      if (a.mean) a.mean[r] = __builtin_isinf(m) ? m : m + e;  // an infinite m: differences are no numbers
      if (a.rstd) a.rstd[r] = rho;
    }
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      float w[NV], b[NV];
      span(k).template param<T>(a.w, a.w_f32, w);
#pragma unroll
      for (int i = 0; i < NV; ++i) b[i] = 0.f;
      if (a.b) span(k).template param<T>(a.b, a.w_f32, b);
#pragma unroll
      for (int i = 0; i < NV; ++i) v[k][i] = fmaf((v[k][i] - e) * rho, w[i], b[i]);
      if (a.y) span(k).store(reinterpret_cast<T*>(a.y) + r * a.ldy, v[k]);
      if (a.q) span(k).store_eight(a.q + r * a.ldq, a.s + r * a.lds, v[k], a.e5m2);
    }
  }
}

// Rows r0, r0 + gridDim RPB, ...: dx, and this workgroup's column sums of dy hh
// and of dy into a.partial[2 blockIdx.x] and the row behind it.  Rows stay as they
// are stored until they are used, which leaves registers for the next row's loads.
template <typename T, int TPR, int CH, bool FEW>
__global__ __launch_bounds__((kBackThreads<TPR, CH>)) void layer_norm_backward_kernel(const LayerNormArgs a) {
  constexpr int RPB = kBackThreads<TPR, CH> / TPR, NV = 8;
  __shared__ float red[2][16];
  __shared__ float cols[RPB > 1 ? TPR * CH * NV : 1];
  int t = RPB == 1 ? (int)threadIdx.x : (int)threadIdx.x % TPR;  // place among the row's threads
  const float inv_width = 1.f / (float)a.width;
  float dw[CH][NV], db[CH][NV];
#pragma unroll
  for (int k = 0; k < CH; ++k)
#pragma unroll
    for (int i = 0; i < NV; ++i) dw[k][i] = db[k][i] = 0.f;
  Raw8<T> dy[CH], h[CH];
  float rho = 0.f, mu = 0.f;
  const int64_t step = (int64_t)gridDim.x * RPB;
  // the next row's loads are under way while one is worked on, but for float32 in four chunks of 512 threads, which take
  // all registers
  constexpr bool kAhead = sizeof(T) == 2 || TPR == 64 || CH < 4;
  auto span = [&](int k) { return Span<TPR, CH, FEW>(t, k, a.width); };
  auto load = [&](int64_t r) {
    const T* from_dy = reinterpret_cast<const T*>(a.dy) + r * a.lddy;
    const T* from_h = reinterpret_cast<const T*>(a.x) + r * a.ldx;
    rho = a.rstd_in[r], mu = a.mean_in[r];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      dy[k] = span(k).load(from_dy);
      h[k] = span(k).load(from_h);
    }
  };
  int64_t r = (int64_t)blockIdx.x * RPB + (RPB == 1 ? 0 : threadIdx.x / TPR);
  auto ahead = [&](int64_t r) {
    if (r < a.rows) {
      load(r);
    } else {  // no row: nothing to the sums
      rho = mu = 0.f;
#pragma unroll
      for (int k = 0; k < CH; ++k) dy[k] = h[k] = Raw8<T>{};
    }
  };
  ahead(r);
  for (int64_t r0 = (int64_t)blockIdx.x * RPB; r0 < a.rows; r0 += step, r += step) {
    const bool on = r < a.rows;
    if (TPR == 64 && !on) break;  // whole waves; the barriers below come after the loop
    asm volatile("" : "+v"(t));  // columns and addresses are worked out per row, not kept in registers over the loop
    float sg = 0.f, dot = 0.f;
    Raw8<T> now_dy[CH], now_h[CH], rr[CH];
    const float now_rho = rho, now_mu = mu;
    const T* res = a.res ? reinterpret_cast<const T*>(a.res) + r * a.ldres : nullptr;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      now_dy[k] = dy[k], now_h[k] = h[k];
      if (res && on) rr[k] = span(k).load(res);
    }
    if (kAhead) ahead(r + step);
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      float w[NV], g[NV], hh[NV];
      span(k).template param<T>(a.w, a.w_f32, w);
      widen8(now_dy[k], g);
      widen8(now_h[k], hh);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        hh[i] = (hh[i] - now_mu) * now_rho;
        dw[k][i] = fmaf(g[i], hh[i], dw[k][i]);
        db[k][i] += g[i];
        g[i] *= w[i];
      }
      if (k == CH - 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const bool in = span(k).mine(i);
          sg += in ? g[i] : 0.f;
          dot += in ? g[i] * hh[i] : 0.f;
        }
      } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          sg += g[i];
          dot = fmaf(g[i], hh[i], dot);
        }
      }
    }
    row_sum2<TPR>(sg, dot, red);
    const float c0 = sg * inv_width, c1 = dot * inv_width;
    T* dx = reinterpret_cast<T*>(a.y) + r * a.ldy;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      float w[NV], g[NV], hh[NV], u[NV];
      span(k).template param<T>(a.w, a.w_f32, w);
      widen8(now_dy[k], g);
      widen8(now_h[k], hh);
#pragma unroll
      for (int i = 0; i < NV; ++i) u[i] = 0.f;
      if (res) widen8(rr[k], u);
#pragma unroll
      for (int i = 0; i < NV; ++i) u[i] += now_rho * (g[i] * w[i] - c0 - (hh[i] - now_mu) * now_rho * c1);
      if (on) span(k).store(dx, u);
    }
    if (!kAhead) ahead(r + step);
  }
  if (!a.partial) return;
  float* out = a.partial + 2 * (int64_t)blockIdx.x * a.width;
  if constexpr (RPB > 1) {
    auto join = [&](float (&s)[CH][NV], int w) {  // the wth rows' threads add to the first's
      __syncthreads();
      if ((int)threadIdx.x / TPR == w) {
#pragma unroll
        for (int k = 0; k < CH; ++k)
#pragma unroll
          for (int i = 0; i < NV; ++i) cols[(k * NV + i) * TPR + t] = s[k][i];
      }
      __syncthreads();
      if ((int)threadIdx.x < TPR) {
#pragma unroll
        for (int k = 0; k < CH; ++k)
#pragma unroll
          for (int i = 0; i < NV; ++i) s[k][i] += cols[(k * NV + i) * TPR + t];
      }
    };
    for (int w = 1; w < RPB; ++w) {
      join(dw, w);
      join(db, w);
    }
    if ((int)threadIdx.x >= TPR) return;
  }
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    span(k).store(out, dw[k]);
    span(k).store(out + a.width, db[k]);
  }
}

// dweight and dbias from the workgroups' sums: 32 of the 2 width columns per
// workgroup, 8 lanes of four columns and 128 groups of lanes over every 128th
// row, joined in a fixed order.
__global__ __launch_bounds__(1024) void layer_norm_join_kernel(const float* partial, int blocks, int width,
                                                               float* dweight, float* dbias) {
  __shared__ float part[128][33];
  const int l = threadIdx.x & 7, g = threadIdx.x >> 3;
  const int c = blockIdx.x * 32 + 4 * l, n = 2 * width;
  f4 s = {0.f, 0.f, 0.f, 0.f};
  if (c + 4 <= n) {
#pragma unroll 4
    for (int b = g; b < blocks; b += 128) {
      const v4u u = *reinterpret_cast<const v4u_any*>(partial + (int64_t)b * n + c);
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] += __uint_as_float(u[i]);
    }
  } else {
    for (int b = g; b < blocks; b += 128)
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (c + i < n) s[i] += partial[(int64_t)b * n + c + i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) part[g][4 * l + i] = s[i];
  __syncthreads();
  const int col = threadIdx.x & 31, h = threadIdx.x >> 5;  // 32 groups of four
  float t = (part[4 * h][col] + part[4 * h + 1][col]) + (part[4 * h + 2][col] + part[4 * h + 3][col]);
  __syncthreads();
  part[h][col] = t;
  __syncthreads();
  const int out = blockIdx.x * 32 + col;
  if (h == 0 && out < n) {
    t = part[0][col];
#pragma unroll
    for (int i = 1; i < 32; ++i) t += part[i][col];
    if (out < width) {
      if (dweight) dweight[out] = t;
    } else if (dbias) {
      dbias[out - width] = t;
    }
  }
}

// ------------------------------------------------------------ launchers
namespace {

constexpr int kMaxBlocks = 2048;  // 8 workgroups per CU

template <typename T, int TPR, int CH, bool FEW = false>
hipError_t go(const LayerNormArgs& a, bool backward, int blocks, hipStream_t s) {
  if (backward)
    hipLaunchKernelGGL((layer_norm_backward_kernel<T, TPR, CH, FEW>), dim3(blocks), dim3(kBackThreads<TPR, CH>), 0, s, a);
  else
    hipLaunchKernelGGL((layer_norm_forward_kernel<T, TPR, CH, FEW>), dim3(blocks), dim3(kNormThreads<TPR>), 0, s, a);
  return hipGetLastError();
}

template <typename T>
hipError_t pick(const LayerNormArgs& a, bool backward, int blocks, hipStream_t s) {
  const int w = a.width;
  if (w < 8) return go<T, 64, 1, true>(a, backward, blocks, s);
  if (w <= 512) return go<T, 64, 1>(a, backward, blocks, s);
  if (w <= 1024) return go<T, 64, 2>(a, backward, blocks, s);
  if (w <= 1536) return go<T, 64, 3>(a, backward, blocks, s);
  if (w <= 2048) return go<T, 64, 4>(a, backward, blocks, s);
  if (w <= 4096) return go<T, 256, 2>(a, backward, blocks, s);
  if (w <= 6144) return go<T, 256, 3>(a, backward, blocks, s);
  if (w <= 8192) return go<T, 256, 4>(a, backward, blocks, s);
  if (w <= 12288) return go<T, 512, 3>(a, backward, blocks, s);
  return go<T, 512, 4>(a, backward, blocks, s);
}

hipError_t pick_type(const LayerNormArgs& a, mr_dtype dt, bool backward, int blocks, hipStream_t s) {
  if (dt == MR_F32) return pick<float>(a, backward, blocks, s);
  if (dt == MR_F16) return pick<_Float16>(a, backward, blocks, s);
  return pick<bf16_t>(a, backward, blocks, s);
}

int64_t row_groups(int64_t rows, int64_t width) { return width <= 2048 ? (rows + 3) / 4 : rows; }

}  // namespace

hipError_t launch_layer_norm_forward(const LayerNormArgs& a, mr_dtype dt, hipStream_t s) {
  const int64_t g = row_groups(a.rows, a.width);
  return pick_type(a, dt, false, (int)(g < kMaxBlocks ? g : kMaxBlocks), s);
}

// As many workgroups as registers let the CUs hold, where each gets four rounds of
// rows, and the least of those at least (each leaves two rows of sums to be joined).
// One chunk of eight columns in a thread: five to a CU (16384 x 512 bf16 with three
// streams: 23 us, with 512 workgroups 29); two: three (8000 x 4096: 65 us, with 512 71,
// with 1024 78; 4801 x 2944: 38, 43, 46; rows of one wave, 16384 x 1024: 34, with 512
// 37, with 1280 41; 16384 x 768: 30, 33, 37; float32 alone does better with 512, 51
// against 53 at 16384 x 1024); more: two, or one of twice the threads.
int layer_norm_backward_blocks(int64_t rows, int64_t width) {
  const bool two = width > 4096 && width <= 8192;  // rows at a time of 512 threads
  const int64_t g = two ? (rows + 1) / 2 : row_groups(rows, width);
  const int64_t held = width <= 512 ? 1280 : width <= 1024 || (width > 2048 && width <= 4096) ? 768 : two ? 256 : 512;
  const int64_t least = two ? 256 : 512;
  const int64_t most = g / 4 < least ? least : g / 4 < held ? g / 4 : held;
  return (int)(g < most ? g : most);
}

hipError_t launch_layer_norm_backward(const LayerNormArgs& a, mr_dtype dt, int blocks, hipStream_t s) {
  return pick_type(a, dt, true, blocks, s);
}

hipError_t launch_layer_norm_join(const float* partial, int blocks, int width, float* dweight, float* dbias, hipStream_t s) {
  hipLaunchKernelGGL(layer_norm_join_kernel, dim3((2 * width + 31) / 32), dim3(1024), 0, s, partial, blocks, width, dweight, dbias);
  return hipGetLastError();
}

}  // namespace mr
