// Quantisation of a matrix to 8 bits with a float32 scale per block of 128:
//
//   s_b = max(max_{i in b} |x_i|, 2^-100) / F,  q_i = x_i / s_b rounded,
//
// b being 128 consecutive columns of a row (and, for the transposed copy, 128
// consecutive rows of a column) or a square of 128 x 128.  One workgroup per
// 128 x 128 tile reads it once into registers (4 x 8 values per thread) and
// writes it in one or both orders; the transposed bytes pass through LDS so
// that both go out in 128-byte runs.  HBM-bound: nothing is read twice (8192 x 2048
// float32 in both orders: 17 us, 5.9 TB/s; 8191 x 1024 bf16: 12.5 us, 2.7 TB/s,
// where two workgroups per CU leave the latency of one pass through them).
#include "linear_common.hpp"
#include "mr_common.hpp"

namespace mr {

// RT rows x 8 columns per thread, 16 threads across and 128 / RT down.
template <typename T, int RT>
__global__ __launch_bounds__(2048 / RT) void quantize_kernel(const QuantArgs a) {
  constexpr int NW = 32 / RT;
  __shared__ uint32_t colmax[NW][kBlock];
  __shared__ float colinv[kBlock];
  __shared__ __align__(16) unsigned char tile[kBlock][kBlock + 16];
  const int t = threadIdx.x, cg = t & 15, rg = t >> 4, wave = t >> 6;
  const int across = (a.n + kBlock - 1) / kBlock;
  const int bx = blockIdx.x % across;      // block of columns
  const int64_t by = blockIdx.x / across;  // block of rows
  const int c0 = bx * kBlock;
  const int64_t r0 = by * kBlock;
  const int c = c0 + 8 * cg;
  const int64_t r = r0 + RT * rg;
  const T* x = reinterpret_cast<const T*>(a.x);
  float v[RT][8];
#pragma unroll
  for (int p = 0; p < RT; ++p) {
    const T* row = x + (r + p) * a.ldx;
    if (r + p < a.m && c + 8 <= a.n) {
      widen8(load8<T>(row + c), v[p]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[p][i] = r + p < a.m && c + i < a.n ? widen(row[c + i]) : 0.f;
    }
  }

  float square = 0.f;
  if (a.square) {
    uint32_t m = 0;
#pragma unroll
    for (int p = 0; p < RT; ++p)
#pragma unroll
      for (int i = 0; i < 8; ++i) m = umax(m, magnitude(v[p][i]));
    m = max64(m);
    if ((t & 63) == 0) colmax[wave][0] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NW; ++w) m = umax(m, colmax[w][0]);
    square = block_scale(m, a.e5m2);
    if (t == 0) {
      if (a.q) a.s[by * a.lds + bx] = square;
      if (a.qt) a.st[bx * a.ldst + by] = square;
    }
  }

  if (a.q) {
#pragma unroll
    for (int p = 0; p < RT; ++p) {
      float s = square;
      if (!a.square) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = umax(m, magnitude(v[p][i]));
        s = block_scale(max16(m), a.e5m2);
        if (cg == 0 && r + p < a.m) a.s[(r + p) * a.lds + bx] = s;
      }
      const float inv = 1.f / s;
      v2u b;
      b[0] = pack4(v[p][0] * inv, v[p][1] * inv, v[p][2] * inv, v[p][3] * inv, a.e5m2);
      b[1] = pack4(v[p][4] * inv, v[p][5] * inv, v[p][6] * inv, v[p][7] * inv, a.e5m2);
      if (r + p < a.m) {
        unsigned char* q = a.q + (r + p) * a.ldq + c;
        if (c + 8 <= a.n) {
          *reinterpret_cast<v2u_any*>(q) = b;
        } else {
#pragma unroll
          for (int i = 0; i < 7; ++i)
            if (c + i < a.n) q[i] = (unsigned char)(b[i >> 2] >> (8 * (i & 3)));
        }
      }
    }
  }
  if (!a.qt) return;

  if (!a.square) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t m = 0;
#pragma unroll
      for (int p = 0; p < RT; ++p) m = umax(m, magnitude(v[p][i]));
      m = umax(m, (uint32_t)__shfl_xor((int)m, 16));
      m = umax(m, (uint32_t)__shfl_xor((int)m, 32));
      if ((t & 63) < 16) colmax[wave][8 * cg + i] = m;
    }
    __syncthreads();
    if (t < kBlock) {
      uint32_t m = 0;
#pragma unroll
      for (int w = 0; w < NW; ++w) m = umax(m, colmax[w][t]);
      const float s = block_scale(m, a.e5m2);
      colinv[t] = 1.f / s;
      if (c0 + t < a.n) a.st[(int64_t)(c0 + t) * a.ldst + by] = s;
    }
    __syncthreads();
  }
  const float sq_inv = a.square ? 1.f / square : 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float inv = a.square ? sq_inv : colinv[8 * cg + i];
#pragma unroll
    for (int p = 0; p < RT; p += 4)
      *reinterpret_cast<uint32_t*>(&tile[8 * cg + i][RT * rg + p]) =
          pack4(v[p][i] * inv, v[p + 1][i] * inv, v[p + 2][i] * inv, v[p + 3][i] * inv, a.e5m2);
  }
  __syncthreads();
#pragma unroll
  for (int p = 0; p < RT / 2; ++p) {
    const int col = 256 / RT * p + (t >> 3), part = 16 * (t & 7);
    if (c0 + col >= a.n || r0 + part >= a.m) continue;
    unsigned char* q = a.qt + (int64_t)(c0 + col) * a.ldqt + r0 + part;
    if (r0 + part + 16 <= a.m) {
      *reinterpret_cast<v4u_any*>(q) = *reinterpret_cast<const v4u*>(&tile[col][part]);
    } else {
      for (int i = 0; i < 16 && r0 + part + i < a.m; ++i) q[i] = tile[col][part + i];
    }
  }
}

hipError_t launch_quantize(const QuantArgs& a, mr_dtype dt, hipStream_t s) {
  const dim3 grid((unsigned)((a.n + kBlock - 1) / kBlock * ((a.m + kBlock - 1) / kBlock)));
  constexpr int RT = 4;  // 8191 x 1024 bf16 in both orders: 12.5 us, with 8 rows per thread 14.3
  if (dt == MR_F32)
    hipLaunchKernelGGL((quantize_kernel<float, RT>), grid, dim3(2048 / RT), 0, s, a);
  else if (dt == MR_F16)
    hipLaunchKernelGGL((quantize_kernel<_Float16, RT>), grid, dim3(2048 / RT), 0, s, a);
  else
    hipLaunchKernelGGL((quantize_kernel<bf16_t, RT>), grid, dim3(2048 / RT), 0, s, a);
  return hipGetLastError();
}

}  // namespace mr
