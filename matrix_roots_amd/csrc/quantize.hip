// Quantisation of a matrix to 8 bits with a float32 scale per block of 128:
//
//   s_b = max(max_{i in b} |x_i|, 2^-100) / F,  q_i = x_i / s_b (in float32) rounded,
//
// b being 128 consecutive columns of a row (and, for the transposed copy, 128
// consecutive rows of a column) or a square of 128 x 128.  One workgroup per
// 128 x 128 tile reads it once into registers (4 x 8 values per thread) and
// writes it in one or both orders; the transposed bytes pass through LDS so
// that both go out in 128-byte runs.  HBM-bound: nothing is read twice (8192 x 2048
// float32 in both orders: 17.5 us, 5.8 TB/s; 8191 x 1024 bf16: 13.2 us, 2.5 TB/s,
// where two workgroups per CU leave the latency of one pass through them).
#include <type_traits>

#include "linear_common.hpp"
#include "mr_common.hpp"

namespace mr {

// RT rows x 8 columns per thread, 16 threads across and 128 / RT down.  SQUARE
// squares (one scale, so both orders take the same quotients; decided at run
// time, 8192 x 2048 float32 takes 19.4 us for 17.5), else blocks of 128 in a line.
template <typename T, int RT, bool SQUARE>
__global__ __launch_bounds__(2048 / RT) void quantize_kernel(const QuantArgs a) {
  constexpr int NW = 32 / RT;
  __shared__ uint32_t colmax[NW][kBlock];
  __shared__ float colscale[kBlock];
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

  if constexpr (SQUARE) {  // one scale: the quotients of both orders at once
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
    const float square = block_scale(m, a.e5m2);
    if (t == 0) {
      if (a.q) a.s[by * a.lds + bx] = square;
      if (a.qt) a.st[bx * a.ldst + by] = square;
    }
    const Quotient over(square);
#pragma unroll
    for (int p = 0; p < RT; ++p)
#pragma unroll
      for (int i = 0; i < 8; ++i) v[p][i] = over(v[p][i]);
  }

  if (a.q) {
#pragma unroll
    for (int p = 0; p < RT; ++p) {
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = v[p][i];
      if constexpr (!SQUARE) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = umax(m, magnitude(v[p][i]));
        const float s = block_scale(max16(m), a.e5m2);
        if (cg == 0 && r + p < a.m) a.s[(r + p) * a.lds + bx] = s;
        const Quotient over(s);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = over(v[p][i]);
      }
      v2u b;
      b[0] = pack4(y[0], y[1], y[2], y[3], a.e5m2);
      b[1] = pack4(y[4], y[5], y[6], y[7], a.e5m2);
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

  if constexpr (!SQUARE) {
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
      colscale[t] = s;
      if (c0 + t < a.n) a.st[(int64_t)(c0 + t) * a.ldst + by] = s;
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (!SQUARE) {
      const Quotient over(colscale[8 * cg + i]);
#pragma unroll
      for (int p = 0; p < RT; ++p) v[p][i] = over(v[p][i]);
    }
#pragma unroll
    for (int p = 0; p < RT; p += 4)
      *reinterpret_cast<uint32_t*>(&tile[8 * cg + i][RT * rg + p]) =
          pack4(v[p][i], v[p + 1][i], v[p + 2][i], v[p + 3][i], a.e5m2);
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
  constexpr int RT = 4;  // 8191 x 1024 bf16 in both orders: 13.2 us, with 8 rows per thread 15.2
  auto go = [&](auto t, auto square) {
    hipLaunchKernelGGL((quantize_kernel<decltype(t), RT, decltype(square)::value>), grid, dim3(2048 / RT), 0, s, a);
  };
  auto go_type = [&](auto t) { a.square ? go(t, std::true_type{}) : go(t, std::false_type{}); };
  if (dt == MR_F32)
    go_type(float{});
  else if (dt == MR_F16)
    go_type(_Float16{});
  else
    go_type(bf16_t{});
  return hipGetLastError();
}

}  // namespace mr
