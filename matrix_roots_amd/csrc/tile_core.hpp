// LDS tiles of the linear-layer products: operand chunks of 128 bytes of the
// contraction per row, copied straight from global memory (16 bytes per lane)
// where whole units exist, element by element at the edges.
//
// Two forms of an operand tile with R rows of the product:
//  * along:  the contraction is contiguous in memory.  R LDS rows of 128 bytes
//    (8 units of 16); unit u of row r lies in slot u ^ ((r / 2) % 8), so the 16
//    rows one read cycle touches lie in 16 different bank groups.
//  * across: the product's rows are contiguous in memory (the transposed
//    operand; 16-bit types).  64 LDS rows (steps of the contraction) of 2 R
//    bytes; unit u of row r lies in slot u ^ across_swap(r), so that the four
//    rows a transposing read takes at once lie in different banks.
#pragma once

#include "linear_common.hpp"
#include "mr_common.hpp"

namespace mr {

constexpr int kChunkBytes = 128;

template <int R>
__device__ __forceinline__ int across_swap(int row) {
  constexpr int UPR = R / 8;
  return UPR >= 16 ? 4 * (row & 3) : 2 * (row & 3);
}

// A chunk of an `along` tile by direct copies: rows row0 .. row0 + R - 1 of P
// (row pointers at base + row * ld bytes), the 128 bytes from byte k0.  Rows
// past `valid` re-read the last one: they only feed outputs that are never
// stored.
template <int R, int NW>
__device__ __forceinline__ void copy_along(const unsigned char* base, int64_t ld_bytes, int64_t row0, int valid, int64_t k0,
                                           unsigned char* stage, int wave, int lane) {
  constexpr int N = R * 8 / 64 / NW;
  static_assert(N * 64 * NW == R * 8, "copies cover the chunk");
  const char* p = wave_uniform(base + row0 * ld_bytes + k0);
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int u0 = (j * NW + wave) * 64;
    const int u = u0 + lane, row = u >> 3;
    uint32_t off = (uint32_t)min(row, valid - 1) * (uint32_t)ld_bytes + (uint32_t)(dl_slot(row, u & 7, 8) * 16);
    asm volatile("" : "+v"(off));  // opaque per copy: the offset stays a 32-bit lane value
    __builtin_amdgcn_global_load_lds((global_void_ptr)(p + off), (lds_void_ptr)(stage + u0 * 16), 16, 0, 0);
  }
}

// A chunk of an `across` tile: contraction rows k0 .. k0 + 63, the R columns
// from col0 (16-bit elements), all inside the matrix.
template <int R, int NW>
__device__ __forceinline__ void copy_across(const unsigned char* base, int64_t ld_bytes, int64_t k0, int64_t col0, int valid,
                                            unsigned char* stage, int wave, int lane) {
  constexpr int UPR = R / 8, N = 64 * UPR / 64 / NW;
  static_assert(N * NW == UPR, "copies cover the chunk");
  const char* p = wave_uniform(base + k0 * ld_bytes + col0 * 2);
  const int units = (valid + 7) >> 3;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int u0 = (j * NW + wave) * 64;
    const int u = u0 + lane, row = u / UPR;
    const int unit = (u % UPR) ^ across_swap<R>(row);
    uint32_t off = (uint32_t)row * (uint32_t)ld_bytes + (uint32_t)(min(unit, units - 1) * 16);
    asm volatile("" : "+v"(off));
    __builtin_amdgcn_global_load_lds((global_void_ptr)(p + off), (lds_void_ptr)(stage + u0 * 16), 16, 0, 0);
  }
}

// 16 bytes at p of which the first `n` (elements of ES bytes) exist; zeros after.
template <int ES>
__device__ __forceinline__ v4u edge_unit(const unsigned char* p, int n, bool aligned) {
  v4u r = {0, 0, 0, 0};
  if (n >= 16 / ES && aligned) return *reinterpret_cast<const v4u*>(p);
#pragma unroll
  for (int i = 0; i < 16 / ES; ++i)
    if (i < n) {
      const uint32_t e = ES == 1 ? p[i] : (uint32_t) * reinterpret_cast<const uint16_t*>(p + 2 * i);
      r[i * ES / 4] |= e << (8 * ES * (i & (4 / ES - 1)));
    }
  return r;
}

// The same chunks with every element checked: rows past `valid` and contraction
// steps past k_left are zeros, so that nothing that lies there (not even a NaN)
// reaches the sums.
template <int R, int THREADS, int ES>
__device__ __forceinline__ void edge_along(const unsigned char* base, int64_t ld_bytes, int64_t row0, int valid, int64_t k0,
                                           int k_left, bool aligned, unsigned char* stage) {
  for (int u = threadIdx.x; u < R * 8; u += THREADS) {
    const int row = u >> 3, unit = u & 7;
    v4u v = {0, 0, 0, 0};
    if (row < valid) v = edge_unit<ES>(base + (row0 + row) * ld_bytes + k0 + unit * 16, k_left - unit * (16 / ES), aligned);
    *reinterpret_cast<v4u*>(stage + (row * 8 + dl_slot(row, unit, 8)) * 16) = v;
  }
}
template <int R, int THREADS>
__device__ __forceinline__ void edge_across(const unsigned char* base, int64_t ld_bytes, int64_t k0, int k_left, int64_t col0,
                                            int valid, bool aligned, unsigned char* stage) {
  constexpr int UPR = R / 8;
  for (int u = threadIdx.x; u < 64 * UPR; u += THREADS) {
    const int row = u / UPR, unit = u % UPR;
    v4u v = {0, 0, 0, 0};
    if (row < k_left) v = edge_unit<2>(base + (k0 + row) * ld_bytes + (col0 + unit * 8) * 2, valid - unit * 8, aligned);
    *reinterpret_cast<v4u*>(stage + (row * UPR + (unit ^ across_swap<R>(row))) * 16) = v;
  }
}

// Four consecutive outputs of a row, `left` of them inside the matrix.
template <typename T>
__device__ __forceinline__ void put4(T* p, const float (&v)[4], int left, bool vec, bool accumulate) {
  float x[4] = {v[0], v[1], v[2], v[3]};
  if (accumulate) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < left) x[i] += widen(p[i]);
  }
  if (vec && left >= 4) {
    T t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = narrow<T>(x[i]);
    if constexpr (sizeof(T) == 4) {
      v4u u;
      __builtin_memcpy(&u, t, 16);
      *reinterpret_cast<v4u*>(p) = u;
    } else {
      v2u u;
      __builtin_memcpy(&u, t, 8);
      *reinterpret_cast<v2u*>(p) = u;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < left) p[i] = narrow<T>(x[i]);
}
__device__ __forceinline__ void put4_as(void* c, int64_t at, const float (&v)[4], int left, int type, bool vec,
                                        bool accumulate) {
  if (type == MR_F32)
    put4(reinterpret_cast<float*>(c) + at, v, left, vec, accumulate);
  else if (type == MR_F16)
    put4(reinterpret_cast<_Float16*>(c) + at, v, left, vec, accumulate);
  else
    put4(reinterpret_cast<bf16_t*>(c) + at, v, left, vec, accumulate);
}

// This wave's copies and LDS stores are done, and so are every other wave's.
__device__ __forceinline__ void stage_barrier() {
  wait_vmcnt<0>();
  wait_lgkmcnt0();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

}  // namespace mr
