// LDS tiles of the linear-layer products: operand chunks of 64 or 128 bytes of
// the contraction per row, copied straight from global memory (16 bytes per lane)
// where whole units exist, element by element at the edges.
//
// Two forms of an operand tile with R rows of the product:
//  * along:  the contraction is contiguous in memory.  R LDS rows of UPR units of
//    16 bytes; unit u of row r lies in slot dl_slot(r, u, UPR), so the 16 rows
//    one read cycle touches lie in 16 different bank groups.
//  * across: the product's rows are contiguous in memory (the transposed
//    operand; 16-bit types).  LDS rows are steps of the contraction, of 2 R
//    bytes; unit u of row r lies in slot u ^ across_swap(r), so that the four
//    rows a transposing read takes at once lie in different banks.
#pragma once

#include <atomic>

#include "linear_common.hpp"
#include "mr_common.hpp"

namespace mr {

constexpr int kChunkBytes = 128;

template <int R>
__device__ __forceinline__ int across_swap(int row) {
  constexpr int UPR = R / 8;
  return UPR >= 16 ? 4 * (row & 3) : 2 * (row & 3);
}

// A chunk of an `along` tile by direct copies of NW waves: rows row0 .. row0 + R
// - 1 of P (row pointers at base + row * ld bytes), the 16 UPR bytes from byte
// k0.  Rows past `valid` re-read the last one: they only feed outputs that are
// never stored.  Units past the first `units` re-read the last one: the reader
// masks those steps.
template <int R, int NW, int UPR>
constexpr int along_copies = R * UPR / 64 / NW;  // per wave
// Copy j of a wave; p: the chunk's first byte of the tile's first row.
template <int R, int NW, int UPR>
__device__ __forceinline__ void copy_along_one(const char* p, int64_t ld_bytes, int valid, int units, unsigned char* stage,
                                               int wave, int lane, int j) {
  static_assert(along_copies<R, NW, UPR> * 64 * NW == R * UPR, "copies cover the chunk");
  const int u0 = (j * NW + wave) * 64;
  const int u = u0 + lane, row = u / UPR;
  uint32_t off = (uint32_t)min(row, valid - 1) * (uint32_t)ld_bytes +
                 (uint32_t)(min(dl_slot(row, u % UPR, UPR), units - 1) * 16);
  asm volatile("" : "+v"(off));  // opaque per copy: the offset stays a 32-bit lane value
  __builtin_amdgcn_global_load_lds((global_void_ptr)(p + off), (lds_void_ptr)(stage + u0 * 16), 16, 0, 0);
}
template <int R, int NW, int UPR>
__device__ __forceinline__ void copy_along(const unsigned char* base, int64_t ld_bytes, int64_t row0, int valid, int64_t k0,
                                           int units, unsigned char* stage, int wave, int lane) {
  const char* p = wave_uniform(base + row0 * ld_bytes + k0);
#pragma unroll
  for (int j = 0; j < along_copies<R, NW, UPR>; ++j)
    copy_along_one<R, NW, UPR>(p, ld_bytes, valid, units, stage, wave, lane, j);
}

// A chunk of an `across` tile: contraction rows k0 .. k0 + BK - 1, the R columns
// from col0 (16-bit elements); steps past `left` re-read the last one, columns
// past `valid` (a multiple of 8 there) the last unit.
template <int R, int NW, int BK>
__device__ __forceinline__ void copy_across(const unsigned char* base, int64_t ld_bytes, int64_t k0, int left, int64_t col0,
                                            int valid, unsigned char* stage, int wave, int lane) {
  constexpr int UPR = R / 8, N = BK * UPR / 64 / NW;
  static_assert(N * NW * 64 == BK * UPR, "copies cover the chunk");
  const char* p = wave_uniform(base + k0 * ld_bytes + col0 * 2);
  const int units = (valid + 7) >> 3;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int u0 = (j * NW + wave) * 64;
    const int u = u0 + lane, row = u / UPR;
    const int unit = (u % UPR) ^ across_swap<R>(row);
    uint32_t off = (uint32_t)min(row, left - 1) * (uint32_t)ld_bytes + (uint32_t)(min(unit, units - 1) * 16);
    asm volatile("" : "+v"(off));
    __builtin_amdgcn_global_load_lds((global_void_ptr)(p + off), (lds_void_ptr)(stage + u0 * 16), 16, 0, 0);
  }
}

// 16 bytes at p (any address) of which the first `n` (elements of ES bytes)
// exist; zeros after.
template <int ES>
__device__ __forceinline__ v4u edge_unit(const unsigned char* p, int n) {
  v4u r = {0, 0, 0, 0};
  if (n >= 16 / ES) return *reinterpret_cast<const v4u_any*>(p);
#pragma unroll
  for (int i = 0; i < 16 / ES; ++i)
    if (i < n) {
      const uint32_t e = ES == 1 ? p[i] : (uint32_t) * reinterpret_cast<const uint16_t*>(p + 2 * i);
      r[i * ES / 4] |= e << (8 * ES * (i & (4 / ES - 1)));
    }
  return r;
}

// The same chunks by THREADS threads through registers, for rows at any address
// and ragged ends, in two halves (the loads of one chunk can run ahead of its
// stores): rows past `valid` and contraction steps past k_left become zeros, so
// that nothing that lies there (not even a NaN) reaches the sums.
template <int R, int THREADS, int ES, int UPR>
struct EdgeAlong {
  static constexpr int N = (R * UPR + THREADS - 1) / THREADS, EU = 16 / ES;
  v4u v[N];
  __device__ __forceinline__ void load(const unsigned char* base, int64_t ld_bytes, int64_t row0, int valid, int64_t k0,
                                       int k_left, int thread) {
    const unsigned char* p = base + row0 * ld_bytes + k0;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int u = thread + j * THREADS, row = u / UPR, unit = u % UPR;
      v[j] = {0, 0, 0, 0};
      if (u < R * UPR && row < valid && unit * EU + EU <= k_left)
        v[j] = *reinterpret_cast<const v4u_any*>(p + row * ld_bytes + unit * 16);
    }
    if (k_left >= UPR * EU || k_left % EU == 0) return;
#pragma unroll
    for (int j = 0; j < N; ++j) {  // the unit that the contraction ends in, element by element
      const int u = thread + j * THREADS, row = u / UPR, unit = u % UPR;
      if (u < R * UPR && row < valid && unit == k_left / EU) v[j] = edge_unit<ES>(p + row * ld_bytes + unit * 16, k_left % EU);
    }
  }
  __device__ __forceinline__ void store(unsigned char* stage, int thread) const {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int u = thread + j * THREADS, row = u / UPR, unit = u % UPR;
      if (u < R * UPR) *reinterpret_cast<v4u*>(stage + (row * UPR + dl_slot(row, unit, UPR)) * 16) = v[j];
    }
  }
};
template <int R, int THREADS, int BK>
struct EdgeAcross {
  static constexpr int UPR = R / 8, N = (BK * UPR + THREADS - 1) / THREADS;
  v4u v[N];
  __device__ __forceinline__ void load(const unsigned char* base, int64_t ld_bytes, int64_t k0, int k_left, int64_t col0,
                                       int valid, int thread) {
    const unsigned char* p = base + k0 * ld_bytes + col0 * 2;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int u = thread + j * THREADS, row = u / UPR, unit = u % UPR;
      v[j] = {0, 0, 0, 0};
      if (u < BK * UPR && row < k_left && unit * 8 + 8 <= valid)
        v[j] = *reinterpret_cast<const v4u_any*>(p + row * ld_bytes + unit * 16);
    }
    if (valid >= R || valid % 8 == 0) return;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int u = thread + j * THREADS, row = u / UPR, unit = u % UPR;
      if (u < BK * UPR && row < k_left && unit == valid / 8) v[j] = edge_unit<2>(p + row * ld_bytes + unit * 16, valid % 8);
    }
  }
  __device__ __forceinline__ void store(unsigned char* stage, int thread) const {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int u = thread + j * THREADS, row = u / UPR, unit = u % UPR;
      if (u < BK * UPR) *reinterpret_cast<v4u*>(stage + (row * UPR + (unit ^ across_swap<R>(row))) * 16) = v[j];
    }
  }
};

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

// ROWS rows of outputs of one wave through LDS, so that they leave in 16-byte
// units: 128 bytes of O to a row, unit u of row r in slot u ^ (r % 8).  The
// wave's LDS instructions run in order, so only the compiler has to keep them so.
template <typename O, int ROWS>
struct Slab {
  static constexpr int COLS = 128 / (int)sizeof(O), BYTES = ROWS * 128, EU = 16 / (int)sizeof(O);
  static __device__ __forceinline__ void put4(unsigned char* slab, int row, int col, const float (&v)[4]) {
    O t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = narrow<O>(v[i]);
    unsigned char* p = slab + row * 128 + ((col / EU) ^ (row & 7)) * 16 + col % EU * (int)sizeof(O);
    if constexpr (sizeof(O) == 4) {
      v4u u;
      __builtin_memcpy(&u, t, 16);
      *reinterpret_cast<v4u*>(p) = u;
    } else {
      v2u u;
      __builtin_memcpy(&u, t, 8);
      *reinterpret_cast<v2u*>(p) = u;
    }
  }
  static __device__ __forceinline__ void fence() {
    wait_lgkmcnt0();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
  }
  // rows_left x cols_left of the slab exist in c.  A 16-bit c that is added to takes a
  // float32 slab, so that the sum is rounded once.
  template <typename C>
  static __device__ __forceinline__ void store(const unsigned char* slab, C* c, int64_t ldc, int rows_left, int cols_left,
                                               bool vec, bool accumulate, int lane) {
#pragma unroll
    for (int j = 0; j < ROWS / 8; ++j) {
      const int row = 8 * j + (lane >> 3), unit = lane & 7, col = unit * EU;
      if (row >= rows_left || col >= cols_left) continue;
      const v4u x = *reinterpret_cast<const v4u*>(slab + row * 128 + (unit ^ (row & 7)) * 16);
      C* p = c + row * ldc + col;
      O t[EU];
      __builtin_memcpy(t, &x, 16);
      if constexpr (sizeof(O) != sizeof(C)) {
        mr::put4(p, t, cols_left - col, vec, accumulate);
        continue;
      }
      if (vec && !accumulate && col + EU <= cols_left) {
        *reinterpret_cast<v4u*>(p) = x;
        continue;
      }
#pragma unroll
      for (int i = 0; i < EU; ++i)
        if (col + i < cols_left) p[i] = narrow<C>(accumulate ? widen(t[i]) + widen(p[i]) : widen(t[i]));
    }
  }
};

// This wave's copies and LDS operations are done, and so are every other wave's.
__device__ __forceinline__ void stage_barrier() {
  wait_vmcnt<0>();
  wait_lgkmcnt0();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// Tiles of a persistent workgroup: tile k of slot b / 8 on XCD b % 8, where
// every XCD owns one run of `total` / 8 tiles and walks it in order, so that
// the tiles in flight on an XCD are neighbours and share operands in its L2.
struct Walk {
  int at, step, end;
  // tiles begin .. end of this XCD
  __device__ __forceinline__ Walk(int begin, int end_)
      : at(begin + blockIdx.x / kNumXcd), step(gridDim.x / kNumXcd), end(end_) {}
  __device__ __forceinline__ explicit Walk(int total)
      : Walk((int)((int64_t)total * (blockIdx.x % kNumXcd) / kNumXcd),
             (int)((int64_t)total * (blockIdx.x % kNumXcd + 1) / kNumXcd)) {}
};
// Workgroups of a launch over at most `tiles` tiles: what the CUs hold at a
// time, a multiple of the XCDs.
inline unsigned persistent_blocks(int64_t tiles, int per_cu) {
  const int64_t most = 256 * per_cu;
  return (unsigned)(tiles < most ? (tiles + kNumXcd - 1) / kNumXcd * kNumXcd : most);
}

// Once per kernel and device: dynamic LDS beyond 64 KiB.  `done` holds a bit per
// device.
template <class K>
inline hipError_t raise_lds(K kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (done.load(std::memory_order_relaxed) & bit) return hipSuccess;
  e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Wave roles of a streamed kernel: the last kLoaders waves of a workgroup copy
// operands to LDS, the others multiply and store.
constexpr int kLoaders = 4;

// The loader waves' side of a stream of chunks through NST stages: issue(j) puts
// the stream's chunk j into stage j % NST, false past the end.  With DIRECT by
// COPIES direct copies a wave, else by LDS stores.  One barrier per chunk:
// before it the loaders wait for that chunk alone, after it the stage of its
// predecessor is free.
template <int NST, bool DIRECT, int COPIES, class Issue>
__device__ __forceinline__ void copy_chunks(Issue&& issue) {
  static_assert((NST - 2) * COPIES < 64, "the wait counts to 63");
  int issued = 0;
  auto next = [&] {
    const bool r = issue(issued);
    issued += r;
    return r;
  };
  for (int i = 0; i < NST - 1; ++i) next();
  for (int j = 0;; ++j) {
    if constexpr (DIRECT) {
      // chunk j has landed once at most the copies of the NST - 2 after it are in flight
      if (issued - 1 - j == NST - 2)
        wait_vmcnt<(NST - 2) * COPIES>();
      else
        wait_vmcnt<0>();
    }
    wait_lgkmcnt0();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();  // chunk j is in LDS; every wave is done with chunk j - 1
    asm volatile("" ::: "memory");
    if (!next() && j == issued) return;
  }
}
// The other waves' barrier of a chunk.
__device__ __forceinline__ void join_chunk() {
  wait_lgkmcnt0();
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

}  // namespace mr
