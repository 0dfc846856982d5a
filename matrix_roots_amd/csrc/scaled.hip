// Products of 8-bit matrices with a float32 scale per block of 128 of the
// contraction:
//
//   C_ij = sum_b sa_ib sb_jb sum_{l in b} A_il B_jl.
//
// Every inner sum of 128 is one v_mfma_f32_16x16x128_f8f6f4 (hardware scales at
// 1); its result is scaled and added to a float32 accumulator by the vector
// units.  That instruction adds the products of eight steps on a common
// exponent and keeps 17 bits below the largest (measured: next to 2^16 the
// smallest product that counts is 2^0 among its eight, 2^-7 among the others),
// an error of about 1e-5 of the result: far below the last place of a 16-bit C,
// but over 100 of float32.  For a float32 C the operands are therefore widened
// to fp16 in registers (exactly: both 8-bit types are subsets) and the sums run
// on v_mfma_f32_16x16x32_f16, which adds in float32, at half the rate.  B is the instruction's row operand
// ("P"), A its column operand ("Q"): a lane then holds one row of C, so A's
// scale is one value per lane and column block, B's (one per 128 rows in the
// square form) one per wave, and their product costs one multiplication per
// column block beside one FMA per output.  The instruction's order of the 128
// steps within a lane does not matter, since both operands use the same one.
#include "tile_core.hpp"

namespace mr {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef int v4i __attribute__((ext_vector_type(4)));

// D(16 x 16) = P(16 x 128) Q(16 x 128)^T; lane l: row l % 16 of either, D
// value v is D[4 (l / 16) + v][l % 16].  Operand formats: 0 e4m3, 1 e5m2.
template <int QF>
__device__ __forceinline__ v4f mfma8(v8i p, v8i q) {
  const v4f zero = {0.f, 0.f, 0.f, 0.f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(p, q, zero, 0, QF, 0, 0x7f7f7f7f, 0, 0x7f7f7f7f);
}

// The same 32 bytes per lane as fp16, and the sum of 128 steps as four of 32.
struct Wide {
  v8h h[4];
};
template <int F>
__device__ __forceinline__ Wide widen32(v8i x) {
  typedef _Float16 h2 __attribute__((ext_vector_type(2)));
  Wide w;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    h2 lo, hi;
    if constexpr (F == 0) {
      lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x[i], 1.f, false);
      hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(x[i], 1.f, true);
    } else {  // e5m2 is the upper byte of fp16
      lo = __builtin_bit_cast(h2, __builtin_amdgcn_perm(0u, (uint32_t)x[i], 0x010c000cu));
      hi = __builtin_bit_cast(h2, __builtin_amdgcn_perm(0u, (uint32_t)x[i], 0x030c020cu));
    }
    const int at = 4 * (i & 1);
    w.h[i >> 1][at] = lo[0];
    w.h[i >> 1][at + 1] = lo[1];
    w.h[i >> 1][at + 2] = hi[0];
    w.h[i >> 1][at + 3] = hi[1];
  }
  return w;
}
__device__ __forceinline__ v4f mfma_wide(const Wide& p, const Wide& q) {
  v4f d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) d = __builtin_amdgcn_mfma_f32_16x16x32_f16(p.h[i], q.h[i], d, 0, 0, 0);
  return d;
}
// Fragments of either kind.
template <bool WIDE, int F>
struct Frag8 {
  typedef v8i type;
  static __device__ __forceinline__ v8i of(v8i x) { return x; }
};
template <int F>
struct Frag8<true, F> {
  typedef Wide type;
  static __device__ __forceinline__ Wide of(v8i x) { return widen32<F>(x); }
};
template <int QF>
__device__ __forceinline__ v4f product(v8i p, v8i q) {
  return mfma8<QF>(p, q);
}
template <int QF>
__device__ __forceinline__ v4f product(const Wide& p, const Wide& q) {
  return mfma_wide(p, q);
}

__device__ __forceinline__ v8i join(v4i a, v4i b) {
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Fragment of rows row .. row + 15 of an LDS chunk: bytes 16 g and 64 + 16 g, g = lane / 16.
__device__ __forceinline__ v8i frag8(const unsigned char* st, int row, int lane) {
  const int r = row + (lane & 15), g = lane >> 4;
  const v4i a = *reinterpret_cast<const v4i*>(st + (r * 8 + dl_slot(r, g, 8)) * 16);
  const v4i b = *reinterpret_cast<const v4i*>(st + (r * 8 + dl_slot(r, g + 4, 8)) * 16);
  return join(a, b);
}

}  // namespace

template <int BP_, int BQ_, int WP_, int WQ_>
struct ScaledShape {
  static constexpr int BP = BP_, BQ = BQ_, WP = WP_, WQ = WQ_, NW = WP * WQ, THREADS = 64 * NW;
  static constexpr int RB = BP / WP / 16, CB = BQ / WQ / 16;
  static constexpr int P_BYTES = BP * kChunkBytes, Q_BYTES = BQ * kChunkBytes;
  static constexpr int STAGE = P_BYTES + Q_BYTES + BP * 4;  // P, Q, P's scales (vector form)
  static constexpr int LDS = 2 * STAGE;
};

template <class S, int QF, bool PVEC, bool WIDE>
__global__ __launch_bounds__(S::THREADS) void scaled_tile_kernel(const ScaledArgs a) {
  extern __shared__ __align__(256) unsigned char lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wp = wave / S::WQ, wq = wave % S::WQ;
  const int tp = (a.n + S::BP - 1) / S::BP;
  const int tq = (int)((a.m + S::BQ - 1) / S::BQ);
  int ti, tj;
  full_tile_grouped((int)xcd_remap(blockIdx.x, gridDim.x), tq, tp, ti, tj);
  const int64_t q0 = (int64_t)ti * S::BQ;
  const int p0 = tj * S::BP;
  const int pv = min(S::BP, a.n - p0), qv = (int)min((int64_t)S::BQ, a.m - q0);
  const int chunks = (a.k + kChunkBytes - 1) / kChunkBytes;
  const int c_begin = (int)((int64_t)chunks * blockIdx.y / a.splits);
  const int c_end = (int)((int64_t)chunks * (blockIdx.y + 1) / a.splits);

  v4f acc[S::RB][S::CB];
#pragma unroll
  for (int rb = 0; rb < S::RB; ++rb)
#pragma unroll
    for (int cb = 0; cb < S::CB; ++cb) acc[rb][cb] = {0.f, 0.f, 0.f, 0.f};

  const float* sq[S::CB];
#pragma unroll
  for (int cb = 0; cb < S::CB; ++cb) {
    const int64_t r = q0 + min(wq * (S::BQ / S::WQ) + cb * 16 + (lane & 15), qv - 1);
    sq[cb] = a.sq + (r >> a.q_shift) * a.ldsq;
  }
  // square form: the wave's rows of P lie in one 128-block of scales
  const float* sp = a.sp + (int64_t)((p0 + wp * (S::BP / S::WP)) / kBlock) * a.ldsp;
  if (!PVEC && p0 + wp * (S::BP / S::WP) >= a.n) sp = a.sp;

  auto issue = [&](int c) {
    unsigned char* st = lds + (c & 1) * S::STAGE;
    const int64_t k0 = (int64_t)c * kChunkBytes;
    const int left = a.k - (int)k0;
    if (a.fast && left >= kChunkBytes) {
      copy_along<S::BP, S::NW, 8>(a.p, a.ldp, p0, pv, k0, 8, st, wave, lane);
      copy_along<S::BQ, S::NW, 8>(a.q, a.ldq, q0, qv, k0, 8, st + S::P_BYTES, wave, lane);
    } else {
      edge_along<S::BP, S::THREADS, 1, 8>(a.p, a.ldp, p0, pv, k0, left, a.fast, st, threadIdx.x);
      edge_along<S::BQ, S::THREADS, 1, 8>(a.q, a.ldq, q0, qv, k0, left, a.fast, st + S::P_BYTES, threadIdx.x);
    }
    if (PVEC) {
      float* s = reinterpret_cast<float*>(st + S::P_BYTES + S::Q_BYTES);
      for (int t = threadIdx.x; t < S::BP; t += S::THREADS) s[t] = t < pv ? a.sp[(int64_t)(p0 + t) * a.ldsp + c] : 0.f;
    }
  };

  if (c_begin < c_end) issue(c_begin);
  for (int c = c_begin; c < c_end; ++c) {
    float sc[S::CB];
#pragma unroll
    for (int cb = 0; cb < S::CB; ++cb) sc[cb] = sq[cb][c];
    if (!PVEC) {
      const float s = sp[c];
#pragma unroll
      for (int cb = 0; cb < S::CB; ++cb) sc[cb] *= s;
    }
    stage_barrier();  // chunk c is in LDS; every wave is done with chunk c - 1
    if (c + 1 < c_end) issue(c + 1);
    const unsigned char* st = lds + (c & 1) * S::STAGE;
    typename Frag8<WIDE, QF>::type fq[S::CB];
#pragma unroll
    for (int cb = 0; cb < S::CB; ++cb)
      fq[cb] = Frag8<WIDE, QF>::of(frag8(st + S::P_BYTES, wq * (S::BQ / S::WQ) + cb * 16, lane));
#pragma unroll
    for (int rb = 0; rb < S::RB; ++rb) {
      const int row = wp * (S::BP / S::WP) + rb * 16;
      const typename Frag8<WIDE, 0>::type fp = Frag8<WIDE, 0>::of(frag8(st, row, lane));
      v4f d[S::CB];
#pragma unroll
      for (int cb = 0; cb < S::CB; ++cb) d[cb] = product<QF>(fp, fq[cb]);
      if (PVEC) {
        const f4 s = *reinterpret_cast<const f4*>(st + S::P_BYTES + S::Q_BYTES + (row + 4 * (lane >> 4)) * 4);
#pragma unroll
        for (int cb = 0; cb < S::CB; ++cb)
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[rb][cb][v] = fmaf(d[cb][v] * sc[cb], s[v], acc[rb][cb][v]);
      } else {
#pragma unroll
        for (int cb = 0; cb < S::CB; ++cb)
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[rb][cb][v] = fmaf(d[cb][v], sc[cb], acc[rb][cb][v]);
      }
    }
  }

#pragma unroll
  for (int cb = 0; cb < S::CB; ++cb) {
    const int qr = wq * (S::BQ / S::WQ) + cb * 16 + (lane & 15);
    if (qr >= qv) continue;
#pragma unroll
    for (int rb = 0; rb < S::RB; ++rb) {
      const int pr = wp * (S::BP / S::WP) + rb * 16 + 4 * (lane >> 4);
      if (pr >= pv) continue;
      const float v[4] = {acc[rb][cb][0], acc[rb][cb][1], acc[rb][cb][2], acc[rb][cb][3]};
      if (a.partial)
        put4(a.partial + ((int64_t)blockIdx.y * a.m + q0 + qr) * a.n + p0 + pr, v, pv - pr, a.n % 4 == 0, false);
      else
        put4_as(a.c, (q0 + qr) * a.ldc + p0 + pr, v, pv - pr, a.c_type, a.vec_c, a.accumulate);
    }
  }
}

// Few rows of C (m <= 16 CB): no tile in LDS.  A workgroup of NW waves owns 16
// rows of P (16 columns of C); wave w takes the chunks of 128 steps w, w + NW,
// ..., straight from global memory into the fragments (P's bytes are read once
// over the whole launch), and the waves' sums are added through LDS in wave
// order.
template <int CB, int NW, int QF, bool PVEC, bool WIDE>
__global__ __launch_bounds__(64 * NW) void scaled_rows_kernel(const ScaledArgs a) {
  __shared__ v4f part[NW][CB][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane >> 4, i = lane & 15;
  const int p0 = blockIdx.x * 16;
  const int pr = min(p0 + i, a.n - 1);
  const unsigned char* p = a.p + (int64_t)pr * a.ldp;
  const int chunks = (a.k + kChunkBytes - 1) / kChunkBytes;
  v4f acc[CB];
#pragma unroll
  for (int cb = 0; cb < CB; ++cb) acc[cb] = {0.f, 0.f, 0.f, 0.f};
  auto frag = [&](const unsigned char* row, int c) -> v8i {
    const int64_t k0 = (int64_t)c * kChunkBytes + 16 * g;
    const int left = a.k - (int)k0;
    if (a.fast && c * kChunkBytes + kChunkBytes <= a.k)
      return join(*reinterpret_cast<const v4i*>(row + k0), *reinterpret_cast<const v4i*>(row + k0 + 64));
    const v4u u = edge_unit<1>(row + k0, left, a.fast), v = edge_unit<1>(row + k0 + 64, left - 64, a.fast);
    return join(__builtin_bit_cast(v4i, u), __builtin_bit_cast(v4i, v));
  };
  for (int c = wave; c < chunks; c += NW) {
    const typename Frag8<WIDE, 0>::type fp = Frag8<WIDE, 0>::of(frag(p, c));
    float s[4];
    if (PVEC) {
#pragma unroll
      for (int v = 0; v < 4; ++v) s[v] = a.sp[(int64_t)min(p0 + 4 * g + v, a.n - 1) * a.ldsp + c];
    } else {
      s[0] = a.sp[(int64_t)(p0 / kBlock) * a.ldsp + c];
    }
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) {
      const int64_t r = min((int64_t)(cb * 16 + i), a.m - 1);
      const float sc = a.sq[(r >> a.q_shift) * a.ldsq + c];
      const v4f d = product<QF>(fp, Frag8<WIDE, QF>::of(frag(a.q + r * a.ldq, c)));
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[cb][v] = fmaf(d[v], sc * s[PVEC ? v : 0], acc[cb][v]);
    }
  }
#pragma unroll
  for (int cb = 0; cb < CB; ++cb) part[wave][cb][lane] = acc[cb];
  __syncthreads();
  for (int cb = wave; cb < CB; cb += NW) {
    v4f t = part[0][cb][lane];
#pragma unroll
    for (int w = 1; w < NW; ++w) t += part[w][cb][lane];
    const int64_t r = cb * 16 + i;
    if (r < a.m && p0 + 4 * g < a.n) {
      const float v[4] = {t[0], t[1], t[2], t[3]};
      put4_as(a.c, r * a.ldc + p0 + 4 * g, v, a.n - p0 - 4 * g, a.c_type, a.vec_c, a.accumulate);
    }
  }
}

// C = the sum of the splits' partial products (in split order).
__global__ __launch_bounds__(256) void scaled_join_kernel(const ScaledArgs a) {
  const int quads = (a.n + 3) / 4;
  const int64_t total = a.m * quads;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / quads;
    const int c = (int)(i % quads) * 4, left = a.n - c;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
    for (int z = 0; z < a.splits; ++z) {
      const float* p = a.partial + ((int64_t)z * a.m + r) * a.n + c;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < left) v[j] += p[j];
    }
    put4_as(a.c, r * a.ldc + c, v, left, a.c_type, a.vec_c, a.accumulate);
  }
}

// ------------------------------------------------------------ launchers
namespace {

using Tile128 = ScaledShape<128, 128, 2, 2>;
using Tile256 = ScaledShape<256, 256, 2, 4>;
constexpr int kFewRows = 64;
constexpr int kCus = 256;

template <class S, int QF, bool PVEC, bool WIDE>
hipError_t go_tile(const ScaledArgs& a, hipStream_t s) {
  static bool raised = false;
  if (!raised) {
    hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(scaled_tile_kernel<S, QF, PVEC, WIDE>),
                                       hipFuncAttributeMaxDynamicSharedMemorySize, S::LDS);
    if (e != hipSuccess) return e;
    raised = true;
  }
  const int64_t tiles = (int64_t)((a.n + S::BP - 1) / S::BP) * ((a.m + S::BQ - 1) / S::BQ);
  hipLaunchKernelGGL((scaled_tile_kernel<S, QF, PVEC, WIDE>), dim3((unsigned)tiles, a.splits), dim3(S::THREADS), S::LDS, s,
                     a);
  return hipGetLastError();
}

template <int CB, int QF, bool PVEC, bool WIDE>
hipError_t go_rows(const ScaledArgs& a, hipStream_t s) {
  const dim3 grid((a.n + 15) / 16);
  hipLaunchKernelGGL((scaled_rows_kernel<CB, 8, QF, PVEC, WIDE>), grid, dim3(512), 0, s, a);
  return hipGetLastError();
}

template <int QF, bool PVEC, bool WIDE>
hipError_t go_kind(const ScaledArgs& a, int kind, hipStream_t s) {
  if constexpr (!WIDE)
    if (kind == 2) return go_tile<Tile256, QF, PVEC, WIDE>(a, s);
  if (kind >= 1) return go_tile<Tile128, QF, PVEC, WIDE>(a, s);
  if (a.m <= 16) return go_rows<1, QF, PVEC, WIDE>(a, s);
  if (a.m <= 32) return go_rows<2, QF, PVEC, WIDE>(a, s);
  return go_rows<4, QF, PVEC, WIDE>(a, s);
}

template <int QF, bool PVEC>
hipError_t go_width(const ScaledArgs& a, int kind, hipStream_t s) {
  return a.c_type == MR_F32 ? go_kind<QF, PVEC, true>(a, kind, s) : go_kind<QF, PVEC, false>(a, kind, s);
}

}  // namespace

ScaledPlan scaled_plan(int64_t m, int64_t n, int64_t k) {
  if (m <= kFewRows) return {0, 1};
  const int64_t chunks = (k + kChunkBytes - 1) / kChunkBytes;
  auto tiles = [&](int b) { return ((m + b - 1) / b) * ((n + b - 1) / b); };
  if (tiles(256) >= kCus) return {2, 1};
  const int64_t t = tiles(128);
  int64_t splits = 1;
  while (splits < 16 && t * splits * 2 <= 2 * kCus && chunks / (splits * 2) >= 8) splits *= 2;
  return {1, (int)splits};
}

hipError_t launch_scaled(const ScaledArgs& a, const ScaledPlan& plan, hipStream_t s) {
  if (a.q_e5m2) return a.p_vector ? go_width<1, true>(a, plan.kind, s) : go_width<1, false>(a, plan.kind, s);
  return a.p_vector ? go_width<0, true>(a, plan.kind, s) : go_width<0, false>(a, plan.kind, s);
}

hipError_t launch_scaled_join(const ScaledArgs& a, hipStream_t s) {
  const int64_t quads = a.m * ((a.n + 3) / 4);
  const int64_t blocks = (quads + 255) / 256;
  hipLaunchKernelGGL(scaled_join_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace mr
