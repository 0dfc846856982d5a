// Products of rows grouped by expert (ragged groups, offsets read on the
// device), 16-bit operands, float32 sums on v_mfma_f32_32x32x16:
//
//   forward    y_r = W_e x_r      P = W_e (along k),        Q = x (along k)
//   transpose  y_r = W_e^T x_r    P = W_e^T (across n),     Q = x (along n)
//   weights    DW_e = sum_r dy_r x_r^T
//                                 P = x (across rows),      Q = dy (across rows)
//
// P is the matrix instruction's row operand, so a lane holds four consecutive
// outputs of one output row.  Operands whose contraction is not contiguous in
// memory ("across") go through ds_read_b64_tr_b16, which hands each lane four
// steps of one column; no transposed copy of a weight is ever made.
//
// Row tiles never span two experts.  A launch holds an upper bound of the
// tiles (rows / tile + experts); every workgroup finds its own from the
// offsets (one wave scan per 64 experts), so no size reaches the host and the
// call can be captured and replayed under other sizes.
#include "tile_core.hpp"

namespace mr {

namespace {

typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) v4s* lds_v4s;

template <typename T>
__device__ __forceinline__ v16f mfma16(v8s p, v8s q, v16f c);
template <>
__device__ __forceinline__ v16f mfma16<_Float16>(v8s p, v8s q, v16f c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, p), __builtin_bit_cast(v8h, q), c, 0, 0, 0);
}
template <>
__device__ __forceinline__ v16f mfma16<bf16_t>(v8s p, v8s q, v16f c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8b, p), __builtin_bit_cast(v8b, q), c, 0, 0, 0);
}

// Lane l's part of rows row .. row + 31 at steps 16 ks .. + 15 of a chunk of
// R-row tile `st`: row l % 32, steps 8 (l / 32) .. + 7.
template <int R, bool ACROSS>
__device__ __forceinline__ v8s frag16(const unsigned char* st, int row, int ks, int lane) {
  if constexpr (!ACROSS) {
    const int r = row + (lane & 31);
    return *reinterpret_cast<const v8s*>(st + (r * 8 + dl_slot(r, 2 * ks + (lane >> 5), 8)) * 16);
  } else {
    // 16 lanes read four steps x 16 columns (lane i: step i / 4, columns 4 (i % 4) ..)
    // and each gets the four steps of column i
    constexpr int UPR = R / 8;
    const int i = lane & 15;
    const int unit = (row + 16 * ((lane >> 4) & 1)) / 8 + ((i & 3) >> 1);
    const int k = 16 * ks + 8 * (lane >> 5) + (i >> 2);
    const unsigned char* p = st + (k * UPR + (unit ^ across_swap<R>(k))) * 16 + 8 * (i & 1);
    const v4s a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)p);
    // steps + 4: the same k & 3, so the same slot four LDS rows on
    const v4s b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(p + 4 * UPR * 16));
    return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
  }
}

__device__ __forceinline__ int64_t offset_at(const GroupedArgs& a, int e) {
  const int64_t v = a.wide_offsets ? reinterpret_cast<const int64_t*>(a.offsets)[e]
                                   : (int64_t) reinterpret_cast<const int32_t*>(a.offsets)[e];
  return v < 0 ? 0 : v > a.rows ? a.rows : v;
}
// Segment s of the rows: 0 the rows before the first expert, 1 .. E the
// experts, E + 1 the rows after the last one.
__device__ __forceinline__ void segment(const GroupedArgs& a, int s, int64_t& begin, int64_t& end) {
  begin = s == 0 ? 0 : offset_at(a, s - 1);
  end = s > a.experts ? a.rows : offset_at(a, s);
  if (end < begin) end = begin;
}

// Segment and tile within it of tile `id`, BQ rows to a tile, `across` column
// tiles to a row tile; false past the last one.  Every wave does the same scan.
template <int BQ>
__device__ __forceinline__ bool find_tile(const GroupedArgs& a, int64_t id, int across, int& seg, int64_t& begin,
                                          int64_t& end, int& local) {
  const int lane = threadIdx.x & 63;
  int64_t base = 0;
  for (int s0 = 0; s0 < a.experts + 2; s0 += 64) {
    const int s = s0 + lane;
    int64_t b = 0, e = 0;
    if (s < a.experts + 2) segment(a, s, b, e);
    const int64_t tiles = (e - b + BQ - 1) / BQ * across;
    int64_t sum = tiles;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t up = __shfl_up(sum, d);
      if (lane >= d) sum += up;
    }
    const uint64_t hit = __ballot(id < base + sum);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      seg = s0 + l;
      begin = __shfl(b, l);
      end = __shfl(e, l);
      local = (int)(id - base - (__shfl(sum, l) - __shfl(tiles, l)));
      return true;
    }
    base += __shfl(sum, 63);
  }
  return false;
}

}  // namespace

template <int BP_, int BQ_, int WP_, int WQ_>
struct GroupedShape {
  static constexpr int BP = BP_, BQ = BQ_, WP = WP_, WQ = WQ_, NW = WP * WQ, THREADS = 64 * NW;
  static constexpr int RB = BP / WP / 32, CB = BQ / WQ / 32;
  static constexpr int P_BYTES = BP * kChunkBytes, STAGE = (BP + BQ) * kChunkBytes;
  static constexpr int LDS = 2 * STAGE;
};

// One operand of a tile: rows (products' rows) r0 .. of `valid`, bytes.
struct Operand {
  const unsigned char* base;
  int64_t ld_bytes, r0;
  int valid;
};

// acc = P Q^T over `steps` of the contraction starting at step 0 of both.
template <class S, typename T, bool PA, bool QA>
__device__ __forceinline__ void grouped_tile(const Operand& P, const Operand& Q, int64_t steps, bool fast, unsigned char* lds,
                                             v16f (&acc)[S::RB][S::CB]) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wp = wave / S::WQ, wq = wave % S::WQ;
#pragma unroll
  for (int rb = 0; rb < S::RB; ++rb)
#pragma unroll
    for (int cb = 0; cb < S::CB; ++cb)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[rb][cb][v] = 0.f;
  const int chunks = (int)((steps + 63) / 64);
  // an `across` tile at a ragged column edge that splits a 16-byte unit goes element by element
  const bool p_fast = fast && (!PA || P.valid == S::BP || P.valid % 8 == 0);
  const bool q_fast = fast && (!QA || Q.valid == S::BQ || Q.valid % 8 == 0);
  auto issue = [&](int c) {
    unsigned char* st = lds + (c & 1) * S::STAGE;
    const int64_t k0 = (int64_t)c * 64;
    const int left = (int)min((int64_t)64, steps - k0);
    if constexpr (PA) {
      if (p_fast && left == 64)
        copy_across<S::BP, S::NW>(P.base, P.ld_bytes, k0, P.r0, P.valid, st, wave, lane);
      else
        edge_across<S::BP, S::THREADS>(P.base, P.ld_bytes, k0, left, P.r0, P.valid, fast, st);
    } else {
      if (p_fast && left == 64)
        copy_along<S::BP, S::NW>(P.base, P.ld_bytes, P.r0, P.valid, k0 * 2, st, wave, lane);
      else
        edge_along<S::BP, S::THREADS, 2>(P.base, P.ld_bytes, P.r0, P.valid, k0 * 2, left, fast, st);
    }
    st += S::P_BYTES;
    if constexpr (QA) {
      if (q_fast && left == 64)
        copy_across<S::BQ, S::NW>(Q.base, Q.ld_bytes, k0, Q.r0, Q.valid, st, wave, lane);
      else
        edge_across<S::BQ, S::THREADS>(Q.base, Q.ld_bytes, k0, left, Q.r0, Q.valid, fast, st);
    } else {
      if (q_fast && left == 64)
        copy_along<S::BQ, S::NW>(Q.base, Q.ld_bytes, Q.r0, Q.valid, k0 * 2, st, wave, lane);
      else
        edge_along<S::BQ, S::THREADS, 2>(Q.base, Q.ld_bytes, Q.r0, Q.valid, k0 * 2, left, fast, st);
    }
  };
  if (chunks > 0) issue(0);
  for (int c = 0; c < chunks; ++c) {
    stage_barrier();  // chunk c is in LDS; every wave is done with chunk c - 1
    if (c + 1 < chunks) issue(c + 1);
    const unsigned char* st = lds + (c & 1) * S::STAGE;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      v8s p[S::RB], q[S::CB];
#pragma unroll
      for (int rb = 0; rb < S::RB; ++rb) p[rb] = frag16<S::BP, PA>(st, wp * (S::BP / S::WP) + rb * 32, ks, lane);
#pragma unroll
      for (int cb = 0; cb < S::CB; ++cb) q[cb] = frag16<S::BQ, QA>(st + S::P_BYTES, wq * (S::BQ / S::WQ) + cb * 32, ks, lane);
#pragma unroll
      for (int rb = 0; rb < S::RB; ++rb)
#pragma unroll
        for (int cb = 0; cb < S::CB; ++cb) acc[rb][cb] = mfma16<T>(p[rb], q[cb], acc[rb][cb]);
    }
  }
}

// Rows q0 .. of Y (leading dimension ldy) from the accumulators, or zeros.
template <class S, typename T>
__device__ __forceinline__ void put_tile(const GroupedArgs& a, char* y, int64_t q0, int qv, int p0, int pv,
                                         const v16f (&acc)[S::RB][S::CB]) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int wp = wave / S::WQ, wq = wave % S::WQ;
#pragma unroll
  for (int cb = 0; cb < S::CB; ++cb) {
    const int qr = wq * (S::BQ / S::WQ) + cb * 32 + (lane & 31);
    if (qr >= qv) continue;
    const int64_t row = (q0 + qr) * a.ldy;
#pragma unroll
    for (int rb = 0; rb < S::RB; ++rb)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int pr = wp * (S::BP / S::WP) + rb * 32 + 8 * u + 4 * (lane >> 5);
        if (pr >= pv) continue;
        const float v[4] = {acc[rb][cb][4 * u], acc[rb][cb][4 * u + 1], acc[rb][cb][4 * u + 2], acc[rb][cb][4 * u + 3]};
        if (a.y_f32)
          put4(reinterpret_cast<float*>(y) + row + p0 + pr, v, pv - pr, a.vec_y, a.accumulate);
        else
          put4(reinterpret_cast<T*>(y) + row + p0 + pr, v, pv - pr, a.vec_y, a.accumulate);
      }
  }
}

template <class S, typename T, bool TRANSPOSE>
__global__ __launch_bounds__(S::THREADS) void grouped_tile_kernel(const GroupedArgs a) {
  extern __shared__ __align__(256) unsigned char lds[];
  const int outs = TRANSPOSE ? a.k : a.n, steps = TRANSPOSE ? a.n : a.k;
  const int across = (outs + S::BP - 1) / S::BP;
  int seg, local;
  int64_t begin, end;
  if (!find_tile<S::BQ>(a, xcd_remap(blockIdx.x, gridDim.x), across, seg, begin, end, local)) return;
  // an expert's row tiles follow one another under one panel of its weight
  const int down = (int)((end - begin + S::BQ - 1) / S::BQ);
  const int p0 = local / down * S::BP;
  const int64_t q0 = begin + (int64_t)(local % down) * S::BQ;
  const int pv = min(S::BP, outs - p0), qv = (int)min((int64_t)S::BQ, end - q0);
  const bool expert = seg >= 1 && seg <= a.experts;
  const unsigned char* w = reinterpret_cast<const unsigned char*>(a.w) + (expert ? seg - 1 : 0) * a.w_stride * 2;
  const Operand P{w, a.ldw * 2, p0, pv};
  const Operand Q{reinterpret_cast<const unsigned char*>(a.x), a.ldx * 2, q0, qv};
  v16f acc[S::RB][S::CB];
  grouped_tile<S, T, TRANSPOSE, false>(P, Q, expert ? steps : 0, a.fast, lds, acc);
  put_tile<S, T>(a, reinterpret_cast<char*>(a.y), q0, qv, p0, pv, acc);
}

template <class S, typename T>
__global__ __launch_bounds__(S::THREADS) void grouped_weight_kernel(const GroupedArgs a) {
  extern __shared__ __align__(256) unsigned char lds[];
  const int tp = (a.k + S::BP - 1) / S::BP, tq = (a.n + S::BQ - 1) / S::BQ;
  const int64_t id = xcd_remap(blockIdx.x, gridDim.x);
  const int e = (int)(id / (tp * tq)), local = (int)(id % (tp * tq));
  int64_t begin, end;
  segment(a, e + 1, begin, end);
  const int p0 = local % tp * S::BP, q0 = local / tp * S::BQ;
  const int pv = min(S::BP, a.k - p0), qv = min(S::BQ, a.n - q0);
  const Operand P{reinterpret_cast<const unsigned char*>(a.w) + begin * a.ldw * 2, a.ldw * 2, p0, pv};
  const Operand Q{reinterpret_cast<const unsigned char*>(a.x) + begin * a.ldx * 2, a.ldx * 2, q0, qv};
  v16f acc[S::RB][S::CB];
  grouped_tile<S, T, true, true>(P, Q, end - begin, a.fast, lds, acc);
  char* y = reinterpret_cast<char*>(a.y) + e * a.y_stride * (a.y_f32 ? 4 : 2);
  put_tile<S, T>(a, y, q0, qv, p0, pv, acc);
}

// ------------------------------------------------------------ launchers
namespace {

using Tile128 = GroupedShape<128, 128, 2, 2>;

template <class K>
hipError_t raise_lds(K kernel, int bytes, bool& raised) {
  if (raised) return hipSuccess;
  hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  raised = e == hipSuccess;
  return e;
}

template <class S, typename T, bool TRANSPOSE>
hipError_t go_rows(const GroupedArgs& a, hipStream_t s) {
  static bool raised = false;
  auto kernel = grouped_tile_kernel<S, T, TRANSPOSE>;
  if (hipError_t e = raise_lds(kernel, S::LDS, raised); e != hipSuccess) return e;
  const int64_t outs = TRANSPOSE ? a.k : a.n;
  const int64_t segments = a.experts + 2 < a.rows ? a.experts + 2 : a.rows;
  const int64_t tiles = (a.rows / S::BQ + segments) * ((outs + S::BP - 1) / S::BP);
  hipLaunchKernelGGL(kernel, dim3((unsigned)tiles), dim3(S::THREADS), S::LDS, s, a);
  return hipGetLastError();
}

template <class S, typename T>
hipError_t go_weights(const GroupedArgs& a, hipStream_t s) {
  static bool raised = false;
  auto kernel = grouped_weight_kernel<S, T>;
  if (hipError_t e = raise_lds(kernel, S::LDS, raised); e != hipSuccess) return e;
  const int64_t tiles = (int64_t)a.experts * ((a.k + S::BP - 1) / S::BP) * ((a.n + S::BQ - 1) / S::BQ);
  hipLaunchKernelGGL(kernel, dim3((unsigned)tiles), dim3(S::THREADS), S::LDS, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped(const GroupedArgs& a, mr_dtype dt, bool transpose, hipStream_t s) {
  if (dt == MR_F16) return transpose ? go_rows<Tile128, _Float16, true>(a, s) : go_rows<Tile128, _Float16, false>(a, s);
  return transpose ? go_rows<Tile128, bf16_t, true>(a, s) : go_rows<Tile128, bf16_t, false>(a, s);
}

hipError_t launch_grouped_weight_grad(const GroupedArgs& a, mr_dtype dt, hipStream_t s) {
  return dt == MR_F16 ? go_weights<Tile128, _Float16>(a, s) : go_weights<Tile128, bf16_t>(a, s);
}

}  // namespace mr
