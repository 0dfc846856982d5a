// Products of 8-bit matrices with a float32 scale per block of 128 of the
// contraction:
//
//   C_ij = sum_b sa_ib sb_jb sum_{l in b} A_il B_jl.
//
// Every inner sum of 128 is one v_mfma_f32_16x16x128_f8f6f4; its result is
// scaled and added to a float32 accumulator by the vector units.  That instruction
// adds the products of eight steps on a common exponent and cuts them at 2^-13 of
// the largest one's power of two (next to 2^16 and -2^16 the smallest product that
// counts is 2^3 among their eight, 2^-7 among the others): in the sum of
// magnitudes at most 2^-10, measured 1e-5 at most, and 1.4e-5 to 1.8e-5 of the
// results in the mean square (random and activation-like operands, k = 2048 and
// 8192).  A 16-bit C's own rounding is 1.7e-3 (bf16), 2.1e-4 (fp16) there; where
// large products cancel, what is left loses those places.  A float32 C shows them
// always, and for few rows the bytes bound the product: there the operands are
// widened to fp16 in registers (exactly: both 8-bit types are subsets) and the
// sums run on v_mfma_f32_16x16x32_f16, which adds in float32, at half the rate
// (6e-8 of the results).
//
// B is the instruction's row operand ("P"), A its column operand ("Q"): a lane then
// holds one row of C, so A's scale is one value per lane and column block, B's (one
// per 128 rows in the square form) one per wave, and their product costs one
// multiplication per column block beside one FMA per output.  Where that product is
// no normal number, and for B's scales by row, a sum takes the two in turn.  The
// instruction's order of the 128 steps within a lane does not matter, since both
// operands use the same one.
//
// What bounds it (16384 x 8192 x 2048 to bf16, one MI355X): 289 us, 1.90
// PFLOP/s, against 246 us for the vendor's unscaled 8-bit product.  The matrix
// instructions alone take about 130 us (4.3 PFLOP/s with four additions each,
// registers only); the rest is what they wait for: copies into LDS (64 KB a
// chunk and CU; 247 us without them), the stores of C (32 us, all CUs at once),
// and the clock, which falls to 2 GHz.  8192 x 2048 x 16383 to float32: 555 us,
// 0.99 PFLOP/s, on fp16 instructions (1.5 in the vendor's bf16 product).  There
// vector instructions take 45% of a SIMD's cycles (4.4 per matrix instruction:
// widening, scaling, adding), matrix instructions 41% and LDS 14%; the two waves of
// a SIMD do little of the first two at the same time.  8 x 4096 x 1024: 3.8 us, a
// launch and one pass over 4 MB.
#include <type_traits>

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
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(p, q, zero, 0, QF, 0, 0, 0, 0);  // zeros: the unscaled form
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
// d[i] = P Q_i^T for N column blocks (the fp16 form in four passes over the
// blocks, so that no product waits for the one before it).
template <int QF, int N>
__device__ __forceinline__ void products(v8i p, const v8i (&q)[N], v4f (&d)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) d[i] = mfma8<QF>(p, q[i]);
}
template <int QF, int N>
__device__ __forceinline__ void products(const Wide& p, const Wide (&q)[N], v4f (&d)[N]) {
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const v4f zero = {0.f, 0.f, 0.f, 0.f};
      d[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(p.h[k], q[i].h[k], k == 0 ? zero : d[i], 0, 0, 0);
    }
}

// Whether a lane's part of a fragment holds anything but zeros.
__device__ __forceinline__ bool holds_values(v8i x) {
  int u = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) u |= x[i];
  return (u & 0x7f7f7f7f) != 0;
}
__device__ __forceinline__ bool holds_values(const Wide& x) {
  bool r = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const v4i u = __builtin_bit_cast(v4i, x.h[i]);
    r |= ((u[0] | u[1] | u[2] | u[3]) & 0x7fff7fff) != 0;
  }
  return r;
}

// Scales q and s of a block's sum d, as two factors.  The product of the scales may
// be past float32's range, or among its subnormal numbers, where d q s is not: then
// they are taken in turn, first the one that keeps such a result within range.
struct BothScales {
  float first = 1.f, then;
  bool in_turn;
  __device__ __forceinline__ BothScales(float q, float s) : then(q * s) {
    constexpr int not_normal = 0x2f7, some = 0x198;  // zero, subnormal, infinite or NaN; finite and not zero
    in_turn = __builtin_amdgcn_classf(then, not_normal) && __builtin_amdgcn_classf(q, some) && __builtin_amdgcn_classf(s, some);
    if (in_turn) {
      const bool q_first = (fabsf(then) > 1.f) == (fabsf(q) < fabsf(s));
      first = q_first ? q : s;
      then = q_first ? s : q;
    }
  }
  __device__ __forceinline__ float add(float d, float acc) const { return fmaf(d * first, then, acc); }
};

__device__ __forceinline__ v8i join(v4i a, v4i b) {
  return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Fragment of rows row .. row + 15 (row a multiple of 16) of an LDS chunk: bytes
// 16 g and 64 + 16 g, g = lane / 16.  The slots depend on row % 16 alone, so a
// lane has two offsets for all fragments.
__device__ __forceinline__ v8i frag8(const unsigned char* st, int row, int lane) {
  const int r = lane & 15, g = lane >> 4;
  const unsigned char* p = st + row * kChunkBytes;
  const v4i a = *reinterpret_cast<const v4i*>(p + (r * 8 + dl_slot(r, g, 8)) * 16);
  const v4i b = *reinterpret_cast<const v4i*>(p + (r * 8 + dl_slot(r, g + 4, 8)) * 16);
  return join(a, b);
}

}  // namespace

template <int BP_, int BQ_, int WP_, int WQ_, int BPC_>
struct ScaledShape {
  static constexpr int BP = BP_, BQ = BQ_, WP = WP_, WQ = WQ_, NW = WP * WQ, BPC = BPC_, THREADS = 64 * NW;
  static constexpr int RB = BP / WP / 16, CB = BQ / WQ / 16;
  static constexpr int P_BYTES = BP * kChunkBytes, Q_BYTES = BQ * kChunkBytes;
  // P, Q, P's scales, Q's scales
  static constexpr int SP = P_BYTES + Q_BYTES, SQ = SP + BP * 4, STAGE = SQ + BQ * 4;
  static constexpr int NP = along_copies<BP, NW, 8>, NQ = along_copies<BQ, NW, 8>;  // copies per wave and chunk
  static constexpr int NS = (BP + BQ + 64 * NW - 1) / (64 * NW);
  static constexpr int SLABS = 2 * STAGE, LDS = SLABS + NW * Slab<float, 16>::BYTES;
  static constexpr int WAVES_PER_SIMD = BPC * NW / 4;
  static_assert(RB % 2 == 0 && BPC * LDS <= 160 * 1024, "the stages fit");
};

// One tile of C, or of one part of a split contraction.
template <class S>
struct ScaledTile {
  int64_t q0;
  int p0, pv, qv, part, c_begin, c_end;
  __device__ __forceinline__ void load(const ScaledArgs& a, int id) {
    const int tp = (a.n + S::BP - 1) / S::BP, tq = (int)((a.m + S::BQ - 1) / S::BQ);
    part = id / (tp * tq);
    int ti, tj;
    full_tile_grouped(id % (tp * tq), tq, tp, ti, tj);
    q0 = (int64_t)ti * S::BQ;
    p0 = tj * S::BP;
    pv = min(S::BP, a.n - p0);
    qv = (int)min((int64_t)S::BQ, a.m - q0);
    const int64_t chunks = (a.k + kChunkBytes - 1) / kChunkBytes;
    c_begin = (int)(chunks * part / a.splits);
    c_end = (int)(chunks * (part + 1) / a.splits);
  }
};

// The chunks of a workgroup's tiles in order, for the copies (past the last one
// it stays on that one).  Scalar addresses move along with the chunks; a whole
// tile's copies then cost a scalar addition each (worked out per chunk and copy,
// the addresses took 20 us of 300 at 16384 x 8192 x 2048).
template <class S>
struct ScaledFeed {
  ScaledTile<S> t;
  Walk w;
  int c, left;
  bool whole;  // the tile has all its rows
  unsigned char* st;
  const char *p, *q, *sp, *sq;
  uint32_t p_off, q_off;  // a lane's place in 8 NW rows of P, of Q
  __device__ __forceinline__ ScaledFeed(const ScaledArgs& a, const Walk& w_, int wave, int lane) : w(w_) {
    const int row = wave * 8 + (lane >> 3);
    static_assert(8 * S::NW % 16 == 0, "the slot of a unit is the same in every group of rows");
    const uint32_t slot = (uint32_t)dl_slot(row, lane & 7, 8) * 16u;
    p_off = (uint32_t)row * (uint32_t)a.ldp + slot;
    q_off = (uint32_t)row * (uint32_t)a.ldq + slot;
    enter(a);
  }
  __device__ __forceinline__ void enter(const ScaledArgs& a) {  // the tile at w.at
    t.load(a, w.at);
    c = t.c_begin;
    whole = t.pv == S::BP && t.qv == S::BQ;
    const int64_t k0 = (int64_t)c * kChunkBytes;
    left = (int)min((int64_t)kChunkBytes, a.k - k0);
    p = wave_uniform(a.p + (int64_t)t.p0 * a.ldp + k0);
    q = wave_uniform(a.q + t.q0 * a.ldq + k0);
    sp = wave_uniform(a.sp + (int64_t)(t.p0 >> a.p_shift) * a.ldsp + c);
    sq = wave_uniform(a.sq + (t.q0 >> a.q_shift) * a.ldsq + c);
  }
  template <int N>
  static __device__ __forceinline__ void copy_rows(const char* base, int64_t step, uint32_t off, unsigned char* to) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      asm volatile("" : "+v"(off));
      __builtin_amdgcn_global_load_lds((global_void_ptr)(base + off), (lds_void_ptr)(to + j * S::NW * 1024), 16, 0, 0);
      base += step;
    }
  }
  // The wave's copies of the current chunk into `stage`.
  __device__ __forceinline__ void copy(const ScaledArgs& a, unsigned char* stage, int wave, int lane) {
    st = stage;
    if (whole && left == kChunkBytes) {
      copy_rows<S::NP>(p, (int64_t)(8 * S::NW) * a.ldp, p_off, st + wave * 1024);
      copy_rows<S::NQ>(q, (int64_t)(8 * S::NW) * a.ldq, q_off, st + S::P_BYTES + wave * 1024);
    } else {
      const int units = (left + 15) >> 4;
#pragma unroll
      for (int j = 0; j < S::NP; ++j) copy_along_one<S::BP, S::NW, 8>(p, a.ldp, t.pv, units, st, wave, lane, j);
#pragma unroll
      for (int j = 0; j < S::NQ; ++j) copy_along_one<S::BQ, S::NW, 8>(q, a.ldq, t.qv, units, st + S::P_BYTES, wave, lane, j);
    }
#pragma unroll
    for (int j = 0; j < S::NS; ++j) {
      // the scale of row i of P, then of Q, 64 rows to a copy (rows past the end repeat the last
      // one, surplus copies the first ones); tiles start at multiples of 128 rows
      const int first = ((j * S::NW + wave) * 64) % (S::BP + S::BQ);
      const bool is_p = first < S::BP;
      const int row = min(is_p ? first + lane : first - S::BP + lane, (is_p ? t.pv : t.qv) - 1);
      uint32_t off = (uint32_t)(row >> (is_p ? a.p_shift : a.q_shift)) * (uint32_t)(is_p ? a.ldsp : a.ldsq) * 4u;
      const char* s = is_p ? sp : sq;
      asm volatile("" : "+v"(off));
      asm volatile("" : "+s"(s));
      __builtin_amdgcn_global_load_lds((global_void_ptr)(s + off), (lds_void_ptr)(st + S::SP + first * 4), 4, 0, 0);
    }
  }
  // The current chunk has landed (and a barrier has passed): the bytes past the
  // contraction's end become zeros, so that nothing that lies there reaches a sum.
  __device__ __forceinline__ void clear_end() const {
    for (int r = threadIdx.x; r < S::BP + S::BQ; r += S::THREADS) {
#pragma unroll 1
      for (int u = left >> 4; u < 8; ++u) {
        v4u* unit = reinterpret_cast<v4u*>(st + (r * 8 + dl_slot(r, u, 8)) * 16);  // (BP rows of P, then Q's)
        v4u x = {0, 0, 0, 0};
        const int keep = left - 16 * u;
        if (keep > 0) {
          x = *unit;
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            const int n = keep - 4 * d;
            x[d] = n >= 4 ? x[d] : n <= 0 ? 0u : x[d] & ((1u << (8 * n)) - 1u);
          }
        }
        *unit = x;
      }
    }
  }
  __device__ __forceinline__ void next(const ScaledArgs& a) {
    if (c + 1 < t.c_end) {
      ++c;
      left = min(kChunkBytes, a.k - c * kChunkBytes);
      p += kChunkBytes;
      q += kChunkBytes;
      sp += 4;
      sq += 4;
    } else if (w.at + w.step < w.end) {
      w.at += w.step;
      enter(a);
    }
  }
};

// Rows of C (or of a part's partial sums) from the accumulators, through the slab as O.
template <class S, typename O, typename C>
__device__ __forceinline__ void scaled_put(C* c, int64_t ldc, const ScaledTile<S>& t, bool vec, bool accumulate, int wp, int wq,
                                           int lane, unsigned char* slab, const v4f (&acc)[S::RB][S::CB]) {
  using W = Slab<O, 16>;
  constexpr int RP = S::RB < W::COLS / 16 ? S::RB : W::COLS / 16;
#pragma unroll
  for (int cb = 0; cb < S::CB; ++cb) {
    const int q = wq * (S::BQ / S::WQ) + cb * 16;
#pragma unroll
    for (int r0 = 0; r0 < S::RB; r0 += RP) {
      const int p = wp * (S::BP / S::WP) + r0 * 16;
#pragma unroll
      for (int rb = 0; rb < RP; ++rb) {
        const v4f& x = acc[r0 + rb][cb];
        const float v[4] = {x[0], x[1], x[2], x[3]};
        W::put4(slab, lane & 15, rb * 16 + 4 * (lane >> 4), v);
      }
      W::fence();
      W::store(slab, c + (t.q0 + q) * ldc + t.p0 + p, ldc, t.qv - q, min(t.pv - p, RP * 16), vec, accumulate, lane);
      W::fence();
    }
  }
}

// C in tiles, a workgroup's tiles one after another as one stream of chunks of
// 128 steps through two stages of LDS: the next chunk (the next tile's first,
// at a tile's end) is copied under this one's products, as soon as its stage is
// free.  Every block of 16 x 16 results is scaled and added one step behind its
// product, so that the vector units work under the next products.  The barrier
// of the next chunk comes before a chunk's last step, whose fragments are in
// registers by then; Q's fragments of the next chunk are read as the last
// products release them.  ADD: a 16-bit C is added to (a kernel of its own: with both
// in one the 256 x 256 tile's registers do not do).
template <class S, int QF, bool PVEC, bool WIDE, bool ADD>
__global__ __launch_bounds__(S::THREADS, S::WAVES_PER_SIMD) void scaled_tile_kernel(const ScaledArgs a) {
  extern __shared__ __align__(256) unsigned char lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tiles = ((a.n + S::BP - 1) / S::BP) * (int)((a.m + S::BQ - 1) / S::BQ) * a.splits;
  Walk w(tiles);
  if (w.at >= w.end) return;
  const int wp = wave / S::WQ, wq = wave % S::WQ;
  const int prow = wp * (S::BP / S::WP), qrow = wq * (S::BQ / S::WQ);
  unsigned char* slab = lds + S::SLABS + wave * Slab<float, 16>::BYTES;
  using FP = Frag8<WIDE, 0>;
  using FQ = Frag8<WIDE, QF>;
  v8i raw;                    // P's fragment of the next step
  typename FQ::type fq[S::CB];
  float sc[S::CB], sc_old[S::CB];  // Q's scales (times P's in the square form) of this chunk and the last one
  f4 sr, sr_old;                   // P's scales of a step's four rows (vector form), and the step's before
  int g = 0;                       // chunk of the stream, in stage g & 1
  auto read_q = [&](const unsigned char* st, int cb) { return FQ::of(frag8(st + S::P_BYTES, qrow + cb * 16, lane)); };
  auto read_scales = [&](const unsigned char* st) {
    const float* sp = reinterpret_cast<const float*>(st + S::SP);
    const float* sq = reinterpret_cast<const float*>(st + S::SQ);
#pragma unroll
    for (int cb = 0; cb < S::CB; ++cb) sc[cb] = sq[qrow + cb * 16 + (lane & 15)];
    if (!PVEC) {
      const float s = sp[prow];  // the wave's rows of P lie in one square
#pragma unroll
      for (int cb = 0; cb < S::CB; ++cb) {
        sc[cb] *= s;
      }
    }
  };
  auto read_sr = [&](const unsigned char* st, int rb) {
    if (PVEC) sr = *reinterpret_cast<const f4*>(st + S::SP + (prow + rb * 16 + 4 * (lane >> 4)) * 4);
  };
  ScaledFeed<S> feed(a, w, wave, lane);
  auto land = [&] {  // the chunk being copied is in LDS; every wave has read the one before
    stage_barrier();
    if (feed.left < kChunkBytes) {
      feed.clear_end();
      stage_barrier();
    }
  };
  feed.copy(a, lds, wave, lane);
  land();
  feed.next(a);
  feed.copy(a, lds + S::STAGE, wave, lane);
#pragma unroll
  for (int cb = 0; cb < S::CB; ++cb) fq[cb] = read_q(lds, cb);
  raw = frag8(lds, prow, lane);
  read_scales(lds);
  for (; w.at < w.end; w.at += w.step) {
    ScaledTile<S> t;
    t.load(a, w.at);
    v4f acc[S::RB][S::CB], d[S::CB];
#pragma unroll
    for (int rb = 0; rb < S::RB; ++rb)
#pragma unroll
      for (int cb = 0; cb < S::CB; ++cb) acc[rb][cb] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int cb = 0; cb < S::CB; ++cb) {
      d[cb] = {0.f, 0.f, 0.f, 0.f};
      sc_old[cb] = 0.f;
    }
    sr = {0.f, 0.f, 0.f, 0.f};
    auto add = [&](int rb, int cb, float q, const f4& r) {
#pragma unroll
      for (int v = 0; v < 4; ++v)
        acc[rb][cb][v] = PVEC ? fmaf(d[cb][v] * q, r[v], acc[rb][cb][v]) : fmaf(d[cb][v], q, acc[rb][cb][v]);
      // done here: left free, the compiler gathers the additions behind all products, with all of
      // their results in registers
      asm volatile("" : "+v"(acc[rb][cb]));
    };
    // A chunk some of whose scales' products are no normal numbers: sums whose scales are taken in turn
    // are added here, and nothing for them by the common way.  Q's fragments are in registers, P's come from
    // LDS again.  Between the first step and the second, after the sums of all chunks before.
    auto take_in_turn = [&](const unsigned char* st) {
      // zero rows have the smallest scales: nothing to do for them, unless the product is infinite (a tenth of
      // the rows zero in e5m2, 1024 x 8192 x 8192: 87 us for 79 without such rows; with the scales first, 94)
      bool any = false;
#pragma unroll
      for (int cb = 0; cb < S::CB; ++cb)
        any |= !__builtin_amdgcn_classf(sc[cb], 0x108) && (holds_values(fq[cb]) || __builtin_isinf(sc[cb]));
      if (__ballot(any) == 0) return;
      int l;  // the lane, worked out here: the loops leave no register for what this needs
      asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(l));
      const float* sq = reinterpret_cast<const float*>(st + S::SQ) + qrow + (l & 15);
      const float s = reinterpret_cast<const float*>(st + S::SP)[prow];
#pragma unroll
      for (int cb = 0; cb < S::CB; ++cb)
        if (BothScales(sq[cb * 16], s).in_turn) sc[cb] = 0.f;
#pragma unroll
      for (int cb = 0; cb < S::CB; ++cb) add(0, cb, sc[cb], sr);
#pragma unroll
      for (int rb = 0; rb < S::RB; ++rb) {
        const typename FP::type fp = FP::of(frag8(st, prow + rb * 16, lane));
#pragma unroll
        for (int cb = 0; cb < S::CB; ++cb) {
          const typename FQ::type one[1] = {fq[cb]};
          v4f x[1];
          products<QF>(fp, one, x);
          const BothScales w(sq[cb * 16], s);
          if (w.in_turn) {
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[rb][cb][v] = w.add(x[0][v], acc[rb][cb][v]);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
#pragma unroll
      for (int cb = 0; cb < S::CB; ++cb) d[cb] = {0.f, 0.f, 0.f, 0.f};
      raw = frag8(st, prow + 16, lane);
    };
    for (int c = t.c_begin; c < t.c_end; ++c) {
      unsigned char* st = lds + (g & 1) * S::STAGE;
      const unsigned char* other = lds + ((g + 1) & 1) * S::STAGE;
#pragma unroll
      for (int rb = 0; rb < S::RB; ++rb) {
        const bool last = rb + 1 == S::RB;
        const typename FP::type fp = FP::of(raw);
        sr_old = sr;
        read_sr(st, rb);
        if (last) {
          land();
          raw = frag8(other, prow, lane);  // (past the stream's end: stale bytes that nothing uses)
          // this chunk's stage is free at once: the chunk after the next goes there
          feed.next(a);
          feed.copy(a, st, wave, lane);
        } else {
          raw = frag8(st, prow + (rb + 1) * 16, lane);
        }
        if constexpr (WIDE) {
#pragma unroll
          for (int cb = 0; cb < S::CB; ++cb) add(rb == 0 ? S::RB - 1 : rb - 1, cb, rb == 0 ? sc_old[cb] : sc[cb], sr_old);
          products<QF>(fp, fq, d);
          if (last) {
#pragma unroll
            for (int cb = 0; cb < S::CB; ++cb) fq[cb] = read_q(other, cb);
          }
        } else {
#pragma unroll
          for (int cb = 0; cb < S::CB; ++cb) {
            add(rb == 0 ? S::RB - 1 : rb - 1, cb, rb == 0 ? sc_old[cb] : sc[cb], sr_old);
            d[cb] = mfma8<QF>(fp, fq[cb]);
            if (last) fq[cb] = read_q(other, cb);
            __builtin_amdgcn_sched_barrier(0);  // keep the order: it bounds the registers
          }
        }
        if (last) {
#pragma unroll
          for (int cb = 0; cb < S::CB; ++cb) sc_old[cb] = sc[cb];
          read_scales(other);
        }
        if (!PVEC && rb == 0) {
          // one comparison for all (magnitudes below the first normal number wrap).  16384 x 8192 x 2048, 1024 x
          // 8192 x 8192 to bf16: 289, 80 us; 286, 79 without it; 311, 92 with the scales in turn for every sum
          uint32_t most = 0;
#pragma unroll
          for (int cb = 0; cb < S::CB; ++cb) most = umax(most, 2 * __float_as_uint(sc[cb]) - 0x01000000u);
          if (__builtin_expect(__ballot(most >= 0xfe000000u) != 0, 0)) take_in_turn(st);
        }
      }
      ++g;
    }
#pragma unroll
    for (int cb = 0; cb < S::CB; ++cb) add(S::RB - 1, cb, sc_old[cb], sr);
    if (S::BP == 128 && a.partial)  // only the small tiles split the contraction
      scaled_put<S, float>(a.partial + (int64_t)t.part * a.m * a.n, (int64_t)a.n, t, a.n % 4 == 0, false, wp, wq, lane, slab, acc);
    else if constexpr (WIDE)
      scaled_put<S, float>(reinterpret_cast<float*>(a.c), a.ldc, t, a.vec_c, a.accumulate, wp, wq, lane, slab, acc);
    else if (a.c_type == MR_F16)
      scaled_put<S, std::conditional_t<ADD, float, _Float16>>(reinterpret_cast<_Float16*>(a.c), a.ldc, t, a.vec_c, ADD, wp, wq, lane, slab, acc);
    else
      scaled_put<S, std::conditional_t<ADD, float, bf16_t>>(reinterpret_cast<bf16_t*>(a.c), a.ldc, t, a.vec_c, ADD, wp, wq, lane, slab, acc);
  }
  wait_vmcnt<0>();  // the surplus copies of the last chunk: LDS is given back after them
}

// The general form, for operands whose rows are not whole 16-byte units: tiles
// of 128 x 128, every element of an operand checked, one stage, no overlap.
// Products and sums in the order of the form above.
template <int QF, bool PVEC, bool WIDE>
__global__ __launch_bounds__(256) void scaled_edge_kernel(const ScaledArgs a) {
  using S = ScaledShape<128, 128, 2, 2, 1>;
  extern __shared__ __align__(256) unsigned char lds[];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wp = wave / S::WQ, wq = wave % S::WQ;
  const int prow = wp * 64, qrow = wq * 64;
  ScaledTile<S> t;
  t.load(a, blockIdx.x);
  v4f acc[S::RB][S::CB];
#pragma unroll
  for (int rb = 0; rb < S::RB; ++rb)
#pragma unroll
    for (int cb = 0; cb < S::CB; ++cb) acc[rb][cb] = {0.f, 0.f, 0.f, 0.f};
  for (int c = t.c_begin; c < t.c_end; ++c) {
    const int64_t k0 = (int64_t)c * kChunkBytes;
    const int left = (int)min((int64_t)kChunkBytes, a.k - k0);
    __syncthreads();
    EdgeAlong<S::BP, S::THREADS, 1, 8> ep;
    EdgeAlong<S::BQ, S::THREADS, 1, 8> eq;
    ep.load(a.p, a.ldp, t.p0, t.pv, k0, left, threadIdx.x);
    eq.load(a.q, a.ldq, t.q0, t.qv, k0, left, threadIdx.x);
    ep.store(lds, threadIdx.x);
    eq.store(lds + S::P_BYTES, threadIdx.x);
    __syncthreads();
    typename Frag8<WIDE, QF>::type fq[S::CB];
    float sc[S::CB];
#pragma unroll
    for (int cb = 0; cb < S::CB; ++cb) {
      fq[cb] = Frag8<WIDE, QF>::of(frag8(lds + S::P_BYTES, qrow + cb * 16, lane));
      const int64_t r = t.q0 + min(qrow + cb * 16 + (lane & 15), t.qv - 1);
      sc[cb] = a.sq[(r >> a.q_shift) * a.ldsq + c];
    }
#pragma unroll
    for (int rb = 0; rb < S::RB; ++rb) {
      v4f d[S::CB];
      const typename Frag8<WIDE, 0>::type fp = Frag8<WIDE, 0>::of(frag8(lds, prow + rb * 16, lane));
      products<QF>(fp, fq, d);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int r = t.p0 + min(prow + rb * 16 + 4 * (lane >> 4) + v, t.pv - 1);
        const float s = a.sp[(int64_t)(r >> a.p_shift) * a.ldsp + c];
#pragma unroll
        for (int cb = 0; cb < S::CB; ++cb)
          acc[rb][cb][v] = PVEC ? fmaf(d[cb][v] * sc[cb], s, acc[rb][cb][v]) : BothScales(sc[cb], s).add(d[cb][v], acc[rb][cb][v]);
      }
    }
  }
  unsigned char* slab = lds + S::P_BYTES + S::Q_BYTES + wave * Slab<float, 16>::BYTES;
  auto put = [&](auto* c) {
    using C = std::remove_pointer_t<decltype(c)>;
    if (a.accumulate)
      scaled_put<S, float>(c, a.ldc, t, a.vec_c, true, wp, wq, lane, slab, acc);
    else
      scaled_put<S, C>(c, a.ldc, t, a.vec_c, false, wp, wq, lane, slab, acc);
  };
  if (a.partial)
    scaled_put<S, float>(a.partial + (int64_t)t.part * a.m * a.n, (int64_t)a.n, t, a.n % 4 == 0, false, wp, wq, lane, slab, acc);
  else if constexpr (WIDE)
    put(reinterpret_cast<float*>(a.c));
  else if (a.c_type == MR_F16)
    put(reinterpret_cast<_Float16*>(a.c));
  else
    put(reinterpret_cast<bf16_t*>(a.c));
}

// Few rows of C (m <= 16 CB): no tile in LDS.  A workgroup of NW waves owns 16
// RB rows of P (columns of C); wave w takes the chunks of 128 steps w, w + NW,
// ..., straight from global memory into the fragments (P's bytes are read once
// over the whole launch), and the waves' sums are added through LDS in wave
// order.  The bytes take the time, so every C is summed on fp16 instructions (in
// 8 bits the same: 8 x 4096 x 1024 3.5 us, 64 x 8192 x 2048 11.4; 48 x 8192 x 8192
// 28.3 for 29.6).
template <int CB, int RB, int NW, int QF, bool PVEC>
__global__ __launch_bounds__(64 * NW) void scaled_rows_kernel(const ScaledArgs a) {
  __shared__ v4f part[NW][RB][CB][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane >> 4, i = lane & 15;
  const int p0 = blockIdx.x * 16 * RB;
  const int chunks = (a.k + kChunkBytes - 1) / kChunkBytes;
  v4f acc[RB][CB];
#pragma unroll
  for (int rb = 0; rb < RB; ++rb)
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) acc[rb][cb] = {0.f, 0.f, 0.f, 0.f};
  auto chunk = [&](auto whole_units, int c) {
    auto frag = [&](const unsigned char* row) -> v8i {
      const int64_t k0 = (int64_t)c * kChunkBytes + 16 * g;
      if constexpr (decltype(whole_units)::value)
        return join(*reinterpret_cast<const v4i*>(row + k0), *reinterpret_cast<const v4i*>(row + k0 + 64));
      const int left = a.k - (int)k0;
      const v4u u = edge_unit<1>(row + k0, left), v = edge_unit<1>(row + k0 + 64, left - 64);
      return join(__builtin_bit_cast(v4i, u), __builtin_bit_cast(v4i, v));
    };
    typename Frag8<true, 0>::type fp[RB];
    float s[RB][PVEC ? 4 : 1];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      fp[rb] = Frag8<true, 0>::of(frag(a.p + (int64_t)min(p0 + rb * 16 + i, a.n - 1) * a.ldp));
      if (PVEC) {
#pragma unroll
        for (int v = 0; v < 4; ++v) s[rb][v] = a.sp[(int64_t)min(p0 + rb * 16 + 4 * g + v, a.n - 1) * a.ldsp + c];
      } else {
        s[rb][0] = a.sp[(int64_t)(min(p0 + rb * 16, a.n - 1) / kBlock) * a.ldsp + c];
      }
    }
    typename Frag8<true, QF>::type fq[CB];
    float sc[CB];
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) {
      const int64_t r = min((int64_t)(cb * 16 + i), a.m - 1);
      fq[cb] = Frag8<true, QF>::of(frag(a.q + r * a.ldq));
      sc[cb] = a.sq[(r >> a.q_shift) * a.ldsq + c];
    }
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      v4f d[CB];
      products<QF>(fp[rb], fq, d);
#pragma unroll
      for (int cb = 0; cb < CB; ++cb)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          acc[rb][cb][v] = PVEC ? fmaf(d[cb][v] * sc[cb], s[rb][v], acc[rb][cb][v])
                                : BothScales(sc[cb], s[rb][0]).add(d[cb][v], acc[rb][cb][v]);
    }
  };
  // whole chunks without a branch, so that the loads of several are in flight
  const int end = (int)((int64_t)chunks * (blockIdx.y + 1) / a.splits);
  const int whole = a.fast ? min(a.k / kChunkBytes, end) : 0;
  int c = (int)((int64_t)chunks * blockIdx.y / a.splits) + wave;
#pragma unroll 2
  for (; c < whole; c += NW) chunk(std::true_type{}, c);
  for (; c < end; c += NW) chunk(std::false_type{}, c);
#pragma unroll
  for (int rb = 0; rb < RB; ++rb)
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) part[wave][rb][cb][lane] = acc[rb][cb];
  __syncthreads();
  for (int b = wave; b < RB * CB; b += NW) {
    const int rb = b / CB, cb = b % CB;
    v4f t = part[0][rb][cb][lane];
#pragma unroll
    for (int w = 1; w < NW; ++w) t += part[w][rb][cb][lane];
    const int64_t r = cb * 16 + i;
    const int p = p0 + rb * 16 + 4 * g;
    if (r < a.m && p < a.n) {
      const float v[4] = {t[0], t[1], t[2], t[3]};
      if (a.partial)
        put4(a.partial + ((int64_t)blockIdx.y * a.m + r) * a.n + p, v, a.n - p, a.n % 4 == 0, false);
      else
        put4_as(a.c, r * a.ldc + p, v, a.n - p, a.c_type, a.vec_c, a.accumulate);
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

using TileLarge = ScaledShape<256, 256, 2, 4, 1>;  // 16-bit C
using TileWide = ScaledShape<256, 128, 4, 2, 1>;   // float32 C (fp16 fragments) or P's scales by row: more registers
using Tile128 = ScaledShape<128, 128, 2, 2, 2>;
constexpr int kFewRows = 64;
constexpr int kCus = 256;

template <class S, int QF, bool PVEC, bool WIDE, bool ADD>
hipError_t launch_tile(const ScaledArgs& a, hipStream_t s) {
  static std::atomic<uint64_t> raised{0};
  auto kernel = scaled_tile_kernel<S, QF, PVEC, WIDE, ADD>;
  if (hipError_t e = raise_lds(kernel, S::LDS, raised); e != hipSuccess) return e;
  const int64_t tiles = (int64_t)((a.n + S::BP - 1) / S::BP) * ((a.m + S::BQ - 1) / S::BQ) * a.splits;
  hipLaunchKernelGGL(kernel, dim3(persistent_blocks(tiles, S::BPC)), dim3(S::THREADS), S::LDS, s, a);
  return hipGetLastError();
}

template <class S, int QF, bool PVEC, bool WIDE>
hipError_t go_tile(const ScaledArgs& a, hipStream_t s) {
  if constexpr (!WIDE) {
    if (a.accumulate && !a.partial) return launch_tile<S, QF, PVEC, WIDE, true>(a, s);
  }
  return launch_tile<S, QF, PVEC, WIDE, false>(a, s);
}

template <int QF, bool PVEC, bool WIDE>
hipError_t go_edge(const ScaledArgs& a, hipStream_t s) {
  const int64_t tiles = (int64_t)((a.n + 127) / 128) * ((a.m + 127) / 128) * a.splits;
  constexpr int bytes = 256 * kChunkBytes + 4 * Slab<float, 16>::BYTES;
  hipLaunchKernelGGL((scaled_edge_kernel<QF, PVEC, WIDE>), dim3((unsigned)tiles), dim3(256), bytes, s, a);
  return hipGetLastError();
}

template <int CB, int RB, int NW, int QF, bool PVEC>
hipError_t go_rows(const ScaledArgs& a, hipStream_t s) {
  const dim3 grid((a.n + 16 * RB - 1) / (16 * RB), a.splits);
  hipLaunchKernelGGL((scaled_rows_kernel<CB, RB, NW, QF, PVEC>), grid, dim3(64 * NW), 0, s, a);
  return hipGetLastError();
}

template <int QF, bool PVEC, bool WIDE>
hipError_t go_kind(const ScaledArgs& a, int kind, hipStream_t s) {
  if (kind >= 1 && !a.fast) return go_edge<QF, PVEC, WIDE>(a, s);
  if (kind == 2) return go_tile<std::conditional_t<WIDE || PVEC, TileWide, TileLarge>, QF, PVEC, WIDE>(a, s);
  if (kind >= 1) return go_tile<Tile128, QF, PVEC, WIDE>(a, s);
  if (a.m <= 16) {
    // long contractions under few columns: twice the waves, for bytes in flight
    if (a.n <= 16 * kCus && a.k / a.splits >= 16 * kChunkBytes) return go_rows<1, 1, 16, QF, PVEC>(a, s);
    return go_rows<1, 1, 8, QF, PVEC>(a, s);
  }
  // 32 columns to a workgroup halve what is read of A, where enough workgroups are left (64 x 8192 x
  // 2048: 11.5 us for 15.8; 32 x 4096 x 4096: 12.7 for 10.6)
  const bool wide = a.n >= 32 * kCus;
  if (a.m <= 32) return wide ? go_rows<2, 2, 8, QF, PVEC>(a, s) : go_rows<2, 1, 8, QF, PVEC>(a, s);
  return wide ? go_rows<4, 2, 8, QF, PVEC>(a, s) : go_rows<4, 1, 8, QF, PVEC>(a, s);
}

template <int QF, bool PVEC>
hipError_t go_width(const ScaledArgs& a, int kind, hipStream_t s) {
  return a.c_type == MR_F32 ? go_kind<QF, PVEC, true>(a, kind, s) : go_kind<QF, PVEC, false>(a, kind, s);
}

}  // namespace

// Up to 64 rows the weights' bytes are all there is to it: no tile (64 x 8192 x
// 2048: 11.4 us, 17.3 in tiles), the contraction split where the columns leave CUs
// without work (16 x 1024 x 16384: 11.2 us, 20.3 whole).  256 x 256 tiles once they fill the CUs; below that 128 x 128
// ones (1024 x 8192 x 8192: 87 us, 110 with large tiles), and a long contraction
// split while the tiles leave half of the CUs without work (128 x 1024 x 16384: 25
// us, 94 whole; 2048^3, whose 256 tiles do not: 19 whole, 33 in two parts).
ScaledPlan scaled_plan(int64_t m, int64_t n, int64_t k) {
  const int64_t chunks = (k + kChunkBytes - 1) / kChunkBytes;
  if (m <= kFewRows) {
    int splits = 1;
    while (splits < 16 && (n + 15) / 16 * splits * 2 <= kCus && chunks / (splits * 2) >= 32) splits *= 2;
    return {0, splits};
  }
  auto tiles = [&](int p, int q) { return ((m + q - 1) / q) * ((n + p - 1) / p); };
  if (tiles(256, 256) >= kCus) return {2, 1};
  const int64_t t = tiles(128, 128);
  int64_t splits = 1;
  while (splits < 16 && t * splits * 2 <= kCus && chunks / (splits * 2) >= 8) splits *= 2;
  return {1, (int)splits};
}

hipError_t launch_scaled(const ScaledArgs& a, const ScaledPlan& plan, hipStream_t s) {
  const bool p_vector = a.p_shift == 0;
  if (a.q_e5m2) return p_vector ? go_width<1, true>(a, plan.kind, s) : go_width<1, false>(a, plan.kind, s);
  return p_vector ? go_width<0, true>(a, plan.kind, s) : go_width<0, false>(a, plan.kind, s);
}

hipError_t launch_scaled_join(const ScaledArgs& a, hipStream_t s) {
  const int64_t quads = a.m * ((a.n + 3) / 4);
  const int64_t blocks = (quads + 255) / 256;
  hipLaunchKernelGGL(scaled_join_kernel, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace mr
