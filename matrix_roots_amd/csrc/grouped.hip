// Products of rows grouped by expert (ragged groups, offsets read on the
// device), 16-bit operands, float32 sums on v_mfma_f32_32x32x16:
//
//   forward    y_r = W_e x_r      P = W_e (along k),        Q = x (along k)
//   transpose  y_r = W_e^T x_r    P = W_e^T (across n),     Q = x (along n)
//   weights    DW_e = sum_r dy_r x_r^T
//                                 P = dy (across rows),     Q = x (across rows)
//
// P is the matrix instruction's row operand: a lane holds four consecutive
// rows of P at one row of Q.  Operands whose contraction is not contiguous in
// memory ("across") go through ds_read_b64_tr_b16, which hands each lane four
// steps of one column; no transposed copy of a weight is ever made.
//
// Row tiles never span two experts.  A launch has the
// workgroups that the CUs hold at a time; each finds its tiles from the offsets
// (one wave scan over the experts), so no size reaches the host and the call
// can be captured and replayed under other sizes.
//
// What bounds it: the experts' weights (their gradients in float32) come from
// and go to HBM, and with a few hundred rows per expert that outweighs the
// products.  So a workgroup's tiles are one stream of chunks: four loader waves
// copy two chunks ahead, straight to LDS and on into the next tile, and the
// other four waves never wait for memory.  64 uneven experts, 16384 rows, n =
// 2048, k = 1536, bf16, one MI355X: forward 147 us (520 MB: 3.5 TB/s), rows'
// gradient 148 us, weights' gradient behind it 210 us (0.92 GB: 4.4 TB/s; 218 with
// nothing in the caches); 16 rows 16 us.
// One workgroup per tile with its own copies took 214, 254 and 440 us.
#include <type_traits>

#include "tile_core.hpp"

namespace mr {

namespace {

typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) v4s* lds_v4s;

__device__ __forceinline__ void store_once(float v, float* p) { __builtin_nontemporal_store(v, p); }
__device__ __forceinline__ void store_once(_Float16 v, _Float16* p) { __builtin_nontemporal_store(v, p); }
__device__ __forceinline__ void store_once(bf16_t v, bf16_t* p) { __builtin_nontemporal_store(v.bits, &p->bits); }

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
template <int R, int UPK, bool ACROSS>
__device__ __forceinline__ v8s frag16(const unsigned char* st, int row, int ks, int lane) {
  if constexpr (!ACROSS) {
    // (row is a multiple of 32: the slot depends on the lane alone)
    const int r = lane & 31;
    return *reinterpret_cast<const v8s*>(st + row * UPK * 16 + (r * UPK + dl_slot(r, 2 * ks + (lane >> 5), UPK)) * 16);
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
// Rows of expert e (none where the offsets decrease).
__device__ __forceinline__ void expert_rows(const GroupedArgs& a, int e, int64_t& begin, int64_t& end) {
  begin = offset_at(a, e);
  end = offset_at(a, e + 1);
  if (end < begin) end = begin;
}

// The experts' row tiles, BQ rows to a tile and `across` column tiles to a row
// tile: each lane counts a run of experts, one scan gives every wave the total
// and the means to find a tile.
template <int BQ>
struct RowTiles {
  int per, mine, sum, total, across;
  __device__ __forceinline__ int of(const GroupedArgs& a, int e) const {
    if (e >= a.experts) return 0;
    int64_t b, t;
    expert_rows(a, e, b, t);
    return (int)((t - b + BQ - 1) / BQ) * across;  // all tiles fit a grid
  }
  __device__ __forceinline__ void count(const GroupedArgs& a, int across_) {
    const int lane = threadIdx.x & 63;
    across = across_;
    per = (a.experts + 63) / 64;
    mine = 0;
    for (int i = 0; i < per; ++i) mine += of(a, lane * per + i);
    sum = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int up = __shfl_up(sum, d);
      if (lane >= d) sum += up;
    }
    total = __builtin_amdgcn_readlane(sum, 63);
  }
  // Expert of tile `id` < total, its rows, and the tile's place among its tiles.
  __device__ __forceinline__ void find(const GroupedArgs& a, int id, int& e, int64_t& begin, int64_t& end, int& local) const {
    const uint64_t hit = __ballot(id < sum);
    const int l = hit ? __builtin_ctzll(hit) : 63;
    local = id - (__builtin_amdgcn_readlane(sum, l) - __builtin_amdgcn_readlane(mine, l));
    e = l * per;
    for (int i = 1; i < per; ++i) {
      const int t = of(a, e);
      if (local < t) break;
      local -= t;
      ++e;
    }
    e = min(e, a.experts - 1);
    expert_rows(a, e, begin, end);
  }
};

// The weights' gradients' tiles, `tiles` to an expert, shared out to the XCDs by
// what they cost: an expert's tile takes its chunks of BK rows and, for its
// stores, what kStoreChunks chunks take.  Contiguous runs of equal cost keep an
// expert's operands in one or two L2s (runs of equal length: 300 us with uneven
// experts where even ones took 214).
constexpr int kStoreChunks = 5;
template <int BK>
__device__ __forceinline__ Walk share_experts(const GroupedArgs& a, int tiles) {
  const int lane = threadIdx.x & 63, per = (a.experts + 63) / 64;
  auto cost = [&](int e) -> int64_t {
    if (e >= a.experts) return 0;
    int64_t b, t;
    expert_rows(a, e, b, t);
    return (t - b + BK - 1) / BK + kStoreChunks;
  };
  int64_t mine = 0;
  for (int i = 0; i < per; ++i) mine += cost(lane * per + i);
  int64_t sum = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int64_t up = __shfl_up(sum, d);
    if (lane >= d) sum += up;
  }
  const int64_t total = __shfl(sum, 63);
  // first tile of XCD x: the tiles before it cost x / 8 of all
  auto first = [&](int x) {
    if (x >= kNumXcd) return a.experts * tiles;
    int64_t left = total * tiles * x / kNumXcd;  // (in units of one tile's cost)
    const uint64_t hit = __ballot(left < sum * tiles);
    const int l = hit ? __builtin_ctzll(hit) : 63;
    left -= (__shfl(sum, l) - __shfl(mine, l)) * tiles;
    int e = l * per;
    for (int i = 1; i < per && left >= cost(e) * tiles; ++i) {
      left -= cost(e) * tiles;
      ++e;
    }
    e = min(e, a.experts - 1);
    return e * tiles + (int)min(left / max(cost(e), (int64_t)1), (int64_t)tiles);
  };
  const int x = blockIdx.x % kNumXcd;
  return Walk(first(x), first(x + 1));
}

}  // namespace

// WP x WQ waves multiply, kLoaders waves copy.  NST stages of BK steps in LDS;
// BPC workgroups to a CU.
template <int BP_, int BQ_, int WP_, int WQ_, int BK_, int NST_, int BPC_>
struct GroupedShape {
  static constexpr int BP = BP_, BQ = BQ_, WP = WP_, WQ = WQ_, NW = WP * WQ, BK = BK_, NST = NST_, BPC = BPC_;
  static constexpr int THREADS = 64 * (NW + kLoaders);
  static constexpr int RB = BP / WP / 32, CB = BQ / WQ / 32, KS = BK / 16;
  static constexpr int P_BYTES = BP * BK * 2, STAGE = (BP + BQ) * BK * 2;
  static constexpr int COPIES = STAGE / 1024 / kLoaders;  // direct copies per loader wave and chunk
  static constexpr int SLABS = NST * STAGE;               // where the waves' output slabs start
  static constexpr int LDS = SLABS + NW * Slab<float, 32>::BYTES;
  static constexpr int WAVES_PER_SIMD = (BPC * (NW + kLoaders) + 3) / 4;
  static_assert(KS % 2 == 0 && BPC * LDS <= 160 * 1024, "fragments alternate; the stages fit");
};

// One operand of a tile: rows (products' rows) r0 .. of `valid`, bytes.
struct Operand {
  const unsigned char* base;
  int64_t ld_bytes, r0;
  int valid;
};

// One operand's part of a chunk by direct copies of the loader waves.
template <class S, int R, bool ACROSS>
__device__ __forceinline__ void copy_operand(const Operand& o, int64_t k0, int left, unsigned char* st, int loader, int lane) {
  if constexpr (ACROSS)
    copy_across<R, kLoaders, S::BK>(o.base, o.ld_bytes, k0, left, o.r0, o.valid, st, loader, lane);
  else
    copy_along<R, kLoaders, S::BK / 8>(o.base, o.ld_bytes, o.r0, o.valid, k0 * 2, (left + 7) / 8, st, loader, lane);
}
// ... and through their registers.
template <class S, int R, bool ACROSS>
struct EdgeOperand {
  std::conditional_t<ACROSS, EdgeAcross<R, 64 * kLoaders, S::BK>, EdgeAlong<R, 64 * kLoaders, 2, S::BK / 8>> e;
  __device__ __forceinline__ void load(const Operand& o, int64_t k0, int left, int thread) {
    if constexpr (ACROSS)
      e.load(o.base, o.ld_bytes, k0, left, o.r0, o.valid, thread);
    else
      e.load(o.base, o.ld_bytes, o.r0, o.valid, k0 * 2, left, thread);
  }
};

template <class S>
struct Frags {
  v8s p[S::RB], q[S::CB];
};
template <class S, bool PA, bool QA>
__device__ __forceinline__ void read_frags(const unsigned char* st, int ks, int wp, int wq, int lane, Frags<S>& f) {
#pragma unroll
  for (int rb = 0; rb < S::RB; ++rb) f.p[rb] = frag16<S::BP, S::BK / 8, PA>(st, wp * (S::BP / S::WP) + rb * 32, ks, lane);
#pragma unroll
  for (int cb = 0; cb < S::CB; ++cb)
    f.q[cb] = frag16<S::BQ, S::BK / 8, QA>(st + S::P_BYTES, wq * (S::BQ / S::WQ) + cb * 32, ks, lane);
}

// Instruction order of one step: the next step's fragment reads spread over this
// step's products, first reads first (left alone, the compiler moves every read
// down to its use and the wave waits for LDS at each step).
template <class S, bool PA, bool QA>
__device__ __forceinline__ void spread_reads() {
  constexpr int NR = S::RB * (PA ? 2 : 1) + S::CB * (QA ? 2 : 1), NM = S::RB * S::CB;
  constexpr int PER = (NR + NM - 1) / NM, FULL = NR / PER, REST = NR % PER;  // PER reads before each product
  static_for<FULL>([](auto) {
    __builtin_amdgcn_sched_group_barrier(0x100, PER, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
  });
  if constexpr (REST > 0) __builtin_amdgcn_sched_group_barrier(0x100, REST, 0);
  if constexpr (NM > FULL) __builtin_amdgcn_sched_group_barrier(0x008, NM - FULL, 0);
}

// Steps past `left` of a fragment (steps 16 ks + 8 (lane / 32) ..) set to zero.
__device__ __forceinline__ v8s mask_steps(v8s x, int left) {
  v4u u = __builtin_bit_cast(v4u, x);
#pragma unroll
  for (int d = 0; d < 4; ++d) u[d] = left <= 2 * d ? 0u : left == 2 * d + 1 ? u[d] & 0xffffu : u[d];
  return __builtin_bit_cast(v8s, u);
}

// One tile's operands and contraction.
template <class S>
struct Tile {
  Operand P, Q;
  int64_t steps;
  int chunks;
  int e, p0, pv, qv;
  int64_t q0;
  __device__ __forceinline__ void ready(int64_t n) {
    steps = n;
    chunks = (int)((n + S::BK - 1) / S::BK);
  }
};

// The loader waves' side of stream_tiles.  FAST: every operand by whole 16-byte
// units at 16-byte addresses; else through registers, one chunk's loads ahead.
template <class S, bool PA, bool QA, bool FAST, class Load>
__device__ __forceinline__ void copy_stream(Walk w, unsigned char* lds, Load&& load, int loader, int lane) {
  Tile<S> t;
  t.chunks = 0;
  int c = 0;  // next chunk of t
  auto more = [&] {
    while (c == t.chunks) {
      if (w.at >= w.end) return false;
      load(t, w.at);
      w.at += w.step;
      c = 0;
    }
    return true;
  };
  if constexpr (FAST) {
    copy_chunks<S::NST, true, S::COPIES>([&](int j) {
      if (!more()) return false;
      unsigned char* st = lds + j % S::NST * S::STAGE;
      const int64_t k0 = (int64_t)c * S::BK;
      const int left = (int)min((int64_t)S::BK, t.steps - k0);
      copy_operand<S, S::BP, PA>(t.P, k0, left, st, loader, lane);
      copy_operand<S, S::BQ, QA>(t.Q, k0, left, st + S::P_BYTES, loader, lane);
      ++c;
      return true;
    });
  } else {
    const int thread = loader * 64 + lane;
    EdgeOperand<S, S::BP, PA> p;
    EdgeOperand<S, S::BQ, QA> q;
    bool held = false;
    auto fetch = [&] {
      held = more();
      if (!held) return;
      const int64_t k0 = (int64_t)c * S::BK;
      const int left = (int)min((int64_t)S::BK, t.steps - k0);
      p.load(t.P, k0, left, thread);
      q.load(t.Q, k0, left, thread);
      ++c;
    };
    fetch();
    copy_chunks<S::NST, false, 0>([&](int j) {
      if (!held) return false;
      unsigned char* st = lds + j % S::NST * S::STAGE;
      p.e.store(st, thread);
      q.e.store(st + S::P_BYTES, thread);
      fetch();
      return true;
    });
  }
}

// A workgroup's tiles, one after another, as one stream of chunks through NST
// stages of LDS.  The loader waves copy, up to NST - 1 chunks ahead and into the
// next tile; the other waves multiply and store.  Only the loaders ever wait for
// memory, so stores drain behind the next tile's products, and copies cover
// each other's latency.  One barrier per chunk, before its predecessor's last
// step of products, whose fragments are in registers by then; one more at the
// end of the stream.  load(tile, id) describes tile `id`, put(tile, acc, slab)
// stores one.
template <class S, typename T, bool PA, bool QA, bool FAST, class Load, class Put>
__device__ __forceinline__ void stream_tiles(Walk w, unsigned char* lds, Load&& load, Put&& put) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (wave >= S::NW) {
    __builtin_amdgcn_s_setprio(3);  // copies first: their issue is what the other waves end up waiting for (3%)
    copy_stream<S, PA, QA, FAST>(w, lds, load, wave - S::NW, lane);
    return;
  }
  const int wp = wave / S::WQ, wq = wave % S::WQ;
  unsigned char* slab = lds + S::SLABS + wave * Slab<float, 32>::BYTES;
  Frags<S> f[2];
  int g = 0;  // chunk of the stream, in stage g % NST
  join_chunk();
  read_frags<S, PA, QA>(lds, 0, wp, wq, lane, f[0]);
  v16f acc[S::RB][S::CB];
  // the products of one chunk; `left` steps of it exist
  auto chunk = [&](auto tail, int left) {
    const unsigned char* st = lds + g % S::NST * S::STAGE;
#pragma unroll
    for (int ks = 0; ks < S::KS; ++ks) {
      if (ks + 1 < S::KS) {
        read_frags<S, PA, QA>(st, ks + 1, wp, wq, lane, f[(ks + 1) & 1]);
      } else {
        join_chunk();
        ++g;
        // (past the stream's last chunk these are stale bytes that nothing uses)
        read_frags<S, PA, QA>(lds + g % S::NST * S::STAGE, 0, wp, wq, lane, f[0]);
      }
      Frags<S>& x = f[ks & 1];
      if constexpr (decltype(tail)::value) {
        const int n = left - 16 * ks - 8 * (lane >> 5);
#pragma unroll
        for (int rb = 0; rb < S::RB; ++rb) x.p[rb] = mask_steps(x.p[rb], n);
#pragma unroll
        for (int cb = 0; cb < S::CB; ++cb) x.q[cb] = mask_steps(x.q[cb], n);
      }
#pragma unroll
      for (int rb = 0; rb < S::RB; ++rb)
#pragma unroll
        for (int cb = 0; cb < S::CB; ++cb) acc[rb][cb] = mfma16<T>(x.p[rb], x.q[cb], acc[rb][cb]);
      spread_reads<S, PA, QA>();
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  for (; w.at < w.end; w.at += w.step) {
    Tile<S> t;
    load(t, w.at);
#pragma unroll
    for (int rb = 0; rb < S::RB; ++rb)
#pragma unroll
      for (int cb = 0; cb < S::CB; ++cb)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[rb][cb][v] = 0.f;
    const int whole = (int)(t.steps / S::BK), left = (int)(t.steps % S::BK);
    for (int c = 0; c < whole; ++c) chunk(std::false_type{}, S::BK);
    if (left) chunk(std::true_type{}, left);
    put(t, acc, slab);
  }
}

// Rows q0 .. of Y from the accumulators, 32 rows of the wave at a time through
// its part of LDS (a lane holds four consecutive columns of one row).  The
// lines of a 128-column bf16 tile then leave whole: 25 us less of 181 (64
// experts, 16384 x 2048 outputs).
template <class S, typename O>
__device__ __forceinline__ void put_rows(const GroupedArgs& a, int64_t q0, int qv, int p0, int pv, unsigned char* slab,
                                         const v16f (&acc)[S::RB][S::CB]) {
  using W = Slab<O, 32>;
  constexpr int RP = S::RB < W::COLS / 32 ? S::RB : W::COLS / 32;  // blocks of 32 columns to a slab
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wp = wave / S::WQ, wq = wave % S::WQ;
#pragma unroll
  for (int cb = 0; cb < S::CB; ++cb) {
    const int q = wq * (S::BQ / S::WQ) + cb * 32;
#pragma unroll
    for (int r0 = 0; r0 < S::RB; r0 += RP) {
      const int p = wp * (S::BP / S::WP) + r0 * 32;
#pragma unroll
      for (int rb = 0; rb < RP; ++rb)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const v16f& x = acc[r0 + rb][cb];
          const float v[4] = {x[4 * u], x[4 * u + 1], x[4 * u + 2], x[4 * u + 3]};
          W::put4(slab, lane & 31, rb * 32 + 8 * u + 4 * (lane >> 5), v);
        }
      W::fence();
      W::store(slab, reinterpret_cast<O*>(a.y) + (q0 + q) * a.ldy + p0 + p, a.ldy, qv - q, min(pv - p, RP * 32), a.vec_y,
               false, lane);
      W::fence();
    }
  }
}

// A weight's gradient from the accumulators: P's rows are its rows, Q's its
// columns, so 32 lanes store 32 consecutive columns (a whole 128-byte line of
// float32) of one row.
template <class S, typename O>
__device__ __forceinline__ void put_weight(const GroupedArgs& a, O* w, int p0, int pv, int q0, int qv,
                                           const v16f (&acc)[S::RB][S::CB]) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wp = wave / S::WQ, wq = wave % S::WQ;
  const int p_left = pv - wp * (S::BP / S::WP), q_left = qv - wq * (S::BQ / S::WQ);
  if (p_left <= 0 || q_left <= 0) return;
  if (p_left >= S::BP / S::WP && q_left >= S::BQ / S::WQ && !a.accumulate) {
    // the wave's part is whole: scalar row addresses, one 32-bit lane offset (with the checks of the
    // general form below the stores took longer than the products); past the caches, which the
    // operands need (through them: 300 us for 270, before operands were read ahead)
    O* base = w + (int64_t)(p0 + wp * (S::BP / S::WP)) * a.ldy + q0 + wq * (S::BQ / S::WQ);
    const uint32_t off = (uint32_t)(4 * (lane >> 5)) * (uint32_t)a.ldy + (uint32_t)(lane & 31);
#pragma unroll
    for (int rb = 0; rb < S::RB; ++rb)
#pragma unroll
      for (int v = 0; v < 16; ++v) {
        O* row = base + (int64_t)(rb * 32 + 8 * (v >> 2) + (v & 3)) * a.ldy;
#pragma unroll
        for (int cb = 0; cb < S::CB; ++cb) store_once(narrow<O>(acc[rb][cb][v]), row + off + cb * 32);
      }
    return;
  }
#pragma unroll
  for (int rb = 0; rb < S::RB; ++rb)
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int pr = wp * (S::BP / S::WP) + rb * 32 + f32_row(lane, v);
      if (pr >= pv) continue;
      O* row = w + (int64_t)(p0 + pr) * a.ldy + q0;
#pragma unroll
      for (int cb = 0; cb < S::CB; ++cb) {
        const int qc = wq * (S::BQ / S::WQ) + cb * 32 + (lane & 31);
        if (qc >= qv) continue;
        const float x = a.accumulate ? acc[rb][cb][v] + widen(row[qc]) : acc[rb][cb][v];
        row[qc] = narrow<O>(x);
      }
    }
}

template <class S, typename T, bool TRANSPOSE, bool FAST>
__global__ __launch_bounds__(S::THREADS, S::WAVES_PER_SIMD) void grouped_tile_kernel(const GroupedArgs a) {
  extern __shared__ __align__(256) unsigned char lds[];
  const int outs = TRANSPOSE ? a.k : a.n, steps = TRANSPOSE ? a.n : a.k;
  RowTiles<S::BQ> tiles;
  tiles.count(a, (outs + S::BP - 1) / S::BP);
  auto load = [&](Tile<S>& t, int id) {
    int64_t begin, end;
    int local;
    tiles.find(a, id, t.e, begin, end, local);
    // an expert's row tiles follow one another under one panel of its weight
    // (offsets that decrease break the count: the bounds keep even those tiles inside the matrices)
    const int down = max((int)((end - begin + S::BQ - 1) / S::BQ), 1);
    t.p0 = min(max(local / down, 0), tiles.across - 1) * S::BP;
    t.q0 = begin + (int64_t)max(local % down, 0) * S::BQ;
    t.pv = min(S::BP, outs - t.p0);
    t.qv = (int)min((int64_t)S::BQ, end - t.q0);
    t.P = Operand{reinterpret_cast<const unsigned char*>(a.w) + t.e * a.w_stride * 2, a.ldw * 2, t.p0, t.pv};
    t.Q = Operand{reinterpret_cast<const unsigned char*>(a.x), a.ldx * 2, t.q0, t.qv};
    t.ready(t.qv > 0 ? steps : 0);
  };
  auto put = [&](const Tile<S>& t, const v16f(&acc)[S::RB][S::CB], unsigned char* slab) {
    if (a.y_f32)
      put_rows<S, float>(a, t.q0, t.qv, t.p0, t.pv, slab, acc);
    else
      put_rows<S, T>(a, t.q0, t.qv, t.p0, t.pv, slab, acc);
  };
  stream_tiles<S, T, TRANSPOSE, false, FAST>(Walk(tiles.total), lds, load, put);
  // rows of no expert: before the first and after the last offset
  const int64_t first = offset_at(a, 0), last = max(offset_at(a, a.experts), first);
  const int es = a.y_f32 ? 4 : 2;
  for (int64_t r = blockIdx.x; r < first + a.rows - last; r += gridDim.x) {
    char* row = reinterpret_cast<char*>(a.y) + (r < first ? r : r - first + last) * a.ldy * es;
    for (int c = threadIdx.x; c < outs; c += S::THREADS) {
      if (a.y_f32)
        reinterpret_cast<float*>(row)[c] = 0.f;
      else
        reinterpret_cast<uint16_t*>(row)[c] = 0;
    }
  }
}

// Where an expert's rows last a tile for a few chunks only, all CUs of an XCD wait
// for the same new rows at every expert, each time for a few lines: the operands
// are brought into the last-level cache at its full rate first.
// Reads rows first .. last - 1 of `units` 16-byte units once, the grid's waves a row
// at a time, for the caches' sake.
__device__ __forceinline__ void read_ahead(const void* base, int64_t ld_bytes, int64_t first, int64_t last, int units, int waves) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  uint4 all{0, 0, 0, 0};
  for (int64_t r = first + (int64_t)blockIdx.x * waves + wave; r < last; r += (int64_t)gridDim.x * waves) {
    const uint4* row = reinterpret_cast<const uint4*>(static_cast<const unsigned char*>(base) + r * ld_bytes);
#pragma unroll 4
    for (int u = lane; u < units; u += 64) {
      const uint4 x = row[u];
      all.x ^= x.x, all.y ^= x.y, all.z ^= x.z, all.w ^= x.w;
    }
  }
  asm volatile("" ::"v"(all.x), "v"(all.y), "v"(all.z), "v"(all.w));  // keeps the loads
}

template <class S, typename T, bool FAST>
__global__ __launch_bounds__(S::THREADS, S::WAVES_PER_SIMD) void grouped_weight_kernel(const GroupedArgs a) {
  extern __shared__ __align__(256) unsigned char lds[];
  const int tp = (a.n + S::BP - 1) / S::BP, tq = (a.k + S::BQ - 1) / S::BQ;
  auto load = [&](Tile<S>& t, int id) {
    t.e = id / (tp * tq);
    const int local = id % (tp * tq);
    int64_t begin, end;
    expert_rows(a, t.e, begin, end);
    t.p0 = local / tq * S::BP;
    t.q0 = local % tq * S::BQ;
    t.pv = min(S::BP, a.n - t.p0);
    t.qv = min(S::BQ, a.k - (int)t.q0);
    t.P = Operand{reinterpret_cast<const unsigned char*>(a.x) + begin * a.ldx * 2, a.ldx * 2, t.p0, t.pv};
    t.Q = Operand{reinterpret_cast<const unsigned char*>(a.w) + begin * a.ldw * 2, a.ldw * 2, t.q0, t.qv};
    t.ready(end - begin);
  };
  auto put = [&](const Tile<S>& t, const v16f(&acc)[S::RB][S::CB], unsigned char*) {
    if (a.y_f32)
      put_weight<S>(a, reinterpret_cast<float*>(a.y) + t.e * a.y_stride, t.p0, t.pv, (int)t.q0, t.qv, acc);
    else
      put_weight<S>(a, reinterpret_cast<T*>(a.y) + t.e * a.y_stride, t.p0, t.pv, (int)t.q0, t.qv, acc);
  };
  if (FAST && a.ahead) {
    const int64_t first = offset_at(a, 0), last = offset_at(a, a.experts);
    read_ahead(a.x, a.ldx * 2, first, last, a.n / 8, S::THREADS / 64);
    read_ahead(a.w, a.ldw * 2, first, last, a.k / 8, S::THREADS / 64);
  }
  stream_tiles<S, T, true, true, FAST>(share_experts<S::BK>(a, tp * tq), lds, load, put);
}

// ------------------------------------------------------------ launchers
namespace {

using Large = GroupedShape<256, 128, 2, 2, 64, 3, 1>;
using Middle = GroupedShape<128, 64, 2, 2, 64, 4, 1>;
using Small = GroupedShape<64, 32, 2, 1, 64, 4, 2>;
using Edge = GroupedShape<128, 128, 2, 2, 64, 4, 1>;

template <class S, typename T, bool TRANSPOSE, bool FAST>
hipError_t go_rows(const GroupedArgs& a, hipStream_t s) {
  static std::atomic<uint64_t> raised{0};
  auto kernel = grouped_tile_kernel<S, T, TRANSPOSE, FAST>;
  if (hipError_t e = raise_lds(kernel, S::LDS, raised); e != hipSuccess) return e;
  const int64_t outs = TRANSPOSE ? a.k : a.n;
  const int64_t groups = a.experts < a.rows ? a.experts : a.rows;
  const int64_t tiles = (a.rows / S::BQ + groups) * ((outs + S::BP - 1) / S::BP);  // at most
  hipLaunchKernelGGL(kernel, dim3(persistent_blocks(tiles, S::BPC)), dim3(S::THREADS), S::LDS, s, a);
  return hipGetLastError();
}

template <class S, typename T, bool FAST>
hipError_t go_weights(const GroupedArgs& a, hipStream_t s) {
  static std::atomic<uint64_t> raised{0};
  auto kernel = grouped_weight_kernel<S, T, FAST>;
  if (hipError_t e = raise_lds(kernel, S::LDS, raised); e != hipSuccess) return e;
  const int64_t tiles = (int64_t)a.experts * ((a.n + S::BP - 1) / S::BP) * ((a.k + S::BQ - 1) / S::BQ);
  hipLaunchKernelGGL(kernel, dim3(persistent_blocks(tiles, S::BPC)), dim3(S::THREADS), S::LDS, s, a);
  return hipGetLastError();
}

// Rounds of tiles that the CUs go through.
template <class S>
int64_t rounds(int64_t tiles) {
  const int64_t slots = 256 * S::BPC;
  return (tiles + slots - 1) / slots;
}

// The tile whose rounds times the time of one of its chunks is least: 1.0, 0.7
// and 0.65 us for the large, middle and small one.  It decides as the
// measurements do (large / middle / small tiles, us, n = 2048, k = 1536, bf16):
// 64 experts with 16384 rows 145 / 226 / 367, with 256 rows 79 / 76 / 75; 8
// experts with 1024 rows 22 / 16 / 24, with 64 rows 20 / 13 / 12.
template <typename T, bool TRANSPOSE>
hipError_t pick_rows(const GroupedArgs& a, hipStream_t s) {
  if (!a.fast) return go_rows<Edge, T, TRANSPOSE, false>(a, s);
  const int64_t outs = TRANSPOSE ? a.k : a.n;
  // experts of equal size, as many as can have rows
  const int64_t groups = a.experts < a.rows ? a.experts : a.rows, each = (a.rows + groups - 1) / groups;
  auto tiles = [&](int p, int q) { return groups * ((each + q - 1) / q) * ((outs + p - 1) / p); };
  const int64_t l = 20 * rounds<Large>(tiles(256, 128)), m = 14 * rounds<Middle>(tiles(128, 64)),
                n = 13 * rounds<Small>(tiles(64, 32));
  if (n < l && n < m) return go_rows<Small, T, TRANSPOSE, true>(a, s);
  if (m < l) return go_rows<Middle, T, TRANSPOSE, true>(a, s);
  return go_rows<Large, T, TRANSPOSE, true>(a, s);
}

// Here a tile takes its chunks and its stores: 1.0 us a chunk and 5.4 us for the
// large tile, 0.45 and 1.4 for the middle one (64 equal experts with 16384 rows 191 /
// 290 us, 8 with 4096 rows 42 / 61; 1 with 16384 rows, 1024 x 1024: 155 / 94).
// Operands are read ahead where experts have 64 to 512 rows in the mean and the
// last-level cache (256 MB) holds the operands.  us without / with, 64 uneven
// experts of 2048 x 1536 unless said, behind the rows' gradient, which has just
// read dy, and with nothing in the caches:
//   rows (operands)            behind the rows' gradient   cold
//   2048 (15 MB)               159 / 161                   154 / 161
//   4096 (29 MB)               164 / 158                   172 / 161
//   16384 (117 MB)             263 / 210                   301 / 218
//   16384, 3328 x 2560 (193)   715 / 498                   782 / 529
//   32768 (235)                358 / 323                   398 / 348
//   32768, 2048 x 1792 (252)   404 / 390                   446 / 398
//   32768, 2560 x 2048 (302)   673 / 717                   723 / 767
//   8 experts, 4096 (29)       66 / 59                     72 / 62
//   16, 8192, 2048 x 2048 (67) 126 / 127                   155 / 129
//   24, 24576 (176)            206 / 232                   254 / 254
//   32, 32768 (235)            257 / 283                   320 / 312
// With both operands already in the caches it costs 7% (16384 rows, experts of equal
// size: 201 / 187).
template <typename T>
hipError_t pick_weights(GroupedArgs a, hipStream_t s) {
  if (!a.fast) return go_weights<Edge, T, false>(a, s);
  a.ahead = a.rows >= 64 * (int64_t)a.experts && a.rows <= 512 * (int64_t)a.experts &&
            a.rows * (a.n + (int64_t)a.k) * 2 <= 256 * int64_t(1000000);
  auto tiles = [&](int p, int q) { return (int64_t)a.experts * ((a.n + p - 1) / p) * ((a.k + q - 1) / q); };
  const int64_t chunks = (a.rows / a.experts + 63) / 64;
  const int64_t l = rounds<Large>(tiles(256, 128)) * (chunks * 20 + 108), m = rounds<Middle>(tiles(128, 64)) * (chunks * 9 + 28);
  return m < l ? go_weights<Middle, T, true>(a, s) : go_weights<Large, T, true>(a, s);
}

}  // namespace

hipError_t launch_grouped(const GroupedArgs& a, mr_dtype dt, bool transpose, hipStream_t s) {
  if (dt == MR_F16) return transpose ? pick_rows<_Float16, true>(a, s) : pick_rows<_Float16, false>(a, s);
  return transpose ? pick_rows<bf16_t, true>(a, s) : pick_rows<bf16_t, false>(a, s);
}

hipError_t launch_grouped_weight_grad(const GroupedArgs& a, mr_dtype dt, hipStream_t s) {
  return dt == MR_F16 ? pick_weights<_Float16>(a, s) : pick_weights<bf16_t>(a, s);
}

}  // namespace mr
