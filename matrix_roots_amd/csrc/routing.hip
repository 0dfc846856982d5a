// What lies between tokens and the products of a bank of experts.
//
// Routing: a token's k experts are the k largest of its logits l, ties to the
// lowest index, -inf never; with S all experts or those k,
//   log_sum = log sum_{e in S} exp(l_e),  w_j = exp(l_{e_j} - log_sum),
// and from dw, with c = sum_j w_j dw_j over the chosen,
//   dl_e = [e chosen] w_e (dw_e - c)            (S the chosen)
//   dl_e = [e chosen] w_e dw_e - c exp(l_e) / sum_e exp(l_e)   (S all).
//
// Order: a stable counting sort of the tokens' choices by expert.  place[t, j] is
// the row of choice j of token t; choices of no expert come behind the last
// expert's rows, so the places are a permutation.
//
// Rows: dispatch copies a token's row to the places of its choices (times their
// weights), combine adds a token's rows up (times the weights, and to a
// residual).  Each is the other's gradient; the weights' is the dot product of
// the two rows, which dispatch takes on the way.  HBM-bound: 16384 x 8 rows of
// 2048 bf16 out in 118 us (605 MB, 5.1 TB/s, passes one after another), back with
// weights and residual in 125 (656 MB, 5.2 TB/s); 4001 x 4 rows of 1337 fp16 with
// both gradients 19 us (94 MB).
#include "experts.hpp"
#include "linear_common.hpp"
#include "mr_common.hpp"

namespace mr {

namespace {

// What the lane r places on along its row of 16 holds, in either direction.
template <int R>
__device__ __forceinline__ uint32_t ror(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 | R, 0xf, 0xf, false);
}
template <int R>
__device__ __forceinline__ float ror(float v) {
  return __uint_as_float(ror<R>(__float_as_uint(v)));
}
// What the lane R places back holds, 0 in a row's first R lanes.
template <int R>
__device__ __forceinline__ int shr(int v) {
  return __builtin_amdgcn_update_dpp(0, v, 0x110 | R, 0xf, 0xf, false);
}
// Of numbers (no NaN), without the quieting that fmaxf and fminf add.
__device__ __forceinline__ float larger(float a, float b) { return __builtin_amdgcn_fmed3f(a, b, __builtin_inff()); }
__device__ __forceinline__ float smaller(float a, float b) { return __builtin_amdgcn_fmed3f(a, b, -__builtin_inff()); }
__device__ __forceinline__ uint32_t umin(uint32_t a, uint32_t b) { return a < b ? a : b; }

// Over the LPT = 16 or 64 lanes of a token, in each of them.
template <int LPT, typename V, typename F>
__device__ __forceinline__ V over(V v, F&& f) {
  v = f(v, ror<8>(v));
  v = f(v, ror<4>(v));
  v = f(v, ror<2>(v));
  v = f(v, ror<1>(v));
  if (LPT == 64) {
    v = f(v, __shfl_xor(v, 16));
    v = f(v, __shfl_xor(v, 32));
  }
  return v;
}
template <int LPT>
__device__ __forceinline__ float max_of(float v) {
  return over<LPT>(v, [](float a, float b) { return larger(a, b); });
}
template <int LPT>
__device__ __forceinline__ uint32_t min_of(uint32_t v) {
  return over<LPT>(v, [](uint32_t a, uint32_t b) { return umin(a, b); });
}
template <int LPT>
__device__ __forceinline__ float sum_of(float v) {
  return over<LPT>(v, [](float a, float b) { return a + b; });
}

// Unsigned numbers in the order of the values; the zeros are one.
__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.f);
  return (u >> 31) ? ~u : u | 0x80000000u;
}

template <typename T>
struct Raw4 {
  typedef uint32_t u __attribute__((ext_vector_type(sizeof(T))));
  typedef u any __attribute__((aligned(1)));
};
__device__ __forceinline__ float widen_of(const v4u& r, int i, float) { return __uint_as_float(r[i]); }
__device__ __forceinline__ float widen_of(const v2u& r, int i, bf16_t) {
  return __uint_as_float(i & 1 ? r[i >> 1] & 0xffff0000u : r[i >> 1] << 16);
}
__device__ __forceinline__ float widen_of(const v2u& r, int i, _Float16) {
  const uint16_t h = (uint16_t)(i & 1 ? r[i >> 1] >> 16 : r[i >> 1]);
  _Float16 f;
  __builtin_memcpy(&f, &h, 2);
  return (float)f;
}
// Q times four consecutive logits of a row, from columns c, c + step, ..; -inf
// behind its end.  All loads come before the first use and without a branch that
// lanes take apart: lanes at the end load the row's last four and move them down
// (rows of one to three go to all lanes, and count for the first).
template <typename T, int Q>
__device__ __forceinline__ void load_logits(const T* row, int c, int step, int n, float (&v)[4 * Q]) {
  if (n >= 4) {
    typename Raw4<T>::u r[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int at = c + q * step;
      r[q] = *reinterpret_cast<const typename Raw4<T>::any*>(row + (at + 4 <= n ? at : n - 4));
    }
#pragma unroll
    for (int i = 0; i < 4 * Q; ++i) v[i] = widen_of(r[i / 4], i % 4, T());
    if (n & 3) {
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const int s = c + q * step + 4 - n;
        const bool one = s > 0 && (s & 1), two = s > 0 && (s & 2);
#pragma unroll
        for (int i = 0; i < 3; ++i) v[4 * q + i] = one ? v[4 * q + i + 1] : v[4 * q + i];
#pragma unroll
        for (int i = 0; i < 2; ++i) v[4 * q + i] = two ? v[4 * q + i + 2] : v[4 * q + i];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4 * Q; ++i) v[i] = i < 3 ? widen(row[i < n ? i : 0]) : 0.f;
  }
  if (Q * step == n && step > 0) return;  // whole
#pragma unroll
  for (int q = 0; q < Q; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i) v[4 * q + i] = c + q * step + i < n ? v[4 * q + i] : -__builtin_inff();
}
template <typename T>
__device__ __forceinline__ void store4(T* row, int c, int n, const float (&v)[4]) {
  T t[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) t[i] = narrow<T>(v[i]);
  if (c + 4 <= n) {
    if constexpr (sizeof(T) == 4) {
      v4u u;
      __builtin_memcpy(&u, t, 16);
      *reinterpret_cast<v4u_any*>(row + c) = u;
    } else {
      v2u u;
      __builtin_memcpy(&u, t, 8);
      *reinterpret_cast<v2u_any*>(row + c) = u;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (c + i < n) row[c + i] = t[i];
}

}  // namespace

// ---------------------------------------------------------------- routing
// LPT lanes for each token, Q times four logits in each: columns 4 (lane + LPT q)
// and the three behind.
//
// Up to eight choices by 16 lanes: with tau the k-th largest of the lanes' own
// largest logits, k of a token's logits at least reach tau, so all chosen ones do.
// They are few, go to LDS, and each finds its place by comparing itself with the
// others.  Where more reach tau than there is room for (many are equal), and for
// more choices, one is chosen after another: the largest, its first place, which is
// then taken out.
//
// Room for 16, one in each lane, up to 128 logits, for 32, two in each, above.  How
// many reach tau depends on k more than on the number of experts.  k = 8: 10.5 in the
// mean of 384 normal logits, 10.2 of 128; more than 16 for one token in 125 and one in
// 280, and the few waves that choose one after another for it end behind all others.
// k = 4: 4.4, and more than 16 for none.  Among a few dozen experts the lanes that hold
// any are few, and tau low: of 40 logits 5% of the tokens have more than 16 for k = 8, of
// 32 37%, of 17 to 28 all of them.  None of 200000 tokens of up to 512 had more than 32.
// In a captured graph, float32, with room for 16 / for 32 / one after another:
//   16384 x 384, k = 8   13.5 /  9.9 / 15.5 us (25 MB, 5 us, in one burst of loads before the comparisons)
//   65536 x 128, k = 4   12.8 / 15.0 / 14.5    (the second place's registers halve the resident waves)
//   65536 x 128, k = 8   15.0 / 16.1 / 21.8
//   16384 x 128, k = 8    7.4 /  6.4 /  8.3    (fewer waves than the card holds: they cost nothing)
//   65536 x 64,  k = 8   12.1 / 13.2 / 17.9
//   16384 x 32,  k = 8    7.6 /  7.0 /  7.0
// k = 16, one after another: 16384 x 384 25 us.  k = 8 beyond: 16384 x 512 13 us; one after
// another by 64 lanes 16384 x 513 and x 1024 34, x 2048 59 (134 MB), 4096 x 4096 44.
template <typename T, int LPT, int Q>
__global__ __launch_bounds__(256) void route_kernel(const RouteArgs a) {
  constexpr int TPB = 256 / LPT, N = 4 * Q, kReach = Q <= 2 ? 16 : 32;
  constexpr float kInf = __builtin_inff();
  __shared__ uint64_t reach[LPT == 16 ? TPB : 1][kReach];
  const int lane = threadIdx.x % LPT;
  for (int64_t t0 = (int64_t)blockIdx.x * TPB; t0 < a.tokens; t0 += (int64_t)gridDim.x * TPB) {
    // lanes behind the last token work on that one and store nothing
    const bool held = t0 + threadIdx.x / LPT < a.tokens;
    const int64_t t = held ? t0 + threadIdx.x / LPT : a.tokens - 1;
    const T* row = reinterpret_cast<const T*>(a.logits) + t * a.ldl;
    float v[N];
    load_logits<T, Q>(row, 4 * lane, 4 * LPT, a.n, v);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = v[i] != v[i] ? kInf : v[i];
    auto largest = [&]() {
      float m = v[0];
#pragma unroll
      for (int i = 1; i < N; ++i) m = larger(m, v[i]);
      return m;
    };
    const float own = largest(), top = max_of<LPT>(own);
    float sum = 0.f;
    if (!a.normalize) {
#pragma unroll
      for (int i = 0; i < N; ++i) sum += v[i] == -kInf ? 0.f : expf(v[i] - top);
      sum = sum_of<LPT>(sum);
    }
    // of this lane: one of the chosen, which one of them, its share before the division
    int32_t expert = -1, second = -1;
    int place = lane, second_place = kMaxRouted;
    float part = 0.f, second_part = 0.f;
    bool done = false;
    if constexpr (LPT == 16) {
      if (a.k <= 8) {
        int above = 0;
        static_for<15>([&](auto r) { above += ror<r.value + 1>(own) > own; });
        float tau = over<16>(above < a.k ? own : kInf, [](float x, float y) { return smaller(x, y); });
        tau = larger(tau, -3.402823466e38f);  // -inf is not chosen
        int count = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) count += v[i] >= tau;
        int upto = count;
        upto += shr<1>(upto);
        upto += shr<2>(upto);
        upto += shr<4>(upto);
        upto += shr<8>(upto);
        const int total = over<16>((uint32_t)upto, [](uint32_t x, uint32_t y) { return umax(x, y); });
        done = !__any(total > kReach);
        if (done) {
          uint64_t* mine = reach[threadIdx.x / 16];
          int at = upto - count;
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (v[i] >= tau) mine[at++] = (uint64_t)__float_as_uint(v[i]) << 32 | ~(4u * lane + 64u * (i / 4) + i % 4);
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
          // of lanes behind the last one, whatever lies there
          const uint64_t one = mine[lane], two = mine[kReach - 16 + lane];
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
          const float value = __uint_as_float((uint32_t)(one >> 32)), value2 = __uint_as_float((uint32_t)(two >> 32));
          const uint32_t lo = (uint32_t)one, hi = lane < total ? key_of(value) : 0;
          const uint64_t key = (uint64_t)hi << 32 | lo;
          place = 0;
          static_for<15>([&](auto r) {
            place += ((uint64_t)ror<r.value + 1>(hi) << 32 | ror<r.value + 1>(lo)) > key;
          });
          if (kReach > 16 && __any(total > 16)) {  // some lanes hold two
            const uint32_t lo2 = (uint32_t)two, hi2 = 16 + lane < total ? key_of(value2) : 0;
            const uint64_t key2 = (uint64_t)hi2 << 32 | lo2;
            place += key2 > key;
            second_place = key > key2;
            static_for<15>([&](auto r) {
              const uint64_t other2 = (uint64_t)ror<r.value + 1>(hi2) << 32 | ror<r.value + 1>(lo2);
              place += other2 > key;
              second_place += (((uint64_t)ror<r.value + 1>(hi) << 32 | ror<r.value + 1>(lo)) > key2) + (other2 > key2);
            });
            if (hi2 && second_place < a.k) {
              second = (int32_t)~lo2;
              second_part = expf(value2 - top);
            }
          }
          if (lane >= total) place = lane;  // behind the others
          if (lane < total && place < a.k) {
            expert = (int32_t)~lo;
            part = expf(value - top);
          }
        }
      }
    }
    if (!done) {
      place = lane;
      for (int j = 0; j < a.k; ++j) {
        const float m = max_of<LPT>(largest());
        // the first of the equal ones
        uint32_t at = 0xffffffffu;
#pragma unroll
        for (int i = N - 1; i >= 0; --i) at = v[i] == m ? 4u * LPT * (i / 4) + i % 4 : at;
        at = min_of<LPT>(at == 0xffffffffu ? at : at + 4u * lane);
        const uint32_t here = at - 4u * lane;
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = here == 4u * LPT * (i / 4) + i % 4 ? -kInf : v[i];
        if (lane == j && m > -kInf) {
          expert = (int32_t)at;
          part = expf(m - top);
        }
      }
    }
    if (a.normalize) sum = sum_of<LPT>(part + second_part);
    if (!held) continue;
    if (place < a.k) {
      a.experts[t * a.k + place] = expert;
      a.weights[t * a.k + place] = expert < 0 ? 0.f : part / sum;
    }
    if (second >= 0) {
      a.experts[t * a.k + second_place] = second;
      a.weights[t * a.k + second_place] = second_part / sum;
    }
    if (lane == 0) a.log_sum[t] = top == -kInf ? top : top + logf(sum);
  }
}

// One wave for each token, its choices in the first lanes (8191 x 250 bf16, k = 6:
// 7.6 us with the shares of all, 10 MB; latency).  The softmax over all
// experts is worked out again from the logits (ONE: a row's are at most 256, four in
// each lane): exp(l - log_sum) from a kept log_sum is off by its rounding, which
// for large logits, or rows at the type's lowest value, is more than the result.
template <typename T, bool ONE>
__global__ __launch_bounds__(256) void route_grad_kernel(const RouteGradArgs a) {
  const int lane = threadIdx.x & 63;
  for (int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6); t < a.tokens; t += (int64_t)gridDim.x * 4) {
    int expert = -1;
    float w = 0.f, dw = 0.f;
    if (lane < a.k) {
      expert = a.experts[t * a.k + lane];
      if (expert >= 0 && expert < a.n) {
        w = a.weights[t * a.k + lane];
        dw = a.dweights[t * a.k + lane];
      } else {
        expert = -1;
      }
    }
    const T* row = reinterpret_cast<const T*>(a.logits) + t * a.ldl;
    T* out = reinterpret_cast<T*>(a.dlogits) + t * a.ldd;
    float v[4], top = -__builtin_inff(), sum = 0.f;
    if (!a.normalize) {
      for (int c0 = 0; c0 < (ONE ? 1 : a.n); c0 += 256) {
        load_logits<T, 1>(row, c0 + 4 * lane, 0, a.n, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) top = fmaxf(top, v[i]);
      }
#pragma unroll
      for (int m = 1; m < 64; m <<= 1) top = fmaxf(top, __shfl_xor(top, m));
      for (int c0 = 0; c0 < (ONE ? 1 : a.n); c0 += 256) {
        if (!ONE) load_logits<T, 1>(row, c0 + 4 * lane, 0, a.n, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = v[i] == -__builtin_inff() ? 0.f : expf(v[i] - top);
          sum += v[i];
        }
      }
      sum = sum64(sum);
    }
    const float c = __uint_as_float((uint32_t)__builtin_amdgcn_readfirstlane((int)__float_as_uint(sum_of<16>(w * dw))));
    const float part = a.normalize ? w * (dw - c) : w * dw;
    const float share = sum == 0.f ? 0.f : c / sum;
    for (int c0 = 0; c0 < (ONE ? 1 : a.n); c0 += 256) {
      const int col = c0 + 4 * lane;
      float d[4] = {0.f, 0.f, 0.f, 0.f};
      if (!a.normalize) {
        if (!ONE) {
          load_logits<T, 1>(row, col, 0, a.n, v);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = v[i] == -__builtin_inff() ? 0.f : expf(v[i] - top);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] = -v[i] * share;
      }
      for (int j = 0; j < a.k; ++j) {
        const int e = __builtin_amdgcn_readlane(expert, j) - c0;
        if (e < 0 || e >= 256) continue;
        const float p = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(part), j));
#pragma unroll
        for (int i = 0; i < 4; ++i) d[i] += e == 4 * lane + i ? p : 0.f;
      }
      if (col < a.n) store4<T>(out, col, a.n, d);
    }
  }
}

// ------------------------------------------------------------------ order
namespace {

// Choices of a lane in a round.  All of a few thousand in one workgroup's only
// round spare a launch (4096 choices: 6.5 us, in two launches 8.0); more are
// shared out thinly, as a workgroup's waves wait for one another (131072 choices
// of 64 and of 384 experts: 9.1 and 12.1 us with two, 11.1 and 12.7 with four, 8.6
// and 13.7 with one).
constexpr int kAlone = 4, kShared = 2;

// Expert of choice f, n where it is none.
__device__ __forceinline__ int choice(const OrderArgs& a, int f) {
  const int64_t at = a.lde == a.k ? f : (int64_t)(f / a.k) * a.lde + f % a.k;
  if (a.wide) {
    const int64_t e = reinterpret_cast<const int64_t*>(a.experts)[at];
    return e >= 0 && e < a.n ? (int)e : a.n;
  }
  const int e = reinterpret_cast<const int32_t*>(a.experts)[at];
  return e >= 0 && e < a.n ? e : a.n;
}

// Exclusive sums of v[0 .. n) in LDS, by the whole workgroup; `waves` has a place for each wave.
__device__ __forceinline__ void exclusive_sums(int32_t* v, int n, int32_t* waves) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int per = (n + (int)blockDim.x - 1) / (int)blockDim.x, first = (int)threadIdx.x * per;
  int own = 0;
  for (int i = first; i < first + per && i < n; ++i) own += v[i];
  int upto = own;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(upto, d);
    if (lane >= d) upto += o;
  }
  __syncthreads();
  if (lane == 63) waves[wave] = upto;
  __syncthreads();
  int before = upto - own;
  for (int w = 0; w < wave; ++w) before += waves[w];
  for (int i = first; i < first + per && i < n; ++i) {
    const int c = v[i];
    v[i] = before;
    before += c;
  }
  __syncthreads();
}

}  // namespace

// Bound by latency: a workgroup goes once through loads, comparisons, LDS and stores
// (131072 choices: 5.5 us, 1 MB).
//
// The places of a workgroup's choices, in rounds of R for each lane.  In a
// round each wave takes the next 64 R: lanes of one expert find each other by
// the bits of its number, the first of them keeps the wave's count.  With one
// workgroup, and one round, the places are final; else they count from the
// expert's first row of this workgroup, and order_place_kernel adds where that is.
template <int R>
__global__ __launch_bounds__(1024) void order_rank_kernel(const OrderArgs a) {
  extern __shared__ int32_t lds[];  // waves x bins counts, bins totals, 16 for the scan
  const int bins = a.n + 1, waves = blockDim.x >> 6;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int32_t* count = lds + wave * bins;
  int32_t* total = lds + waves * bins;
  const int64_t begin = (int64_t)blockIdx.x * a.chunk;
  const int64_t end = begin + a.chunk < a.total ? begin + a.chunk : a.total;
  const int round = (int)blockDim.x * R;
  int64_t f = end;
  int e[R], rank[R];
  for (int i = threadIdx.x; i < bins; i += blockDim.x) total[i] = 0;
  for (int64_t f0 = begin; f0 < end; f0 += round) {
    f = f0 + wave * 64 * R + lane;
#pragma unroll
    for (int r = 0; r < R; ++r) e[r] = f + 64 * r < end ? choice(a, (int)(f + 64 * r)) : a.n;
    for (int i = threadIdx.x; i < waves * bins; i += blockDim.x) lds[i] = 0;
    __syncthreads();
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const bool valid = f + 64 * r < end;
      uint64_t same = __ballot(valid);
      for (int b = 0; (bins - 1) >> b; ++b) {
        const bool bit = (e[r] >> b) & 1;
        const uint64_t set = __ballot(bit);
        same &= bit ? set : ~set;
      }
      const int before = __popcll(same & ((uint64_t(1) << lane) - 1));
      if (valid) {
        const int prior = count[e[r]];
        rank[r] = prior + before;
        if (before == 0) count[e[r]] = prior + __popcll(same);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
    __syncthreads();
    // the waves' counts to the sums over what comes before them
    for (int i = threadIdx.x; i < bins; i += blockDim.x) {
      int s = total[i];
#pragma unroll 4
      for (int w = 0; w < waves; ++w) {
        const int c = lds[w * bins + i];
        lds[w * bins + i] = s;
        s += c;
      }
      total[i] = s;
    }
    __syncthreads();
    if (!a.counts) break;  // one workgroup has one round
#pragma unroll
    for (int r = 0; r < R; ++r)
      if (f + 64 * r < end) a.place[f + 64 * r] = rank[r] + count[e[r]];
    __syncthreads();
  }
  if (a.counts) {
    for (int i = threadIdx.x; i < bins; i += blockDim.x) a.counts[(int64_t)blockIdx.x * bins + i] = total[i];
    return;
  }
  __syncthreads();
  exclusive_sums(total, bins, total + bins);
  for (int i = threadIdx.x; i < bins; i += blockDim.x) a.offsets[i] = total[i];
#pragma unroll
  for (int r = 0; r < R; ++r)
    if (f + 64 * r < end) a.place[f + 64 * r] = rank[r] + count[e[r]] + total[e[r]];
}

// Adds to a workgroup's places the rows of lower experts and of its expert in
// earlier workgroups.
__global__ __launch_bounds__(1024) void order_place_kernel(const OrderArgs a) {
  extern __shared__ int32_t lds[];  // bins totals, bins of earlier workgroups, 16 for the scan
  const int bins = a.n + 1;
  int32_t* total = lds;
  int32_t* before = lds + bins;
  for (int i = threadIdx.x; i < 2 * bins; i += blockDim.x) lds[i] = 0;
  __syncthreads();
  // every bin by as many threads as there are for it
  const int by = bins < (int)blockDim.x ? (int)blockDim.x / bins : 1;
  for (int i = threadIdx.x; i < bins * by; i += blockDim.x) {
    const int e = i % bins;
    int s = 0, early = 0;
#pragma unroll 4
    for (int g = i / bins; g < a.blocks; g += by) {
      const int c = a.counts[(int64_t)g * bins + e];
      s += c;
      early += g < (int)blockIdx.x ? c : 0;
    }
    atomicAdd(&total[e], s);
    atomicAdd(&before[e], early);
  }
  __syncthreads();
  exclusive_sums(total, bins, before + bins);
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e < bins; e += blockDim.x) a.offsets[e] = total[e];
  const int64_t begin = (int64_t)blockIdx.x * a.chunk;
  const int64_t end = begin + a.chunk < a.total ? begin + a.chunk : a.total;
  for (int64_t f = begin + threadIdx.x; f < end; f += blockDim.x * kShared) {
    int e[kShared], p[kShared];
#pragma unroll
    for (int r = 0; r < kShared; ++r) {
      const int64_t g = f + (int64_t)blockDim.x * r;
      e[r] = g < end ? choice(a, (int)g) : 0;
      p[r] = g < end ? a.place[g] : 0;
    }
#pragma unroll
    for (int r = 0; r < kShared; ++r) {
      const int64_t g = f + (int64_t)blockDim.x * r;
      if (g < end) a.place[g] = p[r] + total[e[r]] + before[e[r]];
    }
  }
}

// ------------------------------------------------------------------- rows
namespace {

// How many sorted rows belong to an expert, 0 .. rows.
__device__ __forceinline__ int64_t held_rows(const RowsArgs& a, int64_t rows) {
  const int64_t h = a.offsets[a.experts];
  return h < 0 ? 0 : h < rows ? h : rows;
}

// Eight columns from `at` of a row.  At a ragged end they are the row's last eight,
// so that no load or store is taken apart; the first `skip` of them are a
// neighbour's too, which stores the same there.  Rows of less than eight (FEW)
// have one such part.
template <typename T, bool FEW>
struct Part {
  int c, skip, width;
  __device__ __forceinline__ Part(int at, int w) : width(w) {
    c = FEW ? 0 : at + 8 <= w ? at : w - 8;
    skip = FEW ? (at == 0 ? 0 : 8) : at - c;
  }
  __device__ __forceinline__ bool any() const { return skip < 8; }
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
  __device__ __forceinline__ void store(T* row, const Raw8<T>& r) const {
    if constexpr (!FEW) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(T) / 2; ++i) reinterpret_cast<v4u_any*>(row + c)[i] = r.u[i];
    } else {
      T v[8];
      __builtin_memcpy(v, &r, sizeof r);
#pragma unroll
      for (int i = 0; i < 7; ++i)
        if (i < width) row[i] = v[i];
    }
  }
};
template <typename T>
__device__ __forceinline__ Raw8<T> narrow8(const float (&v)[8]) {
  T t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = narrow<T>(v[i]);
  Raw8<T> r;
  __builtin_memcpy(&r, t, sizeof r);
  return r;
}

// Combined rows go in parts of 128 columns, 16 lanes of eight each; the parts of a row
// are neighbours, so that a wave's four are 512 columns of a wide row or four rows.
constexpr int kPartLanes = 16, kPart = 8 * kPartLanes;
constexpr int kChoices = 4;  // of a token, in flight together

// The job of the thread's 16 lanes: part `part` of token t, or t past the end.
__device__ __forceinline__ void part_of(int64_t job, int64_t jobs, int parts, int64_t& t, int& part) {
  t = jobs >> 31 ? job / parts : (int)job / parts;
  part = (int)(job - t * parts);
}

}  // namespace

// To the places of a token's choices.  LPR = 16 or 64 lanes, CH parts of eight columns
// in each, for a piece of its row: wide rows go out in pieces of 4 KB (16384 x 8
// rows of 2048 bf16: 92 us from a clean cache, in pieces of 256 bytes 105).
template <typename T, int LPR, int CH, bool FEW>
__global__ __launch_bounds__(256) void dispatch_kernel(const RowsArgs a) {
  constexpr int GPB = 256 / LPR, kPiece = 8 * LPR * CH;
  const int64_t rows = a.tokens * a.k, held = held_rows(a, rows);
  const int parts = (a.width + kPiece - 1) / kPiece;
  const int64_t jobs = a.tokens * parts;
  for (int64_t job = (int64_t)blockIdx.x * GPB + threadIdx.x / LPR; job < jobs; job += (int64_t)gridDim.x * GPB) {
    int64_t t;
    int part;
    part_of(job, jobs, parts, t, part);
    const int32_t* place = a.place + t * a.k;
    const int c0 = part * kPiece + 8 * (int)(threadIdx.x % LPR);
    Raw8<T> v[CH];
#pragma unroll
    for (int q = 0; q < CH; ++q) v[q] = Part<T, FEW>(c0 + 8 * LPR * q, a.width).load(reinterpret_cast<const T*>(a.x) + t * a.ldx);
    for (int j0 = 0; j0 < a.k; j0 += kChoices) {
      int64_t p[kChoices];
#pragma unroll
      for (int i = 0; i < kChoices; ++i) p[i] = place[j0 + i < a.k ? j0 + i : j0];
#pragma unroll
      for (int i = 0; i < kChoices; ++i) {
        if (j0 + i >= a.k || p[i] < 0 || p[i] >= rows) continue;
        T* y = reinterpret_cast<T*>(a.out) + p[i] * a.ldo;
#pragma unroll
        for (int q = 0; q < CH; ++q) {
          const Part<T, FEW> at(c0 + 8 * LPR * q, a.width);
          if (at.any()) at.store(y, p[i] < held ? v[q] : Raw8<T>{});
        }
      }
    }
  }
}

// LPR = 16 or 64 lanes for each choice, CH parts of eight columns in each at a time:
// the token's row times the choice's weight to its place, and its dot product with
// the row that lies there.  A token's choices are neighbours, so that its row is read from memory once.
template <typename T, int LPR, int CH, bool FEW>
__global__ __launch_bounds__(256) void dispatch_dot_kernel(const RowsArgs a) {
  constexpr int GPB = 256 / LPR;
  const int lane = threadIdx.x % LPR;
  const int64_t rows = a.tokens * a.k, held = held_rows(a, rows);
  for (int64_t f = (int64_t)blockIdx.x * GPB + threadIdx.x / LPR; f < rows; f += (int64_t)gridDim.x * GPB) {
    const int64_t p = a.place[f], t = (int)f / a.k;
    const bool in = p >= 0 && p < held;
    const float w = a.weights ? a.weights[f] : 1.f;
    const T* x = reinterpret_cast<const T*>(a.x) + t * a.ldx;
    const T* z = reinterpret_cast<const T*>(a.rows) + (in ? p : 0) * a.ldr;
    T* y = reinterpret_cast<T*>(a.out) + p * a.ldo;
    float dot = 0.f;
    for (int c0 = 0; c0 < a.width; c0 += 8 * LPR * CH) {
      Raw8<T> rx[CH], rz[CH];
#pragma unroll
      for (int q = 0; q < CH; ++q) rx[q] = Part<T, FEW>(c0 + 8 * (lane + LPR * q), a.width).load(x);
#pragma unroll
      for (int q = 0; q < CH; ++q) rz[q] = in ? Part<T, FEW>(c0 + 8 * (lane + LPR * q), a.width).load(z) : Raw8<T>{};
#pragma unroll
      for (int q = 0; q < CH; ++q) {
        const Part<T, FEW> at(c0 + 8 * (lane + LPR * q), a.width);
        float v[8], u[8];
        widen8(rx[q], v);
        widen8(rz[q], u);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          // (beyond a row of less than eight both are 0)
          dot = i >= at.skip ? fmaf(u[i], v[i], dot) : dot;
          v[i] = in ? w * v[i] : 0.f;
        }
        if (at.any() && p >= 0 && p < rows) at.store(y, narrow8<T>(v));
      }
    }
    dot = sum_of<LPR>(dot);
    if (lane == 0) a.dots[f] = in ? dot : 0.f;
  }
}

// 16 lanes for each token and part of its row: its choices that an expert has, in
// their order, four rows' loads in flight at a time.
template <typename T, bool FEW>
__global__ __launch_bounds__(256) void combine_kernel(const RowsArgs a) {
  const int64_t rows = a.tokens * a.k, held = held_rows(a, rows);
  const int parts = (a.width + kPart - 1) / kPart;
  const int64_t jobs = a.tokens * parts;
  for (int64_t job = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4); job < jobs; job += (int64_t)gridDim.x * 16) {
    int64_t t;
    int part;
    part_of(job, jobs, parts, t, part);
    const Part<T, FEW> at(part * kPart + 8 * (int)(threadIdx.x & 15), a.width);
    if (!at.any()) continue;
    const int32_t* place = a.place + t * a.k;
    const float* weight = a.weights + t * a.k;
    float s[8] = {};
    if (a.x) widen8(at.load(reinterpret_cast<const T*>(a.x) + t * a.ldx), s);
    for (int j0 = 0; j0 < a.k; j0 += kChoices) {
      int64_t p[kChoices];
      float w[kChoices];
      Raw8<T> r[kChoices];
#pragma unroll
      for (int q = 0; q < kChoices; ++q) {
        const int j = j0 + q < a.k ? j0 + q : j0;
        p[q] = place[j];
        w[q] = a.weights ? weight[j] : 1.f;
        if (j0 + q >= a.k || p[q] >= held) p[q] = -1;
      }
#pragma unroll
      for (int q = 0; q < kChoices; ++q)
        if (p[q] >= 0) r[q] = at.load(reinterpret_cast<const T*>(a.rows) + p[q] * a.ldr);
#pragma unroll
      for (int q = 0; q < kChoices; ++q) {
        if (p[q] < 0) continue;
        float u[8];
        widen8(r[q], u);
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = fmaf(w[q], u[i], s[i]);
      }
    }
    at.store(reinterpret_cast<T*>(a.out) + t * a.ldo, narrow8<T>(s));
  }
}

// ------------------------------------------------------------ launchers
namespace {

constexpr int64_t kMaxGroups = 1 << 16;      // workgroups of a launch over tokens; each takes every so manieth
constexpr int64_t kMaxRowGroups = 1 << 20;   // over rows' parts

template <typename T, int LPT, int Q>
hipError_t route_go(const RouteArgs& a, hipStream_t s) {
  constexpr int TPB = 256 / LPT;
  const int64_t g = (a.tokens + TPB - 1) / TPB;
  hipLaunchKernelGGL((route_kernel<T, LPT, Q>), dim3((unsigned)(g < kMaxGroups ? g : kMaxGroups)), dim3(256), 0, s, a);
  return hipGetLastError();
}
template <typename T>
hipError_t route_pick(const RouteArgs& a, hipStream_t s) {
  if (a.n <= 64) return route_go<T, 16, 1>(a, s);
  if (a.n <= 128) return route_go<T, 16, 2>(a, s);
  if (a.n <= 256) return route_go<T, 16, 4>(a, s);
  if (a.n <= 384) return route_go<T, 16, 6>(a, s);
  if (a.n <= 512) return route_go<T, 16, 8>(a, s);
  if (a.n <= 1024) return route_go<T, 64, 4>(a, s);
  if (a.n <= 2048) return route_go<T, 64, 8>(a, s);
  return route_go<T, 64, 16>(a, s);
}

unsigned token_groups(int64_t tokens) {
  const int64_t g = (tokens + 3) / 4;
  return (unsigned)(g < kMaxGroups ? g : kMaxGroups);
}

unsigned row_groups(int64_t jobs, int per_block) {
  const int64_t g = (jobs + per_block - 1) / per_block;
  return (unsigned)(g < kMaxRowGroups ? g : kMaxRowGroups);
}

template <typename T, int LPR, int CH, bool FEW = false>
hipError_t copy_go(const RowsArgs& a, hipStream_t s) {
  constexpr int kPiece = 8 * LPR * CH;
  hipLaunchKernelGGL((dispatch_kernel<T, LPR, CH, FEW>), dim3(row_groups(a.tokens * ((a.width + kPiece - 1) / kPiece), 256 / LPR)),
                     dim3(256), 0, s, a);
  return hipGetLastError();
}
template <typename T, int LPR, int CH, bool FEW = false>
hipError_t dot_go(const RowsArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((dispatch_dot_kernel<T, LPR, CH, FEW>), dim3(row_groups(a.tokens * a.k, 256 / LPR)), dim3(256), 0, s, a);
  return hipGetLastError();
}
template <typename T>
hipError_t dispatch_go(const RowsArgs& a, hipStream_t s) {
  if (a.dots) {
    if (a.width < 8) return dot_go<T, 16, 1, true>(a, s);
    if (a.width <= 128) return dot_go<T, 16, 1>(a, s);
    if (a.width <= 256) return dot_go<T, 16, 2>(a, s);
    if (a.width <= 512) return dot_go<T, 16, 4>(a, s);
    if (a.width <= 1024) return dot_go<T, 64, 2>(a, s);
    return dot_go<T, 64, 4>(a, s);
  }
  if (a.width < 8) return copy_go<T, 16, 1, true>(a, s);
  if (a.width < 1024) return copy_go<T, 16, 1>(a, s);
  return copy_go<T, 64, sizeof(T) == 2 ? 4 : 2>(a, s);
}
template <typename T>
hipError_t combine_go(const RowsArgs& a, hipStream_t s) {
  const unsigned groups = row_groups(a.tokens * ((a.width + kPart - 1) / kPart), 16);
  if (a.width < 8)
    hipLaunchKernelGGL((combine_kernel<T, true>), dim3(groups), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((combine_kernel<T, false>), dim3(groups), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, mr_dtype dt, hipStream_t s) {
  if (dt == MR_F32) return route_pick<float>(a, s);
  if (dt == MR_F16) return route_pick<_Float16>(a, s);
  return route_pick<bf16_t>(a, s);
}

namespace {

template <typename T>
hipError_t route_grad_go(const RouteGradArgs& a, hipStream_t s) {
  if (a.n <= 256)
    hipLaunchKernelGGL((route_grad_kernel<T, true>), dim3(token_groups(a.tokens)), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((route_grad_kernel<T, false>), dim3(token_groups(a.tokens)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route_grad(const RouteGradArgs& a, mr_dtype dt, hipStream_t s) {
  if (dt == MR_F32) return route_grad_go<float>(a, s);
  if (dt == MR_F16) return route_grad_go<_Float16>(a, s);
  return route_grad_go<bf16_t>(a, s);
}

void order_plan(int64_t total, int64_t n, int32_t* chunk, int32_t* blocks, int32_t* waves) {
  // counts of every wave in 64 KB of LDS
  *waves = n < 900 ? 16 : n < 1800 ? 8 : n < 3000 ? 4 : 2;
  int64_t c = 64 * kAlone * *waves;
  if (total > c) {
    c = 64 * kShared * *waves;
    while ((total + c - 1) / c > 256) c *= 2;  // every workgroup reads all workgroups' counts
  }
  *chunk = (int32_t)c;
  *blocks = total > c ? (int32_t)((total + c - 1) / c) : 1;
}

hipError_t launch_order(const OrderArgs& a, hipStream_t s) {
  const size_t bins = (size_t)a.n + 1;
  const size_t lds = (bins * (a.waves + 1) + 16) * 4;
  if (!a.counts) {
    hipLaunchKernelGGL(order_rank_kernel<kAlone>, dim3(1), dim3(64 * a.waves), lds, s, a);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(order_rank_kernel<kShared>, dim3(a.blocks), dim3(64 * a.waves), lds, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(order_place_kernel, dim3(a.blocks), dim3(1024), (bins * 2 + 16) * 4, s, a);
  return hipGetLastError();
}

hipError_t launch_dispatch(const RowsArgs& a, mr_dtype dt, hipStream_t s) {
  if (dt == MR_F32) return dispatch_go<float>(a, s);
  if (dt == MR_F16) return dispatch_go<_Float16>(a, s);
  return dispatch_go<bf16_t>(a, s);
}

hipError_t launch_combine(const RowsArgs& a, mr_dtype dt, hipStream_t s) {
  if (dt == MR_F32) return combine_go<float>(a, s);
  if (dt == MR_F16) return combine_go<_Float16>(a, s);
  return combine_go<bf16_t>(a, s);
}

}  // namespace mr
