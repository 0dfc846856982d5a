// Host-side helpers shared by the ABI's translation units: error messages,
// alias checks, launch checks and event tracing.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <mutex>
#include <string>
#include <vector>

#include "../../include/matrix_roots.h"

namespace mr {

inline thread_local std::string g_err;

inline mr_status fail(mr_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_err = buf;
  return st;
}

inline mr_status hip_fail(hipError_t e, const char* where) {
  return fail(MR_ERR_HIP, "%s: %s", where, hipGetErrorString(e));
}

constexpr int64_t kMaxDim = 65536;

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Byte range of a rows x cols row-major matrix with leading dimension ld.
struct Range {
  uintptr_t lo, hi;
};
inline Range range_of(const void* p, int64_t rows, int64_t cols, int64_t ld, size_t es) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {lo, lo + (uintptr_t)(((rows - 1) * ld + cols) * (int64_t)es)};
}
inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }
// Byte range of a symmetric d x d matrix, full (leading dimension ld) or packed.
inline Range sym_range_of(const void* p, int64_t d, int64_t ld, size_t es, bool packed) {
  return packed ? range_of(p, 1, d * (d + 1) / 2, 0, es) : range_of(p, d, d, ld, es);
}
// All-or-nothing alias check over a whole batch: no byte range a call writes
// may overlap another one it writes or one it reads, within a problem or
// across problems (inputs may share memory with each other).
struct AliasSet {
  struct Tagged {
    Range r;
    int problem;
    const char* name;
  };
  std::vector<Tagged> outs, ins;
  void out(Range r, int i, const char* name) { outs.push_back({r, i, name}); }
  void in(Range r, int i, const char* name) { ins.push_back({r, i, name}); }
  mr_status check() {
    std::sort(outs.begin(), outs.end(), [](const Tagged& a, const Tagged& b) { return a.r.lo < b.r.lo; });
    for (size_t k = 1; k < outs.size(); ++k)
      if (outs[k].r.lo < outs[k - 1].r.hi)
        return fail(MR_ERR_ALIAS, "problem %d: %s overlaps problem %d's %s", outs[k].problem, outs[k].name,
                    outs[k - 1].problem, outs[k - 1].name);
    // the outputs are now disjoint and sorted, so the last one starting before
    // an input ends is the only one that can overlap it
    for (const Tagged& x : ins) {
      auto it = std::lower_bound(outs.begin(), outs.end(), x.r.hi,
                                 [](const Tagged& a, uintptr_t v) { return a.r.lo < v; });
      if (it != outs.begin() && std::prev(it)->r.hi > x.r.lo)
        return fail(MR_ERR_ALIAS, "problem %d: %s overlaps problem %d's %s", std::prev(it)->problem,
                    std::prev(it)->name, x.problem, x.name);
    }
    return MR_OK;
  }
};

// Base dtype and storage flag of an mr_dtype argument.
inline mr_dtype base_dtype(mr_dtype dt) { return dt & ~MR_PACKED; }
inline bool is_packed(mr_dtype dt) { return (dt & MR_PACKED) != 0; }
inline bool valid_dtype(mr_dtype dt) { return (dt & ~(MR_PACKED | 1)) == 0; }

inline bool debug_sync() {
  static const bool on = [] {
    const char* e = getenv("MR_DEBUG_SYNC");
    return e && e[0] == '1';
  }();
  return on;
}

// Check a launch; in debug mode also wait for it and report faults there.
inline mr_status check_launch(hipError_t e, hipStream_t s, const char* what) {
  if (e != hipSuccess) return hip_fail(e, what);
  if (debug_sync()) {
    e = hipStreamSynchronize(s);
    if (e != hipSuccess) return hip_fail(e, what);
  }
  return MR_OK;
}

// ------------------------------------------------------------ tracing
enum TraceClass {
  kTrSyrk, kTrJacobi, kTrStats, kTrBound, kTrInit, kTrNewton64, kTrNewton32, kTrConvert,
  kTrFinalize, kTrInfo, kTrNewtonX3, kTrCansBound, kTrCansInit, kTrCansP, kTrCansYZ, kTrCansFinal, kTrCansInfo,
  kTrPolarStats, kTrPolarBound, kTrPolarInit, kTrPolarA, kTrPolarX, kTrPolarFinal, kTrPolarInfo,
  kTrMomentum, kTrHyperReduce, kTrHyperUpdate, kTrApplyX3, kTrApplySplit, kTrSlice, kTrNewtonI8, kTrMoment,
  kTrNorm, kTrNormGrad, kTrQuantize, kTrScaledMatmul, kTrGrouped, kTrGroupedGrad,
  kTrLayerNorm, kTrLayerNormGrad, kTrRoute, kTrRouteGrad, kTrOrder, kTrDispatch, kTrCombine, kTrClipNorm,
  kTrClipScale, kTrCount
};
inline const char* const kTraceNames[kTrCount] = {"syrk_ema", "jacobi", "root_stats", "root_bound",
                                           "root_init", "newton_f64", "newton_f32", "newton_convert",
                                           "root_finalize", "root_info", "newton_x3", "cans_bound",
                                           "cans_init", "cans_p", "cans_yz", "cans_finalize", "cans_info",
                                           "polar_stats", "polar_bound", "polar_init", "polar_gram",
                                           "polar_update", "polar_finalize", "polar_info", "momentum",
                                           "hyperball_reduce", "hyperball_update", "apply_x3", "apply_split",
                                           "newton_slice", "newton_i8", "root_moment",
                                           "norm", "norm_grad", "quantize", "scaled_matmul", "grouped",
                                           "grouped_grad", "layer_norm", "layer_norm_grad", "route", "route_grad",
                                           "expert_order", "dispatch", "combine", "clip_norm", "clip_scale"};
struct TraceEntry {
  int cls;
  hipEvent_t a, b;
};
struct Trace {
  bool on = false;
  std::vector<hipEvent_t> pool;
  std::vector<TraceEntry> log;
  std::mutex mu;
  hipEvent_t get() {
    if (!pool.empty()) {
      hipEvent_t e = pool.back();
      pool.pop_back();
      return e;
    }
    hipEvent_t e = nullptr;
    if (hipEventCreate(&e) != hipSuccess) return nullptr;
    return e;
  }
};
inline Trace g_trace;

// Launch through `fn`; in trace mode bracket it with events on its stream.
template <class F>
inline mr_status traced(int cls, bool nonempty, hipStream_t s, F&& fn, const char* what) {
  if (!g_trace.on || !nonempty) return check_launch(fn(), s, what);
  std::lock_guard<std::mutex> lk(g_trace.mu);
  hipEvent_t a = g_trace.get(), b = g_trace.get();
  if (!a || !b) return fail(MR_ERR_HIP, "%s: hipEventCreate failed", what);
  hipError_t e = hipEventRecord(a, s);
  if (e == hipSuccess) e = fn();
  if (e == hipSuccess) e = hipEventRecord(b, s);
  g_trace.log.push_back({cls, a, b});
  return check_launch(e, s, what);
}

}  // namespace mr
