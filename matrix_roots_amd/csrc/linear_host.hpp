// Argument checks shared by the host runtimes of the linear-layer operators
// (linear.cpp) and of the operators around a bank of experts (experts.cpp).
#pragma once

#include "host.hpp"
#include "linear.hpp"

namespace mr {

constexpr int64_t kMaxCols = 65536;
constexpr int64_t kMaxLd = int64_t(1) << 22;
constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int64_t kMaxExperts = 4096;

inline bool is_float(mr_dtype t) { return t == MR_F32 || t == MR_F16 || t == MR_BF16; }
inline bool is_half(mr_dtype t) { return t == MR_F16 || t == MR_BF16; }
inline bool is_eight(mr_dtype t) { return t == MR_E4M3 || t == MR_E5M2; }
inline size_t size_of(mr_dtype t) { return t == MR_F32 ? 4 : is_half(t) ? 2 : 1; }
inline int64_t blocks128(int64_t n) { return (n + kBlock - 1) / kBlock; }

// One matrix argument: present, leading dimension, alignment of its type.
inline mr_status check_matrix(const char* name, const void* p, int64_t cols, int64_t ld, size_t es) {
  if (!p) return fail(MR_ERR_NULL, "%s is NULL", name);
  if (ld < cols) return fail(MR_ERR_STRIDE, "%s: leading dimension %lld < %lld columns", name, (long long)ld, (long long)cols);
  if (ld > kMaxLd) return fail(MR_ERR_STRIDE, "%s: leading dimension %lld > %lld", name, (long long)ld, (long long)kMaxLd);
  if (!aligned(p, es)) return fail(MR_ERR_PARAM, "%s is not aligned to its type", name);
  return MR_OK;
}
inline mr_status check_size(const char* name, int64_t v, int64_t lo, int64_t hi) {
  if (v < lo || v > hi)
    return fail(MR_ERR_SHAPE, "%s %lld outside [%lld, %lld]", name, (long long)v, (long long)lo, (long long)hi);
  return MR_OK;
}
inline bool units16(const void* p, int64_t ld, size_t es) { return aligned(p, 16) && (ld * (int64_t)es) % 16 == 0; }

#define MR_TRY(x)                            \
  do {                                       \
    const mr_status st_ = (x);               \
    if (st_ != MR_OK) return st_;            \
  } while (0)

// Alias set whose matrices may have no rows.
struct Aliases {
  AliasSet set;
  void out(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld, size_t es) {
    if (p && rows > 0) set.out(range_of(p, rows, cols, ld, es), 0, name);
  }
  void in(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld, size_t es) {
    if (p && rows > 0) set.in(range_of(p, rows, cols, ld, es), 0, name);
  }
};

// The launch's 128 x 128 tiles (with one ragged tile more for each group) fit a grid.
inline mr_status check_tiles(int64_t rows, int64_t cols, int64_t groups) {
  const int64_t t = (blocks128(rows) + groups) * blocks128(cols);
  return t < (int64_t(1) << 31) ? MR_OK : fail(MR_ERR_SHAPE, "%lld x %lld outputs in one call", (long long)rows, (long long)cols);
}

inline mr_status check_workspace(const void* ws, size_t bytes, size_t need) {
  if (need && (!ws || bytes < need || !aligned(ws, 256)))
    return fail(MR_ERR_WORKSPACE, "workspace %p of %zu bytes; need %zu bytes, 256-byte aligned", ws, bytes, need);
  return MR_OK;
}

}  // namespace mr
