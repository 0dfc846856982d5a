// Host runtime of the linear-layer operators: argument validation
// (all-or-nothing, before anything is enqueued), workspace sizes, launches.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstring>

#include "host.hpp"
#include "linear.hpp"

using namespace mr;

namespace {

constexpr int64_t kMaxCols = 65536;
constexpr int64_t kMaxLd = int64_t(1) << 22;
constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int64_t kMaxExperts = 4096;

bool is_float(mr_dtype t) { return t == MR_F32 || t == MR_F16 || t == MR_BF16; }
bool is_half(mr_dtype t) { return t == MR_F16 || t == MR_BF16; }
bool is_eight(mr_dtype t) { return t == MR_E4M3 || t == MR_E5M2; }
size_t size_of(mr_dtype t) { return t == MR_F32 ? 4 : is_half(t) ? 2 : 1; }
int64_t blocks128(int64_t n) { return (n + kBlock - 1) / kBlock; }

// One matrix argument: present, leading dimension, alignment of its type.
mr_status check_matrix(const char* name, const void* p, int64_t cols, int64_t ld, size_t es) {
  if (!p) return fail(MR_ERR_NULL, "%s is NULL", name);
  if (ld < cols) return fail(MR_ERR_STRIDE, "%s: leading dimension %lld < %lld columns", name, (long long)ld, (long long)cols);
  if (ld > kMaxLd) return fail(MR_ERR_STRIDE, "%s: leading dimension %lld > %lld", name, (long long)ld, (long long)kMaxLd);
  if (!aligned(p, es)) return fail(MR_ERR_PARAM, "%s is not aligned to its type", name);
  return MR_OK;
}
mr_status check_size(const char* name, int64_t v, int64_t lo, int64_t hi) {
  if (v < lo || v > hi)
    return fail(MR_ERR_SHAPE, "%s %lld outside [%lld, %lld]", name, (long long)v, (long long)lo, (long long)hi);
  return MR_OK;
}
bool units16(const void* p, int64_t ld, size_t es) { return aligned(p, 16) && (ld * (int64_t)es) % 16 == 0; }

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
mr_status check_tiles(int64_t rows, int64_t cols, int64_t groups) {
  const int64_t t = (blocks128(rows) + groups) * blocks128(cols);
  return t < (int64_t(1) << 31) ? MR_OK : fail(MR_ERR_SHAPE, "%lld x %lld outputs in one call", (long long)rows, (long long)cols);
}

mr_status check_workspace(const void* ws, size_t bytes, size_t need) {
  if (need && (!ws || bytes < need || !aligned(ws, 256)))
    return fail(MR_ERR_WORKSPACE, "workspace %p of %zu bytes; need %zu bytes, 256-byte aligned", ws, bytes, need);
  return MR_OK;
}

}  // namespace

extern "C" {

// ------------------------------------------------------------------ norm
mr_status rms_norm_forward(const mr_rms_norm_problem* p, void* hip_stream) {
  if (!p) return fail(MR_ERR_NULL, "problem is NULL");
  MR_TRY(check_size("rows", p->rows, 0, kMaxRows));
  MR_TRY(check_size("width", p->width, 1, kNormMaxWidth));
  if (!is_float(p->dtype)) return fail(MR_ERR_PARAM, "dtype %d", p->dtype);
  if (p->w_dtype != p->dtype && p->w_dtype != MR_F32) return fail(MR_ERR_PARAM, "w_dtype %d", p->w_dtype);
  if (!(p->eps >= 0.0) || !std::isfinite(p->eps)) return fail(MR_ERR_PARAM, "eps %g must be >= 0 and finite", p->eps);
  if (p->rows > 0 && !p->y && !p->q) return fail(MR_ERR_NULL, "y and q are both NULL");
  if (!p->weight) return fail(MR_ERR_NULL, "weight is NULL");
  if (p->q && !is_eight(p->q_dtype)) return fail(MR_ERR_PARAM, "q_dtype %d", p->q_dtype);
  const size_t es = size_of(p->dtype), ws = size_of(p->w_dtype);
  if (!aligned(p->weight, ws)) return fail(MR_ERR_PARAM, "weight is not aligned to its type");
  if (p->rstd && !aligned(p->rstd, 4)) return fail(MR_ERR_PARAM, "rstd is not aligned to its type");
  const int64_t w = p->width, nb = blocks128(w);
  if (p->rows == 0) return MR_OK;
  MR_TRY(check_matrix("x", p->x, w, p->ldx, es));
  if (p->residual) {
    MR_TRY(check_matrix("residual", p->residual, w, p->ldres, es));
    MR_TRY(check_matrix("h", p->h, w, p->ldh, es));
  }
  if (p->y) MR_TRY(check_matrix("y", p->y, w, p->ldy, es));
  if (p->q) {
    MR_TRY(check_matrix("q", p->q, w, p->ldq, 1));
    MR_TRY(check_matrix("scales", p->scales, nb, p->lds, 4));
  }
  Aliases al;
  al.in("x", p->x, p->rows, w, p->ldx, es);
  al.in("residual", p->residual, p->rows, w, p->ldres, es);
  al.in("weight", p->weight, 1, w, w, ws);
  if (p->residual) al.out("h", p->h, p->rows, w, p->ldh, es);
  al.out("rstd", p->rstd, 1, p->rows, p->rows, 4);
  al.out("y", p->y, p->rows, w, p->ldy, es);
  al.out("q", p->q, p->rows, w, p->ldq, 1);
  if (p->q) al.out("scales", p->scales, p->rows, nb, p->lds, 4);
  MR_TRY(al.set.check());
  NormArgs a;
  memset(&a, 0, sizeof a);
  a.x = p->x, a.ldx = p->ldx;
  a.res = p->residual, a.ldres = p->ldres;
  a.w = p->weight, a.w_f32 = p->w_dtype == MR_F32;
  a.h = p->h, a.ldh = p->ldh;
  a.rstd = p->rstd;
  a.y = p->y, a.ldy = p->ldy;
  a.q = static_cast<unsigned char*>(p->q), a.ldq = p->ldq;
  a.s = p->scales, a.lds = p->lds;
  a.width = (int32_t)w, a.rows = p->rows, a.eps = (float)p->eps, a.e5m2 = p->q_dtype == MR_E5M2;
  hipStream_t s = reinterpret_cast<hipStream_t>(hip_stream);
  return traced(kTrNorm, true, s, [&] { return launch_norm_forward(a, p->dtype, s); }, "norm forward launch");
}

size_t rms_norm_backward_workspace(const mr_rms_norm_grad_problem* p) {
  if (!p || !p->dweight || p->rows < 1 || p->rows > kMaxRows || p->width < 1 || p->width > kNormMaxWidth) return 0;
  return align256((size_t)norm_backward_blocks(p->rows, p->width) * (size_t)p->width * sizeof(float));
}

mr_status rms_norm_backward(const mr_rms_norm_grad_problem* p, void* ws, size_t ws_bytes, void* hip_stream) {
  if (!p) return fail(MR_ERR_NULL, "problem is NULL");
  MR_TRY(check_size("rows", p->rows, 0, kMaxRows));
  MR_TRY(check_size("width", p->width, 1, kNormMaxWidth));
  if (!is_float(p->dtype)) return fail(MR_ERR_PARAM, "dtype %d", p->dtype);
  if (p->w_dtype != p->dtype && p->w_dtype != MR_F32) return fail(MR_ERR_PARAM, "w_dtype %d", p->w_dtype);
  if (!p->weight) return fail(MR_ERR_NULL, "weight is NULL");
  const size_t es = size_of(p->dtype), wes = size_of(p->w_dtype);
  if (!aligned(p->weight, wes)) return fail(MR_ERR_PARAM, "weight is not aligned to its type");
  if (p->dweight && !aligned(p->dweight, 4)) return fail(MR_ERR_PARAM, "dweight is not aligned to its type");
  const int64_t w = p->width;
  if (p->rows > 0) {
    MR_TRY(check_matrix("dy", p->dy, w, p->lddy, es));
    MR_TRY(check_matrix("h", p->h, w, p->ldh, es));
    if (!p->rstd) return fail(MR_ERR_NULL, "rstd is NULL");
    if (!aligned(p->rstd, 4)) return fail(MR_ERR_PARAM, "rstd is not aligned to its type");
    if (p->dresidual) MR_TRY(check_matrix("dresidual", p->dresidual, w, p->ldres, es));
    MR_TRY(check_matrix("dx", p->dx, w, p->lddx, es));
  }
  Aliases al;
  al.in("dy", p->dy, p->rows, w, p->lddy, es);
  al.in("h", p->h, p->rows, w, p->ldh, es);
  if (p->rows) al.in("rstd", p->rstd, 1, p->rows, p->rows, 4);
  al.in("weight", p->weight, 1, w, w, wes);
  al.in("dresidual", p->dresidual, p->rows, w, p->ldres, es);
  al.out("dx", p->dx, p->rows, w, p->lddx, es);
  al.out("dweight", p->dweight, 1, w, w, 4);
  const size_t need = rms_norm_backward_workspace(p);
  MR_TRY(check_workspace(ws, ws_bytes, need));
  if (need) al.out("workspace", ws, 1, (int64_t)need, (int64_t)need, 1);
  MR_TRY(al.set.check());
  hipStream_t s = reinterpret_cast<hipStream_t>(hip_stream);
  const int blocks = norm_backward_blocks(p->rows, w);
  float* partial = static_cast<float*>(need ? ws : nullptr);
  if (p->rows > 0) {
    NormArgs a;
    memset(&a, 0, sizeof a);
    a.dy = p->dy, a.lddy = p->lddy;
    a.x = p->h, a.ldx = p->ldh;
    a.rstd_in = p->rstd;
    a.w = p->weight, a.w_f32 = p->w_dtype == MR_F32;
    a.res = p->dresidual, a.ldres = p->ldres;
    a.y = p->dx, a.ldy = p->lddx;
    a.partial = partial;
    a.width = (int32_t)w, a.rows = p->rows;
    MR_TRY(traced(kTrNormGrad, true, s, [&] { return launch_norm_backward(a, p->dtype, blocks, s); },
                  "norm backward launch"));
  }
  if (!p->dweight) return MR_OK;
  return traced(kTrNormGrad, true, s, [&] { return launch_norm_weight_grad(partial, blocks, (int)w, p->dweight, s); },
                "norm weight gradient launch");
}

// -------------------------------------------------------------- quantise
mr_status quantize_blocks(const mr_quantize_problem* p, void* hip_stream) {
  if (!p) return fail(MR_ERR_NULL, "problem is NULL");
  MR_TRY(check_size("m", p->m, 0, kMaxRows));
  MR_TRY(check_size("n", p->n, 1, kMaxCols));
  if (!is_float(p->x_dtype)) return fail(MR_ERR_PARAM, "x_dtype %d", p->x_dtype);
  if (!is_eight(p->q_dtype)) return fail(MR_ERR_PARAM, "q_dtype %d", p->q_dtype);
  if (p->block != MR_BLOCK_VECTOR && p->block != MR_BLOCK_SQUARE) return fail(MR_ERR_PARAM, "block %d", p->block);
  if (p->m == 0) return MR_OK;
  if (!p->Q && !p->QT) return fail(MR_ERR_NULL, "Q and QT are both NULL");
  const size_t es = size_of(p->x_dtype);
  const int64_t mb = blocks128(p->m), nb = blocks128(p->n);
  const bool square = p->block == MR_BLOCK_SQUARE;
  // a workgroup of 512 threads for each; a launch has less than 2^32 threads
  if (mb * nb >= (int64_t(1) << 23)) return fail(MR_ERR_SHAPE, "%lld blocks of 128 x 128 in one call", (long long)(mb * nb));
  MR_TRY(check_matrix("X", p->X, p->n, p->ldx, es));
  Aliases al;
  al.in("X", p->X, p->m, p->n, p->ldx, es);
  if (p->Q) {
    MR_TRY(check_matrix("Q", p->Q, p->n, p->ldq, 1));
    MR_TRY(check_matrix("S", p->S, nb, p->lds, 4));
    al.out("Q", p->Q, p->m, p->n, p->ldq, 1);
    al.out("S", p->S, square ? mb : p->m, nb, p->lds, 4);
  }
  if (p->QT) {
    if (p->m > kMaxLd) return fail(MR_ERR_SHAPE, "m %lld > %lld for the transposed order", (long long)p->m, (long long)kMaxLd);
    MR_TRY(check_matrix("QT", p->QT, p->m, p->ldqt, 1));
    MR_TRY(check_matrix("ST", p->ST, mb, p->ldst, 4));
    al.out("QT", p->QT, p->n, p->m, p->ldqt, 1);
    al.out("ST", p->ST, square ? nb : p->n, mb, p->ldst, 4);
  }
  MR_TRY(al.set.check());
  QuantArgs a;
  memset(&a, 0, sizeof a);
  a.x = p->X, a.ldx = p->ldx;
  a.q = static_cast<unsigned char*>(p->Q), a.ldq = p->ldq, a.s = p->S, a.lds = p->lds;
  a.qt = static_cast<unsigned char*>(p->QT), a.ldqt = p->ldqt, a.st = p->ST, a.ldst = p->ldst;
  a.m = p->m, a.n = (int32_t)p->n;
  a.square = square, a.e5m2 = p->q_dtype == MR_E5M2;
  hipStream_t s = reinterpret_cast<hipStream_t>(hip_stream);
  return traced(kTrQuantize, true, s, [&] { return launch_quantize(a, p->x_dtype, s); }, "quantize launch");
}

// --------------------------------------------------- block-scaled product
size_t block_scaled_matmul_workspace(const mr_scaled_matmul_problem* p) {
  if (!p || p->m < 1 || p->m > kMaxRows || p->n < 1 || p->n > kMaxCols || p->k < 1 || p->k > kMaxLd) return 0;
  const ScaledPlan plan = scaled_plan(p->m, p->n, p->k);
  return plan.splits > 1 ? align256((size_t)plan.splits * (size_t)p->m * (size_t)p->n * sizeof(float)) : 0;
}

mr_status block_scaled_matmul(const mr_scaled_matmul_problem* p, void* ws, size_t ws_bytes, void* hip_stream) {
  if (!p) return fail(MR_ERR_NULL, "problem is NULL");
  MR_TRY(check_size("m", p->m, 0, kMaxRows));
  MR_TRY(check_size("n", p->n, 1, kMaxCols));
  MR_TRY(check_size("k", p->k, 1, kMaxLd));
  if (!is_eight(p->a_dtype)) return fail(MR_ERR_PARAM, "a_dtype %d", p->a_dtype);
  if (p->b_dtype == MR_E5M2) return fail(MR_ERR_UNSUPPORTED, "b_dtype MR_E5M2: B is MR_E4M3");
  if (p->b_dtype != MR_E4M3) return fail(MR_ERR_PARAM, "b_dtype %d", p->b_dtype);
  if (!is_float(p->c_dtype)) return fail(MR_ERR_PARAM, "c_dtype %d", p->c_dtype);
  for (const int32_t b : {p->a_block, p->b_block})
    if (b != MR_BLOCK_VECTOR && b != MR_BLOCK_SQUARE) return fail(MR_ERR_PARAM, "block %d", b);
  if (p->m == 0) return MR_OK;
  MR_TRY(check_tiles(p->m, p->n, 0));
  const int64_t kb = blocks128(p->k);
  const bool a_square = p->a_block == MR_BLOCK_SQUARE, b_square = p->b_block == MR_BLOCK_SQUARE;
  const size_t cs = size_of(p->c_dtype);
  MR_TRY(check_matrix("A", p->A, p->k, p->lda, 1));
  MR_TRY(check_matrix("B", p->B, p->k, p->ldb, 1));
  MR_TRY(check_matrix("SA", p->SA, kb, p->ldsa, 4));
  MR_TRY(check_matrix("SB", p->SB, kb, p->ldsb, 4));
  MR_TRY(check_matrix("C", p->C, p->n, p->ldc, cs));
  Aliases al;
  al.in("A", p->A, p->m, p->k, p->lda, 1);
  al.in("B", p->B, p->n, p->k, p->ldb, 1);
  al.in("SA", p->SA, a_square ? blocks128(p->m) : p->m, kb, p->ldsa, 4);
  al.in("SB", p->SB, b_square ? blocks128(p->n) : p->n, kb, p->ldsb, 4);
  al.out("C", p->C, p->m, p->n, p->ldc, cs);
  const size_t need = block_scaled_matmul_workspace(p);
  MR_TRY(check_workspace(ws, ws_bytes, need));
  if (need) al.out("workspace", ws, 1, (int64_t)need, (int64_t)need, 1);
  MR_TRY(al.set.check());
  const ScaledPlan plan = scaled_plan(p->m, p->n, p->k);
  ScaledArgs a;
  memset(&a, 0, sizeof a);
  a.p = static_cast<const unsigned char*>(p->B), a.ldp = p->ldb, a.sp = p->SB, a.ldsp = p->ldsb;
  a.q = static_cast<const unsigned char*>(p->A), a.ldq = p->lda, a.sq = p->SA, a.ldsq = p->ldsa;
  a.c = p->C, a.ldc = p->ldc, a.c_type = p->c_dtype;
  a.partial = static_cast<float*>(need ? ws : nullptr);
  a.m = p->m, a.n = (int32_t)p->n, a.k = (int32_t)p->k;
  a.p_shift = b_square ? 7 : 0, a.q_shift = a_square ? 7 : 0;
  a.fast = units16(p->A, p->lda, 1) && units16(p->B, p->ldb, 1) && (p->k % 16 == 0 || p->padded);
  a.q_e5m2 = p->a_dtype == MR_E5M2;
  a.accumulate = p->accumulate != 0;
  a.vec_c = units16(p->C, p->ldc, cs);
  a.splits = plan.splits;
  hipStream_t s = reinterpret_cast<hipStream_t>(hip_stream);
  MR_TRY(traced(kTrScaledMatmul, true, s, [&] { return launch_scaled(a, plan, s); }, "block-scaled product launch"));
  if (plan.splits == 1) return MR_OK;
  return traced(kTrScaledMatmul, true, s, [&] { return launch_scaled_join(a, s); }, "block-scaled join launch");
}

// -------------------------------------------------------- grouped products
static mr_status check_grouped(int64_t experts, int64_t rows, int64_t n, int64_t k, mr_dtype dt, mr_dtype out_dt,
                               int32_t offset_bits, const void* offsets) {
  MR_TRY(check_size("experts", experts, 1, kMaxExperts));
  MR_TRY(check_size("rows", rows, 0, kMaxRows));
  MR_TRY(check_size("n", n, 1, kMaxCols));
  MR_TRY(check_size("k", k, 1, kMaxCols));
  if (!is_half(dt)) return fail(MR_ERR_PARAM, "dtype %d: MR_F16 or MR_BF16", dt);
  if (out_dt != dt && out_dt != MR_F32) return fail(MR_ERR_PARAM, "output dtype %d: dtype or MR_F32", out_dt);
  if (offset_bits != 32 && offset_bits != 64) return fail(MR_ERR_PARAM, "offset_bits %d: 32 or 64", offset_bits);
  if (!offsets) return fail(MR_ERR_NULL, "offsets is NULL");
  if (!aligned(offsets, offset_bits / 8)) return fail(MR_ERR_PARAM, "offsets is not aligned to its type");
  return MR_OK;
}

mr_status grouped_matmul(const mr_grouped_problem* p, void* hip_stream) {
  if (!p) return fail(MR_ERR_NULL, "problem is NULL");
  MR_TRY(check_grouped(p->experts, p->rows, p->n, p->k, p->dtype, p->y_dtype, p->offset_bits, p->offsets));
  if (p->transpose != 0 && p->transpose != 1) return fail(MR_ERR_PARAM, "transpose %d", p->transpose);
  const int64_t in = p->transpose ? p->n : p->k, out = p->transpose ? p->k : p->n;
  MR_TRY(check_matrix("W", p->W, p->k, p->ldw, 2));
  if (p->w_stride < (p->n - 1) * p->ldw + p->k)
    return fail(MR_ERR_STRIDE, "w_stride %lld: the experts' weights overlap", (long long)p->w_stride);
  if (p->rows == 0) return MR_OK;
  MR_TRY(check_tiles(p->rows, out, p->experts + 2));
  const size_t ys = size_of(p->y_dtype);
  MR_TRY(check_matrix("X", p->X, in, p->ldx, 2));
  MR_TRY(check_matrix("Y", p->Y, out, p->ldy, ys));
  Aliases al;
  al.in("X", p->X, p->rows, in, p->ldx, 2);
  al.in("W", p->W, p->experts, (p->n - 1) * p->ldw + p->k, p->w_stride, 2);
  al.in("offsets", p->offsets, 1, p->experts + 1, p->experts + 1, p->offset_bits / 8);
  al.out("Y", p->Y, p->rows, out, p->ldy, ys);
  MR_TRY(al.set.check());
  GroupedArgs a;
  memset(&a, 0, sizeof a);
  a.x = p->X, a.ldx = p->ldx;
  a.w = p->W, a.ldw = p->ldw, a.w_stride = p->w_stride;
  a.y = p->Y, a.ldy = p->ldy;
  a.offsets = p->offsets, a.wide_offsets = p->offset_bits == 64;
  a.rows = p->rows, a.experts = (int32_t)p->experts, a.n = (int32_t)p->n, a.k = (int32_t)p->k;
  a.fast = units16(p->X, p->ldx, 2) && units16(p->W, p->ldw, 2) && (p->w_stride % 8 == 0 || p->experts == 1) &&
           p->k % 8 == 0 && (!p->transpose || p->n % 8 == 0);
  a.vec_y = units16(p->Y, p->ldy, ys);
  a.y_f32 = p->y_dtype == MR_F32;
  hipStream_t s = reinterpret_cast<hipStream_t>(hip_stream);
  return traced(kTrGrouped, true, s, [&] { return launch_grouped(a, p->dtype, p->transpose, s); }, "grouped product launch");
}

mr_status grouped_weight_grad(const mr_grouped_grad_problem* p, void* hip_stream) {
  if (!p) return fail(MR_ERR_NULL, "problem is NULL");
  MR_TRY(check_grouped(p->experts, p->rows, p->n, p->k, p->dtype, p->dw_dtype, p->offset_bits, p->offsets));
  MR_TRY(check_size("experts x tiles", p->experts * blocks128(p->n) * blocks128(p->k), 1, (int64_t(1) << 31) - 1));
  const size_t ds = size_of(p->dw_dtype);
  MR_TRY(check_matrix("DW", p->DW, p->k, p->lddw, ds));
  if (p->dw_stride < (p->n - 1) * p->lddw + p->k)
    return fail(MR_ERR_STRIDE, "dw_stride %lld: the experts' gradients overlap", (long long)p->dw_stride);
  if (p->rows > 0) {
    MR_TRY(check_matrix("DY", p->DY, p->n, p->lddy, 2));
    MR_TRY(check_matrix("X", p->X, p->k, p->ldx, 2));
  }
  Aliases al;
  al.in("DY", p->DY, p->rows, p->n, p->lddy, 2);
  al.in("X", p->X, p->rows, p->k, p->ldx, 2);
  al.in("offsets", p->offsets, 1, p->experts + 1, p->experts + 1, p->offset_bits / 8);
  al.out("DW", p->DW, p->experts, (p->n - 1) * p->lddw + p->k, p->dw_stride, ds);
  MR_TRY(al.set.check());
  GroupedArgs a;
  memset(&a, 0, sizeof a);
  a.x = p->DY, a.ldx = p->lddy;
  a.w = p->X, a.ldw = p->ldx;
  a.y = p->DW, a.ldy = p->lddw, a.y_stride = p->dw_stride;
  a.offsets = p->offsets, a.wide_offsets = p->offset_bits == 64;
  a.rows = p->rows, a.experts = (int32_t)p->experts, a.n = (int32_t)p->n, a.k = (int32_t)p->k;
  a.fast = units16(p->DY, p->lddy, 2) && units16(p->X, p->ldx, 2) && p->n % 8 == 0 && p->k % 8 == 0;
  a.y_f32 = p->dw_dtype == MR_F32;
  a.accumulate = p->accumulate != 0;
  hipStream_t s = reinterpret_cast<hipStream_t>(hip_stream);
  return traced(kTrGroupedGrad, true, s, [&] { return launch_grouped_weight_grad(a, p->dtype, s); },
                "grouped weight gradient launch");
}

}  // extern "C"
