// The operators around a linear layer (norm, quantisation, block-scaled and
// expert-grouped products): launch descriptors shared by the host runtime
// (linear.cpp) and the kernels.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/matrix_roots.h"

namespace mr {

constexpr int kBlock = 128;             // values per scale along a blocked axis
constexpr int kNormMaxWidth = 16384;    // a row of the norm stays in one workgroup's registers
constexpr float kSmallestAmax = 7.888609052210118e-31f;  // 2^-100
constexpr float kE4m3Max = 448.f, kE5m2Max = 57344.f;

struct NormArgs {
  const void* x;
  const void* res;   // forward: residual; backward: gradient down the residual (either may be null)
  const void* w;
  const void* dy;    // backward
  const float* rstd_in;
  void* h;
  float* rstd;
  void* y;           // backward: dx
  unsigned char* q;
  float* s;
  float* partial;    // backward: one row of `width` sums per workgroup
  int64_t ldx, ldres, lddy, ldh, ldy, ldq, lds;
  int32_t width;
  int64_t rows;
  float eps;
  int32_t w_f32;     // the weight is float32 (else of x's type)
  int32_t e5m2;
};
hipError_t launch_norm_forward(const NormArgs& a, mr_dtype dt, hipStream_t s);
// `blocks` workgroups (norm_backward_blocks), their column sums in a.partial
hipError_t launch_norm_backward(const NormArgs& a, mr_dtype dt, int blocks, hipStream_t s);
hipError_t launch_norm_weight_grad(const float* partial, int blocks, int width, float* dweight, hipStream_t s);
int norm_backward_blocks(int64_t rows, int64_t width);

struct QuantArgs {
  const void* x;
  unsigned char* q;
  float* s;
  unsigned char* qt;
  float* st;
  int64_t ldx, ldq, lds, ldqt, ldst;
  int64_t m;
  int32_t n;
  int32_t square, e5m2;
};
hipError_t launch_quantize(const QuantArgs& a, mr_dtype dt, hipStream_t s);

// C (m x n) = A B^T with block scales.  In the kernels "P" is the operand on
// the matrix instruction's rows (B: a lane holds four consecutive columns of
// C) and "Q" the one on its columns (A: a row of C per lane).
struct ScaledArgs {
  const unsigned char* p;  // B: n x k
  const unsigned char* q;  // A: m x k
  const float* sp;
  const float* sq;
  void* c;
  float* partial;          // split k: splits x m x n float32 (null: write c)
  int64_t ldp, ldq, ldsp, ldsq, ldc;
  int64_t m;
  int32_t n, k;
  int32_t p_shift;         // P's scales: row >> p_shift (0: one per row, 7: per 128 rows)
  int32_t q_shift;         // Q's scales: row >> q_shift (0: one per row, 7: per 128 rows)
  int32_t fast;            // both operands in whole 16-byte units at 16-byte addresses
  int32_t q_e5m2;
  int32_t c_type;          // mr_dtype
  int32_t accumulate;
  int32_t vec_c;           // rows of C take four-element stores
  int32_t splits;
};
struct ScaledPlan {
  int kind;    // 0: few rows (no LDS tile), 1: 128 x 128 tiles, 2: tiles of 256 columns x 128 rows
  int splits;  // parts of k
};
ScaledPlan scaled_plan(int64_t m, int64_t n, int64_t k);
hipError_t launch_scaled(const ScaledArgs& a, const ScaledPlan& plan, hipStream_t s);
hipError_t launch_scaled_join(const ScaledArgs& a, hipStream_t s);

// Products of rows grouped by expert, 16-bit operands.
struct GroupedArgs {
  const void* x;       // Q: rows (the gradient of the outputs for transpose and for the weights' gradient)
  const void* w;       // P: experts' weights; the weights' gradient: the layer's input rows
  void* y;
  const void* offsets;
  int64_t ldx, ldw, w_stride, ldy, y_stride;
  int64_t rows;
  int32_t experts, n, k;
  int32_t wide_offsets;  // 64-bit offsets
  int32_t fast;          // operands in whole 16-byte units at 16-byte addresses
  int32_t vec_y;
  int32_t y_f32;
  int32_t accumulate;
  int32_t ahead;  // the weights' gradient reads its operands once before its tiles (its launcher says)
};
// dt: MR_F16 or MR_BF16
hipError_t launch_grouped(const GroupedArgs& a, mr_dtype dt, bool transpose, hipStream_t s);
hipError_t launch_grouped_weight_grad(const GroupedArgs& a, mr_dtype dt, hipStream_t s);

}  // namespace mr
