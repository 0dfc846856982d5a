// The operators around a bank of experts (routing, order by expert, rows to
// their experts and back): launch descriptors shared by the host runtime
// (experts.cpp) and routing.hip.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/matrix_roots.h"

namespace mr {

constexpr int kMaxRouted = 16;        // experts a token goes to (the lanes of a DPP row)
constexpr int kMaxRouteExperts = 4096;  // a token's logits stay in one wave's registers
constexpr int kMaxChoices = 64;       // choices a token has in an order: one lane of a wave each

struct RouteArgs {
  const void* logits;
  int64_t ldl;
  int32_t* experts;   // tokens x k
  float* weights;     // tokens x k
  float* log_sum;     // tokens
  int64_t tokens;
  int32_t n, k;
  int32_t normalize;
};
hipError_t launch_route(const RouteArgs& a, mr_dtype dt, hipStream_t s);

struct RouteGradArgs {
  const void* logits;
  int64_t ldl;
  const int32_t* experts;
  const float* weights;
  const float* dweights;
  void* dlogits;
  int64_t ldd;
  int64_t tokens;
  int32_t n, k;
  int32_t normalize;
};
hipError_t launch_route_grad(const RouteGradArgs& a, mr_dtype dt, hipStream_t s);

struct OrderArgs {
  const void* experts;  // tokens x k, int32 or int64
  int64_t lde;
  int32_t wide;
  int32_t k, n;
  int32_t total;        // tokens k
  int32_t chunk, blocks;  // choices per workgroup, workgroups
  int32_t waves;        // of a workgroup
  int32_t* offsets;     // n + 1
  int32_t* place;       // tokens x k
  int32_t* counts;      // blocks > 1: blocks x (n + 1)
};
// chunk, blocks and waves of an order of `total` choices among n experts
void order_plan(int64_t total, int64_t n, int32_t* chunk, int32_t* blocks, int32_t* waves);
hipError_t launch_order(const OrderArgs& a, hipStream_t s);

struct RowsArgs {
  const void* x;           // tokens x width: dispatched; combine: residual (may be null)
  const void* rows;        // sorted rows that are read (combine; dispatch: for `dots`, may be null)
  void* out;               // dispatch: sorted rows; combine: tokens x width
  const int32_t* place;    // tokens x k
  const int32_t* offsets;  // experts + 1
  const float* weights;    // tokens x k, may be null
  float* dots;             // tokens x k, dispatch with `rows`
  int64_t ldx, ldr, ldo;
  int64_t tokens;
  int32_t width, k, experts;
};
hipError_t launch_dispatch(const RowsArgs& a, mr_dtype dt, hipStream_t s);
hipError_t launch_combine(const RowsArgs& a, mr_dtype dt, hipStream_t s);

}  // namespace mr
