// Clipping of gradients by their common norm: launch descriptors shared by the
// host runtime (experts.cpp) and clip.hip.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/matrix_roots.h"

namespace mr {

// The gradients of a launch, in its arguments (under 4 KB): contiguous ones, and
// ones whose rows lie `ldg` apart.  A workgroup finds its own by `begin`.
struct ClipFlat {
  static constexpr int kJobs = 104;
  static constexpr bool kRows = false;
  const void* g[kJobs];
  void* out[kJobs];       // g itself where it is scaled in place
  int64_t cols[kJobs];    // values of a row
  int32_t begin[kJobs];   // first workgroup of the launch
  int32_t problem[kJobs];
  uint8_t type[kJobs];    // mr_dtype of g, and four bits up of out
};
struct ClipRows {
  static constexpr int kJobs = 60;
  static constexpr bool kRows = true;
  const void* g[kJobs];
  void* out[kJobs];
  int64_t cols[kJobs];
  int32_t begin[kJobs];
  int32_t problem[kJobs];
  uint8_t type[kJobs];
  int64_t rows[kJobs], ldg[kJobs], ldo[kJobs];
};
template <typename Jobs>
struct ClipBatch {
  Jobs job;
  double* partial;     // a sum of squares for each workgroup of the call
  const double* sums;  // what the whole call's sum is made of: the partial sums, or one sum of them
  double* norms;       // of everything, then of each gradient
  double max_norm;
  int64_t per;         // units of a workgroup: eight values of a row, or the last ones
  int32_t nsums;
  int32_t slot;        // of this launch's first workgroup among the call's
  int32_t njobs, blocks;
};
static_assert(sizeof(ClipBatch<ClipFlat>) <= 4096 && sizeof(ClipBatch<ClipRows>) <= 4096, "kernel arguments");

template <typename Jobs>
hipError_t launch_clip_squares(const ClipBatch<Jobs>& b, hipStream_t s);
template <typename Jobs>
hipError_t launch_clip_scale(const ClipBatch<Jobs>& b, hipStream_t s);
hipError_t launch_clip_fold(const double* partial, int slots, double* sum, hipStream_t s);

}  // namespace mr
