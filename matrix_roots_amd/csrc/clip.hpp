// Clipping of gradients by their common norm: launch descriptors shared by the
// host runtime (experts.cpp) and clip.hip.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/matrix_roots.h"

namespace mr {

// rows x cols values in rows `ldg` apart (contiguous ones are one row).
struct ClipJob {
  const void* g;
  void* out;              // g itself where it is scaled in place
  int64_t rows, cols;
  int64_t ldg, ldo;
  int32_t block_begin;    // this job's first workgroup of the launch
  int32_t slot;           // its partial sum's place of the call
  int32_t dtype, out_dtype;
};
constexpr int kMaxClipJobs = 48;
struct ClipBatch {
  ClipJob job[kMaxClipJobs];
  double* partial;        // a sum of squares for each workgroup of the call
  int32_t* first;         // each gradient's first partial sum
  double* by;             // the factor
  int64_t per_block;      // units of a workgroup: eight values of a row, or the last ones
  int32_t njobs, total_blocks;
  int32_t first_problem;  // of this launch's first job in the call
};
hipError_t launch_clip_squares(const ClipBatch& b, hipStream_t s);
// norms[0]: of everything, norms[1 + i]: of gradient i
hipError_t launch_clip_norms(const double* partial, const int32_t* first, int count, int slots, double max_norm,
                             double* norms, double* by, hipStream_t s);
hipError_t launch_clip_scale(const ClipBatch& b, hipStream_t s);

}  // namespace mr
