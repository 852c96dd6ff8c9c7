// rope_kernels.h -- host-side launchers of the position rotation, and the views
// they take (internal).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

#include "dsa_kernels.h"

namespace dsa {

// A table of cosines and sines, fp32 [positions][dims], rows `stride` apart:
// cosines in columns 0 .. dims/2-1, sines behind them.  dims 0: no rotation.
struct RopeView {
  const float* cs;
  int64_t positions, stride;
  int dims;   // a multiple of 16
  int inter;  // pairs (2j, 2j + 1) instead of (j, j + dims/2)
};

// x bf16 [rows][heads][D], rows x_stride elements apart, to out (rows
// out_stride apart): row r turned by the table's row positions[r], or begin + r.
struct RopeArgs {
  const __nv_bfloat16* x;
  __nv_bfloat16* out;
  int64_t x_stride, out_stride;
  int64_t rows;
  int heads, D;
  const int32_t* positions;  // or null
  int64_t begin;
  float dir;                 // 1, or -1: the inverse
};
cudaError_t launch_rope(const RopeView& r, const RopeArgs& a, const LaunchCtx& ctx);

}  // namespace dsa
