// Internal launch interface of the operators of a transformer block (include/bsq_block.h) between the C ABI
// (bsq_block.cpp) and the kernels. Arguments are validated by the caller; each function enqueues its kernels on `s`
// and returns the launch status.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bsq_block.h"
#include "bsq_launch.hpp"
#include "row_groups.hpp"
#include "serve_launch.hpp"

namespace bsq {

// the axis of each rotated pair
struct RopeAxes {
  int64_t pos_t, pos_a;  // strides of the positions
  int axes;
  bool cycled;
  int sections[4];
};
hipError_t launch_rope_axes(bsq_dtype dt, Strided x, const int64_t* positions, const RopeAxes& axes, Rotation r,
                            bool backward, Strided y, int64_t T, int H, int D, hipStream_t s);

// a row vector for each group, or null
struct GroupVector {
  const void* p;
  int64_t stride;
};
struct NormArgs {
  int norm, post;  // bsq_norm
  float eps, post_eps;
  int rows, dim;
  RowGroups groups;
  const void *weight, *bias, *post_weight;
  GroupVector scale, shift, gate;
};
struct Rows {
  void* p;
  int64_t stride;
};
struct NormForward {
  NormArgs n;
  Rows x, branch, x_out, y;
  int out_format;  // 0, BSQ_FMT_FP8R, BSQ_FMT_NVFP4
  const float* y_global;
  void* y_scale;
};
hipError_t launch_block_norm(bsq_dtype dt, const NormForward& a, hipStream_t s);

struct NormBackward {
  NormArgs n;
  Rows dy, dx_out, x_out, branch, dx, dbranch;
  float *dscale, *dshift, *dgate, *dweight, *dbias, *dpost_weight;
};
size_t block_norm_workspace(int64_t rows, int64_t dim, int64_t groups);
hipError_t launch_block_norm_backward(bsq_dtype dt, const NormBackward& a, void* workspace, hipStream_t s);

// What a linear with an epilogue does with its scaled sums: residual + gate[g(m)] * act(v + bias)
struct Epilogue {
  const uint16_t* bias;  // [N] or null
  const uint16_t* gate;  // [groups] rows gate_stride apart, or null
  int64_t gate_stride;
  const uint16_t* residual;  // [M] rows residual_stride apart, or null
  int64_t residual_stride;
  RowGroups groups;
  int act;  // bsq_act
};
// the few-token kernels (W8A8, W4A4), the tiled W8A8 ones, the tiled W4A4 ones (K % 256 == 0, and any other K)
hipError_t launch_gemm_skinny_epilogue(DecMode mode, const DecArgs& a, const Epilogue& ep, hipStream_t s);
hipError_t launch_gemm_fp8_epilogue(const DecArgs& a, const Epilogue& ep, hipStream_t s);
hipError_t launch_gemm_w4a4_epilogue(const DecArgs& a, const Epilogue& ep, hipStream_t s);
hipError_t launch_gemm_w4a4_any_epilogue(const DecArgs& a, const Epilogue& ep, hipStream_t s);

}  // namespace bsq
