// C ABI of the operators of a transformer block (declared in include/bsq_block.h): argument checks on the host, then
// the launches.
#include "bsq_block.h"

#include <cmath>

#include "block_launch.hpp"

namespace {

constexpr int64_t kMaxStride = (int64_t)1 << 40;
constexpr int64_t kMaxRows = (int64_t)1 << 30;
constexpr int64_t kMaxGroups = (int64_t)1 << 24;

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bsq_status finish(hipError_t e) { return e == hipSuccess ? BSQ_OK : bsq::hip_failure(e); }

bsq_status check_groups(int64_t rows, int64_t groups, const int32_t* starts) {
  if (groups < 1 || groups > kMaxGroups) return BSQ_ERR_SHAPE;
  if (!starts && rows % groups != 0) return BSQ_ERR_SHAPE;
  return aligned(starts, 4) ? BSQ_OK : BSQ_ERR_ALIGN;
}
bsq::RowGroups groups_of(int64_t rows, int64_t groups, const int32_t* starts, bool vectors) {
  if (!vectors) return bsq::RowGroups{starts, 1, (int)rows, (int)rows, (int)groups};
  return bsq::RowGroups{starts, (int)groups, (int)(rows / groups), (int)rows, (int)groups};
}

// ---- block norms ---------------------------------------------------------------------

bool norm_ok(bsq_norm n) { return n == BSQ_NORM_NONE || n == BSQ_NORM_LAYER || n == BSQ_NORM_RMS; }
bool stride_ok(int64_t stride, int64_t dim, int64_t rows, bool input) {
  if (stride < 0 || stride >= kMaxStride || stride % 8 != 0) return false;
  return rows <= 1 || stride >= dim || (input && stride == 0);
}

// the descriptor: shapes and arguments
bsq_status check_block(const bsq_block* b) {
  if (!b) return BSQ_ERR_NULL;
  if (b->dtype != BSQ_BF16 && b->dtype != BSQ_FP16 && b->dtype != BSQ_FP32) return BSQ_ERR_ARG;
  if (!norm_ok(b->norm) || !norm_ok(b->post)) return BSQ_ERR_ARG;
  if (!(b->eps >= 0.0f) || !std::isfinite(b->eps) || !(b->post_eps >= 0.0f) || !std::isfinite(b->post_eps))
    return BSQ_ERR_ARG;
  if (b->norm == BSQ_NORM_NONE && (b->weight || b->bias || b->scale || b->shift)) return BSQ_ERR_ARG;
  if (b->post == BSQ_NORM_NONE && b->post_weight) return BSQ_ERR_ARG;
  if (b->rows < 0 || b->rows > kMaxRows || b->dim < 8 || b->dim > 16384 || b->dim % 8 != 0) return BSQ_ERR_SHAPE;
  bsq_status st = check_groups(b->rows, b->groups, b->group_starts);
  if (st != BSQ_OK) return st;
  if (b->scale && !stride_ok(b->scale_stride, b->dim, b->groups, false)) return BSQ_ERR_SHAPE;
  if (b->shift && !stride_ok(b->shift_stride, b->dim, b->groups, false)) return BSQ_ERR_SHAPE;
  if (b->gate && !stride_ok(b->gate_stride, b->dim, b->groups, false)) return BSQ_ERR_SHAPE;
  for (const void* p : {b->weight, b->bias, b->post_weight, b->scale, b->shift, b->gate})
    if (!aligned(p, 16)) return BSQ_ERR_ALIGN;
  return BSQ_OK;
}
bsq::NormArgs norm_args(const bsq_block* b) {
  bsq::NormArgs n{};
  n.norm = b->norm; n.post = b->post; n.eps = b->eps; n.post_eps = b->post_eps;
  n.rows = (int)b->rows; n.dim = (int)b->dim;
  n.groups = groups_of(b->rows, b->groups, b->group_starts, b->scale || b->shift || b->gate);
  n.weight = b->weight; n.bias = b->bias; n.post_weight = b->post_weight;
  n.scale = bsq::GroupVector{b->scale, b->scale_stride};
  n.shift = bsq::GroupVector{b->shift, b->shift_stride};
  n.gate = bsq::GroupVector{b->gate, b->gate_stride};
  return n;
}
bsq::Rows rows_of(const void* p, int64_t stride) { return bsq::Rows{const_cast<void*>(p), stride}; }

// the threads of a forward launch (block_norm.hip has one workgroup a row, or four rows of up to 512) stay below 2^31;
// the gradient has at most twelve workers a compute unit, whatever the rows
bool launch_fits(int64_t rows, int64_t dim) {
  const int64_t waves = dim <= 2048 ? (dim + 511) / 512 : (dim + 1023) / 1024;
  return rows * waves * 64 < ((int64_t)1 << 31) - 256;
}

}  // namespace

extern "C" {

bsq_status bsq_rope_axes(bsq_dtype dtype, const void* x, int64_t x_stride_t, int64_t x_stride_h,
                         const int64_t* positions, int64_t pos_stride_t, int64_t pos_stride_a, const int64_t* sections,
                         int64_t axes, bsq_axes_order order, const float* inv_freq, bsq_rope_layout layout,
                         float attn_factor, uint32_t flags, void* y, int64_t y_stride_t, int64_t y_stride_h, int64_t T,
                         int64_t H, int64_t D, hipStream_t stream) {
  if (order != BSQ_AXES_BLOCKS && order != BSQ_AXES_CYCLED) return BSQ_ERR_ARG;
  if (axes < 1 || axes > 4) return BSQ_ERR_SHAPE;
  if (!sections) return BSQ_ERR_NULL;
  if (pos_stride_t < 0 || pos_stride_a < 0 || pos_stride_t >= kMaxStride || pos_stride_a >= kMaxStride)
    return BSQ_ERR_SHAPE;
  int64_t pairs = 0;
  for (int64_t c = 0; c < axes; ++c) {
    if (sections[c] < 0 || sections[c] > 512) return BSQ_ERR_SHAPE;
    pairs += sections[c];
  }
  for (int64_t c = 1; c < axes && order == BSQ_AXES_CYCLED; ++c)
    if (sections[c] > 0 && axes * (sections[c] - 1) + c >= pairs) return BSQ_ERR_SHAPE;
  const bsq_status st = bsq::check_rope(dtype, x, x_stride_t, x_stride_h, positions, inv_freq, 2 * pairs, layout,
                                        attn_factor, flags, y, y_stride_t, y_stride_h, T, H, D);
  if (st != BSQ_OK || T == 0 || H == 0) return st;
  bsq::RopeAxes a{};
  a.pos_t = pos_stride_t;
  a.pos_a = pos_stride_a;
  a.axes = (int)axes;
  a.cycled = order == BSQ_AXES_CYCLED;
  for (int64_t c = 0; c < axes; ++c) a.sections[c] = (int)sections[c];
  return finish(bsq::launch_rope_axes(dtype, bsq::Strided{x, x_stride_t, x_stride_h}, positions, a,
                                      bsq::Rotation{inv_freq, (int)(2 * pairs), layout == BSQ_ROPE_INTERLEAVED,
                                                    attn_factor},
                                      (flags & BSQ_ROPE_BACKWARD) != 0, bsq::Strided{y, y_stride_t, y_stride_h}, T,
                                      (int)H, (int)D, stream));
}

bsq_status bsq_block_norm(const bsq_block* b, const void* x, int64_t x_stride, const void* branch,
                          int64_t branch_stride, void* x_out, int64_t x_out_stride, int out_format,
                          const float* y_global, void* y, int64_t y_stride, void* y_scale, hipStream_t stream) {
  bsq_status st = check_block(b);
  if (st != BSQ_OK) return st;
  if (out_format != 0 && out_format != BSQ_FMT_FP8R && out_format != BSQ_FMT_NVFP4) return BSQ_ERR_ARG;
  const bool encoded = out_format != 0, normed = b->norm != BSQ_NORM_NONE;
  if (!branch && (b->gate || x_out || b->post != BSQ_NORM_NONE)) return BSQ_ERR_ARG;
  if (!normed && (encoded || y)) return BSQ_ERR_ARG;
  if ((!encoded && y_scale) || (out_format != BSQ_FMT_NVFP4 && y_global)) return BSQ_ERR_ARG;
  if (encoded && b->dim % 32 != 0) return BSQ_ERR_SHAPE;
  if (!stride_ok(x_stride, b->dim, b->rows, true) || (branch && !stride_ok(branch_stride, b->dim, b->rows, true)) ||
      (x_out && !stride_ok(x_out_stride, b->dim, b->rows, false)) ||
      (normed && !encoded && !stride_ok(y_stride, b->dim, b->rows, false)))
    return BSQ_ERR_SHAPE;
  if (x_out && x_out == x && b->rows > 1 && x_out_stride != x_stride) return BSQ_ERR_SHAPE;
  if (!launch_fits(b->rows, b->dim)) return BSQ_ERR_SHAPE;
  if (b->rows == 0) return BSQ_OK;
  if (!x || (normed && !y) || (!normed && !x_out) || (encoded && !y_scale) ||
      (out_format == BSQ_FMT_NVFP4 && !y_global))
    return BSQ_ERR_NULL;
  for (const void* p : {x, branch, (const void*)x_out, (const void*)y})
    if (!aligned(p, 16)) return BSQ_ERR_ALIGN;
  if (!aligned(y_scale, 4) || !aligned(y_global, 4)) return BSQ_ERR_ALIGN;
  if ((st = bsq::current_device_status()) != BSQ_OK) return st;
  bsq::NormForward a{};
  a.n = norm_args(b);
  a.x = rows_of(x, x_stride);
  a.branch = rows_of(branch, branch_stride);
  a.x_out = rows_of(x_out, x_out_stride);
  a.y = rows_of(y, y_stride);
  a.out_format = out_format;
  a.y_global = y_global;
  a.y_scale = y_scale;
  return finish(bsq::launch_block_norm(b->dtype, a, stream));
}

size_t bsq_block_norm_workspace_bytes(int64_t rows, int64_t dim, int64_t groups) {
  if (rows <= 0 || rows > kMaxRows || dim < 8 || dim > 16384 || dim % 8 != 0 || groups < 1 || groups > kMaxGroups)
    return 0;
  return bsq::block_norm_workspace(rows, dim, groups);
}

bsq_status bsq_block_norm_backward(const bsq_block* b, const void* dy, int64_t dy_stride, const void* dx_out,
                                   int64_t dx_out_stride, const void* x_out, int64_t x_out_stride, const void* branch,
                                   int64_t branch_stride, void* dx, int64_t dx_stride, void* dbranch,
                                   int64_t dbranch_stride, float* dscale, float* dshift, float* dgate, float* dweight,
                                   float* dbias, float* dpost_weight, void* workspace, size_t workspace_bytes,
                                   hipStream_t stream) {
  bsq_status st = check_block(b);
  if (st != BSQ_OK) return st;
  const bool normed = b->norm != BSQ_NORM_NONE;
  if ((dscale && !b->scale) || (dshift && !b->shift) || (dgate && !b->gate) || (dweight && !b->weight) ||
      (dbias && !b->bias) || (dpost_weight && !b->post_weight) || (!normed && dy))
    return BSQ_ERR_ARG;
  if ((normed && (!stride_ok(dy_stride, b->dim, b->rows, true) || !stride_ok(x_out_stride, b->dim, b->rows, true))) ||
      (dx_out && !stride_ok(dx_out_stride, b->dim, b->rows, true)) ||
      (branch && !stride_ok(branch_stride, b->dim, b->rows, true)) ||
      (dx && !stride_ok(dx_stride, b->dim, b->rows, false)) ||
      (dbranch && !stride_ok(dbranch_stride, b->dim, b->rows, false)))
    return BSQ_ERR_SHAPE;
  if (b->rows > 1 && ((dx && dx == dy && dx_stride != dy_stride) || (dx && dx == dx_out && dx_stride != dx_out_stride) ||
                      (dbranch && dbranch == branch && dbranch_stride != branch_stride)))
    return BSQ_ERR_SHAPE;
  const bool vectors = dscale || dshift || dgate || dweight || dbias || dpost_weight;
  if (b->rows == 0 && !vectors) return BSQ_OK;
  if (b->rows > 0) {
    if (normed ? (!dy || !x_out) : !dx_out) return BSQ_ERR_NULL;
    if (!branch && (dgate || dpost_weight || (dbranch && b->post != BSQ_NORM_NONE))) return BSQ_ERR_NULL;
    if (!dx && !dbranch && !vectors) return BSQ_OK;
  }
  for (const void* p : {dy, dx_out, x_out, branch, (const void*)dx, (const void*)dbranch})
    if (!aligned(p, 16)) return BSQ_ERR_ALIGN;
  for (const float* p : {dscale, dshift, dgate, dweight, dbias, dpost_weight})
    if (!aligned(p, 4)) return BSQ_ERR_ALIGN;
  if (vectors && b->rows > 0) {
    if (!workspace || workspace_bytes < bsq::block_norm_workspace(b->rows, b->dim, b->groups)) return BSQ_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return BSQ_ERR_ALIGN;
  }
  if ((st = bsq::current_device_status()) != BSQ_OK) return st;
  bsq::NormBackward a{};
  a.n = norm_args(b);
  a.dy = rows_of(dy, dy_stride);
  a.dx_out = rows_of(dx_out, dx_out_stride);
  a.x_out = rows_of(x_out, x_out_stride);
  a.branch = rows_of(branch, branch_stride);
  a.dx = rows_of(dx, dx_stride);
  a.dbranch = rows_of(dbranch, dbranch_stride);
  a.dscale = dscale; a.dshift = dshift; a.dgate = dgate;
  a.dweight = dweight; a.dbias = dbias; a.dpost_weight = dpost_weight;
  return finish(bsq::launch_block_norm_backward(b->dtype, a, workspace, stream));
}

}  // extern "C"
