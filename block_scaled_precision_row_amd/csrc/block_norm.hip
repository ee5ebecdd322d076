// The gated residual with the norms before and after it, and its gradient (include/bsq_block.h).
//
// Bound by memory: a row is read once, held in fp32 registers by the W waves of one worker (chunk lane + 64 (wave + W k)
// of eight elements, k < C), and written once. The vectors of its group are read again for every row, from the caches.
// A sum over the row is one DPP reduction in each wave and, with W > 1, one exchange through LDS; the variance is taken
// about the mean (a second reduction) rather than from the squares, which would cancel for rows far from zero.
#include <type_traits>
#include <utility>

#include "block_launch.hpp"
#include "serve_device.hpp"

namespace bsq {

namespace {

// ---- sums over a row --------------------------------------------------------------

template <int ctrl, int rows>
__device__ __forceinline__ float dpp_from(float v) {
  return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), ctrl, rows, 0xF, false));
}
// over the wave's 64 lanes, the same in all of them
__device__ __forceinline__ float wave_sum(float v) {
  v += dpp_from<0x111, 0xF>(v);  // within 16 lanes: row_shr 1, 2, 4, 8
  v += dpp_from<0x112, 0xF>(v);
  v += dpp_from<0x114, 0xF>(v);
  v += dpp_from<0x118, 0xF>(v);
  v += dpp_from<0x142, 0xA>(v);  // row_bcast 15: rows 0 and 2 to 1 and 3
  v += dpp_from<0x143, 0xC>(v);  // row_bcast 31: the first half to the second
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}
// the larger, NaN if either is NaN
__device__ __forceinline__ float max_nan(float a, float b) { return a != a || a > b ? a : b; }
__device__ __forceinline__ float wave_max_nan(float v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v = max_nan(v, __shfl_xor(v, off, 64));
  return v;
}

// Sums (or the maximum) over the W waves of a worker. Each reduction of a row has LDS of its own, and rows alternate between two sets of
// it: a wave that is a row ahead has passed a barrier that the others reach only after they have read the set before.
constexpr int kReductions = 6, kMostSums = 2;  // of a row at most: two norms of two each, and one for each gradient
template <int W>
struct RowSums {
  float (*slots)[W][kMostSums];  // [kReductions] of this row's parity
  int wave, lane, at;
  template <int K>
  __device__ __forceinline__ void sum(float (&v)[K]) {
    static_assert(K <= kMostSums, "room");
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = wave_sum(v[k]);
    if constexpr (W > 1) {
      float(*s)[kMostSums] = slots[at++];
      if (lane == 0) {
#pragma unroll
        for (int k = 0; k < K; ++k) s[wave][k] = v[k];
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < K; ++k) {
        v[k] = s[0][k];
#pragma unroll
        for (int w = 1; w < W; ++w) v[k] += s[w][k];
      }
    }
  }
  __device__ __forceinline__ float max(float v) {
    v = wave_max_nan(v);
    if constexpr (W > 1) {
      float(*s)[kMostSums] = slots[at++];
      if (lane == 0) s[wave][0] = v;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < W; ++w) v = max_nan(v, s[w][0]);
    }
    return v;
  }
};

template <int W>
constexpr int threads_of() { return W == 1 ? 256 : 64 * W; }
template <int W>
constexpr int workers_of() { return W == 1 ? 4 : 1; }  // in a workgroup

// v becomes v - mean (BSQ_NORM_LAYER); returns 1 / sqrt(mean v^2 + eps)
template <int W, int C>
__device__ __forceinline__ float size_of(float (&v)[C][8], bool layer, float eps, float inv_dim, const bool (&has)[C],
                                         RowSums<W>& rs) {
  if (layer) {
    float s[1] = {0.0f};
#pragma unroll
    for (int k = 0; k < C; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) s[0] += v[k][e];  // (elements that are not there are 0)
    rs.sum(s);
    const float mean = s[0] * inv_dim;
#pragma unroll
    for (int k = 0; k < C; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) v[k][e] = has[k] ? v[k][e] - mean : 0.0f;
  }
  float s[1] = {0.0f};
#pragma unroll
  for (int k = 0; k < C; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) s[0] = fmaf(v[k][e], v[k][e], s[0]);
  rs.sum(s);
  return 1.0f / sqrtf(s[0] * inv_dim + eps);
}

template <class E>
__device__ __forceinline__ const typename E::elem* row_of(const Rows& r, int64_t row) {
  return static_cast<const typename E::elem*>(r.p) + row * r.stride;
}
template <class E>
__device__ __forceinline__ const typename E::elem* row_of(const GroupVector& v, int g) {
  return static_cast<const typename E::elem*>(v.p) + (int64_t)g * v.stride;
}

// ---- forward ------------------------------------------------------------------------

// the encodings of include/bsq.h for the fp32 values of a row
__device__ __forceinline__ uint32_t block_scale(float a, float G, float& r) {
  const float u = (a / kE2M1Max) * G;
  const uint32_t sf = u != u ? 0x7Fu : enc_e4m3(u);
  const float v = dec_e4m3<0>(sf);
  r = v != v ? v : (v > 0.0f ? G / v : 0.0f);
  return sf;
}

template <class E, int W, int C>
__global__ __launch_bounds__(threads_of<W>()) void block_norm(NormForward a) {
  typedef typename E::elem elem;
  __shared__ float slots[W > 1 ? kReductions : 1][W][kMostSums];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int row = blockIdx.x * workers_of<W>() + (W == 1 ? wave : 0);
  const int part = W == 1 ? 0 : wave;
  const NormArgs& n = a.n;
  if (row >= group_limit(n.groups)) return;  // (the whole worker)
  const int chunks = n.dim >> 3;
  const float inv_dim = 1.0f / (float)n.dim;
  RowSums<W> rs{slots, part, lane, 0};
  int at[C];
  bool has[C];
  float v[C][8];
  const elem* x = row_of<E>(a.x, row);
#pragma unroll
  for (int k = 0; k < C; ++k) {
    const int c = lane + 64 * (part + W * k);
    has[k] = c < chunks;
    at[k] = 8 * c;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[k][e] = 0.0f;
    if (has[k]) load8<E>(x + at[k], v[k]);
  }
  const int g = n.scale.p || n.shift.p || n.gate.p ? group_of_wave(n.groups, row, lane) : 0;
  if (a.branch.p) {
    float h[C][8];
    const elem* b = row_of<E>(a.branch, row);
#pragma unroll
    for (int k = 0; k < C; ++k) {
#pragma unroll
      for (int e = 0; e < 8; ++e) h[k][e] = 0.0f;
      if (has[k]) load8<E>(b + at[k], h[k]);
    }
    if (n.post != BSQ_NORM_NONE) {
      const float r = size_of<W, C>(h, n.post == BSQ_NORM_LAYER, n.post_eps, inv_dim, has, rs);
#pragma unroll
      for (int k = 0; k < C; ++k) {
        float w[8] = {1, 1, 1, 1, 1, 1, 1, 1};
        if (n.post_weight && has[k]) load8<E>(static_cast<const elem*>(n.post_weight) + at[k], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[k][e] = h[k][e] * r * w[e];
      }
    }
#pragma unroll
    for (int k = 0; k < C; ++k) {
      if (!has[k]) continue;
      float w[8] = {1, 1, 1, 1, 1, 1, 1, 1};
      if (n.gate.p) load8<E>(row_of<E>(n.gate, g) + at[k], w);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[k][e] = fmaf(w[e], h[k][e], v[k][e]);
      if (a.x_out.p) store8<E>(const_cast<elem*>(row_of<E>(a.x_out, row)) + at[k], v[k]);
    }
  }
  if (n.norm == BSQ_NORM_NONE) return;
  const float r = size_of<W, C>(v, n.norm == BSQ_NORM_LAYER, n.eps, inv_dim, has, rs);
  float most = 0.0f;
#pragma unroll
  for (int k = 0; k < C; ++k) {
    if (!has[k]) continue;
    float w[8] = {1, 1, 1, 1, 1, 1, 1, 1};
    if (n.weight) load8<E>(static_cast<const elem*>(n.weight) + at[k], w);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[k][e] = v[k][e] * r * w[e];
    if (n.bias) {
      load8<E>(static_cast<const elem*>(n.bias) + at[k], w);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[k][e] += w[e];
    }
    if (n.scale.p) {
      load8<E>(row_of<E>(n.scale, g) + at[k], w);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[k][e] *= 1.0f + w[e];
    }
    if (n.shift.p) {
      load8<E>(row_of<E>(n.shift, g) + at[k], w);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[k][e] += w[e];
    }
    if (a.out_format == 0) store8<E>(const_cast<elem*>(row_of<E>(a.y, row)) + at[k], v[k]);
#pragma unroll
    for (int e = 0; e < 8; ++e) most = max_nan(most, fabsf(v[k][e]));
  }
  if (a.out_format == BSQ_FMT_FP8R) {
    most = rs.max(most);
    const float d = most / kE4M3Max;
    const float q = d > 0.0f ? 1.0f / d : (d != d ? d : 0.0f);
    uint8_t* y = static_cast<uint8_t*>(a.y.p) + (int64_t)row * n.dim;
#pragma unroll
    for (int k = 0; k < C; ++k) {
      if (!has[k]) continue;
      uint2 o;
      o.x = enc_e4m3x4(v[k][0] * q, v[k][1] * q, v[k][2] * q, v[k][3] * q);
      o.y = enc_e4m3x4(v[k][4] * q, v[k][5] * q, v[k][6] * q, v[k][7] * q);
      *reinterpret_cast<uint2*>(y + at[k]) = o;
    }
    if (part == 0 && lane == 0) static_cast<float*>(a.y_scale)[row] = d;
  }
  if (a.out_format == BSQ_FMT_NVFP4) {
    const float G = 1.0f / a.y_global[0];
    uint8_t* y = static_cast<uint8_t*>(a.y.p) + (int64_t)row * (n.dim >> 1);
    uint8_t* ys = static_cast<uint8_t*>(a.y_scale) + (int64_t)row * (n.dim >> 4);
#pragma unroll
    for (int k = 0; k < C; ++k) {
      float m = 0.0f;  // of the lane's half of a block of 16; its neighbour has the other (dim % 16 == 0: both or none)
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max_nan(m, fabsf(v[k][e]));
      m = max_nan(m, __shfl_xor(m, 1, 64));
      if (!has[k]) continue;
      float q;
      const uint32_t sf = block_scale(m, G, q);
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = v[k][e] * q;
      *reinterpret_cast<uint32_t*>(y + (at[k] >> 1)) = enc_e2m1x8(f);
      if ((lane & 1) == 0) ys[at[k] >> 4] = (uint8_t)sf;
    }
  }
}

// ---- backward -----------------------------------------------------------------------
// A worker takes `run` consecutive rows and sums, over the rows of one group, dy n, dy and c h' (before its weight) for
// its columns in registers; when the group changes, and at the end, the sums go to slot (worker + group) of the
// workspace, [slot][3][dim] (no two have the same: the group grows from slot to slot where the worker does not). A
// second kernel adds the slots of each group in their order, and a third the groups for the gradients that all share.

template <class E, int W, int C>
__global__ __launch_bounds__(threads_of<W>()) void block_norm_backward(NormBackward a, int run, float* part_sums) {
  typedef typename E::elem elem;
  __shared__ float slots[W > 1 ? 2 * kReductions : 1][W][kMostSums];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int worker = blockIdx.x * workers_of<W>() + (W == 1 ? wave : 0);
  const int part = W == 1 ? 0 : wave;
  const NormArgs& n = a.n;
  const int limit = group_limit(n.groups), first = worker * run;
  const int last = limit - first < run ? limit : first + run;
  if (first >= last) return;
  const int chunks = n.dim >> 3;
  const float inv_dim = 1.0f / (float)n.dim;
  const bool layer = n.norm == BSQ_NORM_LAYER, post_layer = n.post == BSQ_NORM_LAYER;
  const bool normed = n.norm != BSQ_NORM_NONE, post = n.post != BSQ_NORM_NONE, branch = a.branch.p != nullptr;
  int at[C];
  bool has[C];
  float sums[3][C][8];
#pragma unroll
  for (int k = 0; k < C; ++k) {
    const int c = lane + 64 * (part + W * k);
    has[k] = c < chunks;
    at[k] = 8 * c;
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[0][k][e] = sums[1][k][e] = sums[2][k][e] = 0.0f;
  }
  auto flush = [&](int g) {
    float* to = part_sums + (int64_t)(worker + g) * 3 * n.dim;
#pragma unroll
    for (int q = 0; q < 3; ++q)
#pragma unroll
      for (int k = 0; k < C; ++k) {
        if (has[k]) store8<Fp32>(to + (int64_t)q * n.dim + at[k], sums[q][k]);
#pragma unroll
        for (int e = 0; e < 8; ++e) sums[q][k][e] = 0.0f;
      }
  };
  auto load = [&](const elem* p, float (&f)[C][8]) {
#pragma unroll
    for (int k = 0; k < C; ++k) {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[k][e] = 0.0f;
      if (has[k]) load8<E>(p + at[k], f[k]);
    }
  };
  int g = group_of_wave(n.groups, first, lane);
  for (int row = first; row < last; ++row) {
    if (row > first && n.groups.groups > 1) {
      const int now = group_of_wave(n.groups, row, lane);
      if (now != g) {
        if (part_sums) flush(g);
        g = now;
      }
    }
    RowSums<W> rs{slots + (W > 1 ? (row & 1) * kReductions : 0), part, lane, 0};
    float c[C][8], v[C][8], d[C][8], h[C][8];
    if (a.dx_out.p) load(row_of<E>(a.dx_out, row), c);
    else
#pragma unroll
      for (int k = 0; k < C; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) c[k][e] = 0.0f;
    if (branch) load(row_of<E>(a.branch, row), h);
    float hr = 1.0f;
    if (branch && post) {
      hr = size_of<W, C>(h, post_layer, n.post_eps, inv_dim, has, rs);
#pragma unroll
      for (int k = 0; k < C; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) h[k][e] *= hr;
    }
    if (normed) {
      load(row_of<E>(a.x_out, row), v);
      load(row_of<E>(a.dy, row), d);
      const float r = size_of<W, C>(v, layer, n.eps, inv_dim, has, rs);
      float s[2] = {0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < C; ++k) {
        float w[8] = {1, 1, 1, 1, 1, 1, 1, 1}, m[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (n.weight && has[k]) load8<E>(static_cast<const elem*>(n.weight) + at[k], w);
        if (n.scale.p && has[k]) load8<E>(row_of<E>(n.scale, g) + at[k], m);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[k][e] *= r;
          sums[0][k][e] = fmaf(d[k][e], v[k][e], sums[0][k][e]);
          sums[1][k][e] += d[k][e];
          d[k][e] *= (1.0f + m[e]) * w[e];
          s[0] = fmaf(d[k][e], v[k][e], s[0]);
          s[1] += d[k][e];
        }
      }
      rs.sum(s);
      const float along = s[0] * inv_dim, mean = layer ? s[1] * inv_dim : 0.0f;
#pragma unroll
      for (int k = 0; k < C; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) c[k][e] = fmaf(r, d[k][e] - mean - v[k][e] * along, c[k][e]);
    }
#pragma unroll
    for (int k = 0; k < C; ++k) {
      if (!has[k]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) c[k][e] = 0.0f;
      }
      if (a.dx.p && has[k]) store8<E>(const_cast<elem*>(row_of<E>(a.dx, row)) + at[k], c[k]);
      if (branch) {
#pragma unroll
        for (int e = 0; e < 8; ++e) sums[2][k][e] = fmaf(c[k][e], h[k][e], sums[2][k][e]);
      }
    }
    if (!a.dbranch.p) continue;
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < C; ++k) {
      float w[8] = {1, 1, 1, 1, 1, 1, 1, 1};
      if (n.gate.p && has[k]) {
        load8<E>(row_of<E>(n.gate, g) + at[k], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) c[k][e] *= w[e];
      }
      if (post && n.post_weight && has[k]) {
        load8<E>(static_cast<const elem*>(n.post_weight) + at[k], w);
#pragma unroll
        for (int e = 0; e < 8; ++e) c[k][e] *= w[e];
      }
      if (post) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          s[0] = fmaf(c[k][e], h[k][e], s[0]);
          s[1] += c[k][e];
        }
      }
    }
    if (post) {
      rs.sum(s);
      const float along = s[0] * inv_dim, mean = post_layer ? s[1] * inv_dim : 0.0f;
#pragma unroll
      for (int k = 0; k < C; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) c[k][e] = hr * (c[k][e] - mean - h[k][e] * along);
    }
#pragma unroll
    for (int k = 0; k < C; ++k)
      if (has[k]) store8<E>(const_cast<elem*>(row_of<E>(a.dbranch, row)) + at[k], c[k]);
  }
  if (part_sums) flush(g);
}

template <class E>
__device__ __forceinline__ float one(const void* p, int64_t at) {
  if constexpr (sizeof(typename E::elem) == 4) return static_cast<const float*>(p)[at];
  else return E::up(static_cast<const uint16_t*>(p)[at]);
}
template <class E>
__device__ __forceinline__ float one(const GroupVector& v, int g, int col) {
  return one<E>(v.p, (int64_t)g * v.stride + col);
}

constexpr int kCols = 32, kLanes = 32;  // columns of a workgroup, and threads that share a column's sum

// the sum over the threads of a column, in all of them (sum[][] is free again after it)
__device__ __forceinline__ float column_sum(float v, float (*sum)[kCols], int col, int lane) {
  sum[lane][col] = v;
  __syncthreads();
#pragma unroll
  for (int s = kLanes / 2; s >= 1; s >>= 1) {
    if (lane < s) sum[lane][col] += sum[lane + s][col];
    __syncthreads();
  }
  v = sum[0][col];
  __syncthreads();
  return v;
}

// the gradients that all groups share, from the sums of one group (or of all)
template <class E>
__device__ __forceinline__ void add_shared(const NormBackward& a, int g, int col, const float (&s)[3], float (&t)[3]) {
  const float m = a.n.scale.p ? 1.0f + one<E>(a.n.scale, g, col) : 1.0f;
  const float k = a.n.gate.p ? one<E>(a.n.gate, g, col) : 1.0f;
  t[0] = fmaf(m, s[0], t[0]);
  t[1] = fmaf(m, s[1], t[1]);
  t[2] = fmaf(k, s[2], t[2]);
}
__device__ __forceinline__ void put_shared(const NormBackward& a, int col, const float (&t)[3]) {
  if (a.dweight) a.dweight[col] = t[0];
  if (a.dbias) a.dbias[col] = t[1];
  if (a.dpost_weight) a.dpost_weight[col] = t[2];
}

// The sums of each group: grid.x over columns, grid.y (striding) over groups. With one group also what all groups share;
// otherwise, where that is asked for, the sums go to `group_sums` [groups][3][dim].
template <class E>
__global__ __launch_bounds__(kCols * kLanes) void norm_group_sums(NormBackward a, int run, const float* part_sums,
                                                                  float* group_sums) {
  __shared__ float sum[kLanes][kCols];
  const int c = threadIdx.x & (kCols - 1), lane = threadIdx.x / kCols, col = blockIdx.x * kCols + c;
  const bool live = col < a.n.dim;
  const RowGroups& rg = a.n.groups;
  for (int g = blockIdx.y; g < rg.groups; g += gridDim.y) {
    int r0, r1;
    if (rg.starts) {
      const int limit = group_limit(rg);
      r0 = rg.starts[g];
      r1 = rg.starts[g + 1];
      r0 = r0 < 0 ? 0 : r0;
      r1 = r1 < limit ? r1 : limit;
    } else {
      r0 = g * rg.per;
      r1 = r0 + rg.per;
    }
    float s[3] = {0.0f, 0.0f, 0.0f};
    if (r1 > r0 && live) {
      const int w1 = (r1 - 1) / run;
      for (int w = r0 / run + lane; w <= w1; w += kLanes) {
        const float* p = part_sums + (int64_t)(w + g) * 3 * a.n.dim + col;
#pragma unroll
        for (int q = 0; q < 3; ++q) s[q] += p[(int64_t)q * a.n.dim];
      }
    }
#pragma unroll
    for (int q = 0; q < 3; ++q) s[q] = column_sum(s[q], sum, c, lane);
    if (!live || lane != 0) continue;
    if (a.dscale) {
      float d = a.n.weight ? s[0] * one<E>(a.n.weight, col) : s[0];
      if (a.n.bias) d = fmaf(one<E>(a.n.bias, col), s[1], d);
      a.dscale[(int64_t)g * a.n.dim + col] = d;
    }
    if (a.dshift) a.dshift[(int64_t)g * a.n.dim + col] = s[1];
    if (a.dgate)
      a.dgate[(int64_t)g * a.n.dim + col] = a.n.post_weight ? s[2] * one<E>(a.n.post_weight, col) : s[2];
    if (group_sums) {
#pragma unroll
      for (int q = 0; q < 3; ++q) group_sums[((int64_t)g * 3 + q) * a.n.dim + col] = s[q];
    } else if (rg.groups == 1) {
      float t[3] = {0.0f, 0.0f, 0.0f};
      add_shared<E>(a, g, col, s, t);
      put_shared(a, col, t);
    }
  }
}

template <class E>
__global__ __launch_bounds__(kCols * kLanes) void norm_shared_sums(NormBackward a, const float* group_sums) {
  __shared__ float sum[kLanes][kCols];
  const int c = threadIdx.x & (kCols - 1), lane = threadIdx.x / kCols, col = blockIdx.x * kCols + c;
  const bool live = col < a.n.dim;
  float t[3] = {0.0f, 0.0f, 0.0f};
  if (live) {
    for (int g = lane; g < a.n.groups.groups; g += kLanes) {
      float s[3];
#pragma unroll
      for (int q = 0; q < 3; ++q) s[q] = group_sums[((int64_t)g * 3 + q) * a.n.dim + col];
      add_shared<E>(a, g, col, s, t);
    }
  }
#pragma unroll
  for (int q = 0; q < 3; ++q) t[q] = column_sum(t[q], sum, c, lane);
  if (live && lane == 0) put_shared(a, col, t);
}

// a call without rows: the gradients of the vectors are sums over nothing
__global__ __launch_bounds__(256) void zero(float* p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = 0.0f;
}

// ---- launches -----------------------------------------------------------------------

// f(waves of a worker, chunks of a lane): a wave holds rows of up to 1024 elements, four waves up to 8192, eight up to 16384
template <class F>
hipError_t with_shape(int dim, F f) {
  using std::integral_constant;
#define BSQ_SHAPE(W, C) return f(integral_constant<int, W>{}, integral_constant<int, C>{})
  if (dim <= 512) BSQ_SHAPE(1, 1);
  if (dim <= 1024) BSQ_SHAPE(1, 2);
  if (dim <= 2048) BSQ_SHAPE(4, 1);
  if (dim <= 4096) BSQ_SHAPE(4, 2);
  if (dim <= 6144) BSQ_SHAPE(4, 3);
  if (dim <= 8192) BSQ_SHAPE(4, 4);
  if (dim <= 12288) BSQ_SHAPE(8, 3);
  BSQ_SHAPE(8, 4);
#undef BSQ_SHAPE
}
int waves_of(int64_t dim) { return dim <= 1024 ? 1 : dim <= 8192 ? 4 : 8; }

template <class E>
hipError_t forward(const NormForward& a, hipStream_t s) {
  return with_shape(a.n.dim, [&](auto w, auto c) {
    constexpr int W = decltype(w)::value, C = decltype(c)::value, per = workers_of<W>();
    hipLaunchKernelGGL((block_norm<E, W, C>), dim3((unsigned)((a.n.rows + per - 1) / per)), dim3(threads_of<W>()), 0, s,
                       a);
    return hipGetLastError();
  });
}

// rows of a worker in the backward pass
int run_of(int64_t rows, int64_t dim) {
  const int64_t want = dim <= 1024 ? 4096 : 1024;  // workers that fill the 256 compute units
  const int64_t n = (rows + want - 1) / want;
  return (int)(n < 4 ? 4 : n);
}
size_t pad256(size_t n) { return (n + 255) & ~(size_t)255; }
size_t slot_bytes(int64_t rows, int64_t dim, int64_t groups) {
  const int run = run_of(rows, dim);
  return pad256((size_t)((rows + run - 1) / run + groups) * 3 * (size_t)dim * 4);
}

template <class E>
hipError_t backward(const NormBackward& a, void* workspace, hipStream_t s) {
  const bool shared = a.dweight || a.dbias || a.dpost_weight, vectors = a.dscale || a.dshift || a.dgate || shared;
  if (a.n.rows == 0) {
    const int64_t all = (int64_t)a.n.groups.groups * a.n.dim;
    for (const auto& [p, n] : {std::pair<float*, int64_t>{a.dscale, all}, {a.dshift, all}, {a.dgate, all},
                               {a.dweight, a.n.dim}, {a.dbias, a.n.dim}, {a.dpost_weight, a.n.dim}}) {
      if (!p) continue;
      const int64_t blocks = (n + 255) / 256;
      hipLaunchKernelGGL(zero, dim3((unsigned)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, s, p, n);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    return hipSuccess;
  }
  const int run = run_of(a.n.rows, a.n.dim), workers = (a.n.rows + run - 1) / run, groups = a.n.groups.groups;
  float* parts = vectors ? static_cast<float*>(workspace) : nullptr;
  hipError_t e = with_shape(a.n.dim, [&](auto w, auto c) {
    constexpr int W = decltype(w)::value, C = decltype(c)::value, per = workers_of<W>();
    hipLaunchKernelGGL((block_norm_backward<E, W, C>), dim3((unsigned)((workers + per - 1) / per)),
                       dim3(threads_of<W>()), 0, s, a, run, parts);
    return hipGetLastError();
  });
  if (e != hipSuccess || !vectors) return e;
  float* sums = nullptr;
  if (shared && groups > 1)
    sums = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + slot_bytes(a.n.rows, a.n.dim, groups));
  const unsigned cols = (unsigned)((a.n.dim + kCols - 1) / kCols);
  hipLaunchKernelGGL(norm_group_sums<E>, dim3(cols, (unsigned)(groups < 65535 ? groups : 65535)), dim3(kCols * kLanes),
                     0, s, a, run, parts, sums);
  if ((e = hipGetLastError()) != hipSuccess || !sums) return e;
  hipLaunchKernelGGL(norm_shared_sums<E>, dim3(cols), dim3(kCols * kLanes), 0, s, a, sums);
  return hipGetLastError();
}

}  // namespace

size_t block_norm_workspace(int64_t rows, int64_t dim, int64_t groups) {
  return slot_bytes(rows, dim, groups) + (groups > 1 ? (size_t)groups * 3 * (size_t)dim * 4 : 0);
}

hipError_t launch_block_norm(bsq_dtype dt, const NormForward& a, hipStream_t s) {
  if (dt == BSQ_BF16) return forward<Bf16>(a, s);
  if (dt == BSQ_FP16) return forward<Fp16>(a, s);
  return forward<Fp32>(a, s);
}

hipError_t launch_block_norm_backward(bsq_dtype dt, const NormBackward& a, void* workspace, hipStream_t s) {
  if (dt == BSQ_BF16) return backward<Bf16>(a, workspace, s);
  if (dt == BSQ_FP16) return backward<Fp16>(a, workspace, s);
  return backward<Fp32>(a, workspace, s);
}

}  // namespace bsq
