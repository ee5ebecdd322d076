// The gated residual with the norms before and after it, and its gradient (include/bsq_block.h).
//
// Bound by memory: a row is read once, held in registers by the waves of one worker, and written once. Forward, a worker
// has one row, and other workers' loads run under its sums (several rows with the next one's loads under way: 111 us
// where this takes 64); backward it takes several, with the next one's loads under way, and keeps the vectors and the
// columns' sums in registers (which spill for rows of more than 12288 elements: 1024 rows of bf16 with post norm and weights
// 72.9 us at 12288, 189 at 16384). A sum over the row is one DPP reduction in each wave and, where a worker has several, one
// exchange through LDS; the variance is taken about the mean (a second reduction) rather than from the squares, which would
// cancel for rows far from zero.
#include <type_traits>
#include <utility>

#include "block_launch.hpp"
#include "serve_device.hpp"

namespace bsq {

namespace {

// ---- sums over a row --------------------------------------------------------------

template <int ctrl, int rows>
__device__ __forceinline__ uint32_t dpp_from(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, rows, 0xF, false);
}
template <int ctrl, int rows>
__device__ __forceinline__ uint32_t max_from(uint32_t v) {
  const uint32_t o = dpp_from<ctrl, rows>(v);
  return o > v ? o : v;
}
template <int ctrl, int rows>
__device__ __forceinline__ float add_from(float v) {
  return v + __uint_as_float(dpp_from<ctrl, rows>(__float_as_uint(v)));
}
__device__ __forceinline__ float row_sum(float v) {  // over 16 lanes, in the last of them: row_shr 1, 2, 4, 8
  return add_from<0x118, 0xF>(add_from<0x114, 0xF>(add_from<0x112, 0xF>(add_from<0x111, 0xF>(v))));
}
// Over the wave's 64 lanes, the same in all of them (row_bcast 15: rows 0 and 2 to 1 and 3; row_bcast 31: the first half
// to the second). On the matrix cores (v as a 16 x 4 operand against ones, twice) this is 5 instructions rather than 14,
// but takes longer: the gradient at 4608 x 2560 53 us against 47.
__device__ __forceinline__ float wave_sum(float v) {
  v = add_from<0x143, 0xC>(add_from<0x142, 0xA>(row_sum(v)));
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v), 63));
}
// the largest, likewise
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max_from<0x118, 0xF>(max_from<0x114, 0xF>(max_from<0x112, 0xF>(max_from<0x111, 0xF>(v))));
  v = max_from<0x143, 0xC>(max_from<0x142, 0xA>(v));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// Sums (or the maximum) over the waves of a worker: over the lanes, then through LDS, where each reduction of a row has
// room of its own and rows alternate between two sets of it: a wave that is a row ahead has passed a barrier that the
// others reach only after they have read the set before. ONE: the worker is one wave.
constexpr int kReductions = 5, kMostSums = 4;  // of a row at most (forward: two norms of two each, and the maximum)
constexpr int kMostWaves = 16;
struct Slots {
  float s[2][kReductions][kMostSums][kMostWaves];
};
template <bool ONE>
struct RowSums {
  Slots* slots;
  int wave, waves, lane, row, at;
  template <int K>
  __device__ __forceinline__ void sum(float (&v)[K]) {
    static_assert(K <= kMostSums, "room");
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = wave_sum(v[k]);
    if constexpr (!ONE) {
      auto& s = slots->s[row & 1][at++];
      if (lane == 0) {
#pragma unroll
        for (int k = 0; k < K; ++k) s[k][wave] = v[k];
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < K; ++k) {  // (the first 16 lanes)
        const float o = row_sum(lane < waves ? s[k][lane & (kMostWaves - 1)] : 0.0f);
        v[k] = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(o), kMostWaves - 1));
      }
    }
  }
  __device__ __forceinline__ float max(float most) {  // of magnitudes: their bits order as they do, NaN above all
    uint32_t v = wave_max(__float_as_uint(most));
    if constexpr (!ONE) {
      auto& s = slots->s[row & 1][at++];
      if (lane == 0) s[0][wave] = __uint_as_float(v);
      __syncthreads();
      v = wave_max(lane < waves ? __float_as_uint(s[0][lane & (kMostWaves - 1)]) : 0u);
    }
    return __uint_as_float(v);
  }
};

// ---- a worker's piece of a row --------------------------------------------------------

// A worker's waves share a row: chunk lane + 64 (wave + waves k) of eight elements, k < C. One wave takes rows of up to
// 512 elements, four such workers in a workgroup; longer rows have a workgroup of up to sixteen waves forward and eight
// backward.
template <bool ONE>
constexpr int most_threads() { return ONE ? 256 : 64 * kMostWaves; }
constexpr int kBackwardThreads = 512;

template <class E>
struct Chunk {  // eight elements as they are in memory
  uint4 q;
  __device__ __forceinline__ void load(const typename E::elem* p) { q = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { q = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&f)[8]) const { unpack8<E>(q, f); }
};
template <>
struct Chunk<Fp32> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
};

template <bool ONE, int C>
struct Place {
  int worker, part, parts, lane;
  uint32_t at[C];  // first element of the chunk
  bool has[C];
  __device__ __forceinline__ Place(int dim) {
    lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
    worker = ONE ? blockIdx.x * 4 + wave : blockIdx.x;
    part = ONE ? 0 : wave;
    parts = ONE ? 1 : __builtin_amdgcn_readfirstlane((int)blockDim.x >> 6);
#pragma unroll
    for (int k = 0; k < C; ++k) {
      const int c = lane + 64 * (part + parts * k);
      has[k] = c < dim >> 3;
      at[k] = 8u * (uint32_t)c;
    }
  }
  // the worker's chunks of the row behind p (zeros where it has none, or without a row)
  template <class E>
  __device__ __forceinline__ void load(Chunk<E> (&r)[C], const typename E::elem* p) const {
#pragma unroll
    for (int k = 0; k < C; ++k) {
      r[k].zero();
      if (p && has[k]) r[k].load(p + at[k]);
    }
  }
};

// A vector along the row: held in registers from row to row, or read again for each (HOLD: registers allow it)
template <class E, int C, bool HOLD>
struct Vector {
  const typename E::elem* p;
  Chunk<E> r[HOLD ? C : 1];
  template <class P>
  __device__ __forceinline__ void set(const P& me, const typename E::elem* to) {
    p = to;
    if constexpr (HOLD) me.load(r, to);
  }
  // chunk k as fp32, of a vector that is there (anything where the worker has no chunk)
  template <class P>
  __device__ __forceinline__ void get(const P& me, int k, float (&f)[8]) const {
    if constexpr (HOLD) {
      r[k].get(f);
    } else {
      Chunk<E> c;
      c.zero();
      if (me.has[k]) c.load(p + me.at[k]);
      c.get(f);
    }
  }
};

// v becomes v - mean (BSQ_NORM_LAYER); returns 1 / sqrt(mean v^2 + eps)
template <bool ONE, int C>
__device__ __forceinline__ float size_of(float (&v)[C][8], bool layer, float eps, float inv_dim, const bool (&has)[C],
                                         RowSums<ONE>& rs) {
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
  return r.p ? static_cast<const typename E::elem*>(r.p) + row * r.stride : nullptr;
}
template <class E>
__device__ __forceinline__ typename E::elem* out_of(const Rows& r, int64_t row) {
  return static_cast<typename E::elem*>(r.p) + row * r.stride;
}
template <class E>
__device__ __forceinline__ const typename E::elem* row_of(const GroupVector& v, int g) {
  return v.p ? static_cast<const typename E::elem*>(v.p) + (int64_t)g * v.stride : nullptr;
}
template <class E>
__device__ __forceinline__ const typename E::elem* row_of(const void* v) {
  return static_cast<const typename E::elem*>(v);
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

// the larger of two magnitudes, NaN if one is (one instruction, of three operands)
__device__ __forceinline__ float larger(float a, float b) { return __builtin_elementwise_maximum(a, b); }

// One row a worker: with some 20 waves on a compute unit the loads of other rows run under a row's sums.
template <class E, bool ONE, int C, bool GROUPED>
__global__ __launch_bounds__(most_threads<ONE>()) void block_norm(NormForward a) {
  __shared__ Slots slots;
  const NormArgs& n = a.n;
  const Place<ONE, C> me(n.dim);
  const int row = me.worker;
  if (row >= n.groups.rows) return;  // (the whole worker)
  Chunk<E> x[C], h[C];
  me.load(x, row_of<E>(a.x, row));
  me.load(h, row_of<E>(a.branch, row));
  Vector<E, C, !GROUPED> weight, bias, pw;
  pw.set(me, row_of<E>(n.post_weight));
  weight.set(me, row_of<E>(n.weight));
  bias.set(me, row_of<E>(n.bias));
  if (row >= group_limit(n.groups)) return;
  const int g = GROUPED ? group_of_wave(n.groups, row, me.lane) : 0;
  Vector<E, C, false> scale, shift, gate;
  if constexpr (GROUPED) {
    gate.set(me, row_of<E>(n.gate, g));
    scale.set(me, row_of<E>(n.scale, g));
    shift.set(me, row_of<E>(n.shift, g));
  }
  const float inv_dim = 1.0f / (float)n.dim;
  RowSums<ONE> rs{&slots, me.part, me.parts, me.lane, 0, 0};
  float v[C][8];
#pragma unroll
  for (int k = 0; k < C; ++k) x[k].get(v[k]);
  if (a.branch.p) {
    float f[C][8];
#pragma unroll
    for (int k = 0; k < C; ++k) h[k].get(f[k]);
    if (n.post != BSQ_NORM_NONE) {
      const float r = size_of<ONE, C>(f, n.post == BSQ_NORM_LAYER, n.post_eps, inv_dim, me.has, rs);
#pragma unroll
      for (int k = 0; k < C; ++k) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[k][e] *= r;
        if (pw.p) {
          float w[8];
          pw.get(me, k, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) f[k][e] *= w[e];
        }
      }
    }
#pragma unroll
    for (int k = 0; k < C; ++k) {
      if (GROUPED && gate.p) {
        float w[8];
        gate.get(me, k, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[k][e] = fmaf(w[e], f[k][e], v[k][e]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[k][e] += f[k][e];
      }
      if (a.x_out.p && me.has[k]) store8<E>(out_of<E>(a.x_out, row) + me.at[k], v[k]);
    }
  }
  if (n.norm == BSQ_NORM_NONE) return;
  const float r = size_of<ONE, C>(v, n.norm == BSQ_NORM_LAYER, n.eps, inv_dim, me.has, rs);
  float most = 0.0f;
#pragma unroll
  for (int k = 0; k < C; ++k) {
    if (!me.has[k]) continue;
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[k][e] *= r;
    if (weight.p) {
      weight.get(me, k, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[k][e] *= w[e];
    }
    if (bias.p) {
      bias.get(me, k, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[k][e] += w[e];
    }
    if constexpr (GROUPED) {
      if (scale.p) {
        scale.get(me, k, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[k][e] = fmaf(v[k][e], w[e], v[k][e]);  // (v (1 + scale))
      }
      if (shift.p) {
        shift.get(me, k, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[k][e] += w[e];
      }
    }
    if (a.out_format == 0) {
      store8<E>(out_of<E>(a.y, row) + me.at[k], v[k]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; e += 2) most = larger(larger(most, fabsf(v[k][e])), fabsf(v[k][e + 1]));
    }
  }
  if (a.out_format == BSQ_FMT_FP8R) {
    const float d = rs.max(most) / kE4M3Max;
    const float q = d > 0.0f ? 1.0f / d : (d != d ? d : 0.0f);
    uint8_t* y = static_cast<uint8_t*>(a.y.p) + (int64_t)row * n.dim;
#pragma unroll
    for (int k = 0; k < C; ++k) {
      if (!me.has[k]) continue;
      uint2 o;
      o.x = enc_e4m3x4(v[k][0] * q, v[k][1] * q, v[k][2] * q, v[k][3] * q);
      o.y = enc_e4m3x4(v[k][4] * q, v[k][5] * q, v[k][6] * q, v[k][7] * q);
      *reinterpret_cast<uint2*>(y + me.at[k]) = o;
    }
    if (me.part == 0 && me.lane == 0) static_cast<float*>(a.y_scale)[row] = d;
  }
  if (a.out_format == BSQ_FMT_NVFP4) {
    const float G = 1.0f / a.y_global[0];
    uint8_t* y = static_cast<uint8_t*>(a.y.p) + (int64_t)row * (n.dim >> 1);
    uint8_t* ys = static_cast<uint8_t*>(a.y_scale) + (int64_t)row * (n.dim >> 4);
#pragma unroll
    for (int k = 0; k < C; ++k) {
      float m = 0.0f;  // of the lane's half of a block of 16; its neighbour has the other (dim % 16 == 0: both or none)
#pragma unroll
      for (int e = 0; e < 8; e += 2) m = larger(larger(m, fabsf(v[k][e])), fabsf(v[k][e + 1]));
      m = larger(m, __uint_as_float(dpp_from<0xB1, 0xF>(__float_as_uint(m))));  // quad_perm 1, 0, 3, 2
      if (!me.has[k]) continue;
      float q;
      const uint32_t sf = block_scale(m, G, q);
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = v[k][e] * q;
      *reinterpret_cast<uint32_t*>(y + (me.at[k] >> 1)) = enc_e2m1x8(f);
      if ((me.lane & 1) == 0) ys[me.at[k] >> 4] = (uint8_t)sf;
    }
  }
}

// ---- backward -----------------------------------------------------------------------
// A worker takes `run` consecutive rows and sums, over the rows of one group, dy n, dy and c h' (before its weight) for
// its columns in registers; when the group changes, and at the end, the sums go to slot (worker + group) of the
// workspace, [slot][3][dim] (no two have the same: the group grows from slot to slot where the worker does not). A
// second kernel adds the slots of each group in their order, and a third the groups for the gradients that all share.

enum { kSumScale = 1, kSumShift = 2, kSumGate = 4 };  // which of the three sums a call needs

// A row's tensors stay as they are in memory and are taken to fp32 again in each of its passes: (A) the means, (B) the
// sizes and, with them, the sums along the gradient, (C) the gradients; with a post norm also (D) the sums along the
// branch's. The next row's loads are under way meanwhile.
template <class E, bool ONE, int C, bool GROUPED, bool POST>
__global__ __launch_bounds__(ONE ? 256 : kBackwardThreads) void block_norm_backward(NormBackward a, int run, int need,
                                                                                    float* part_sums) {
  typedef typename E::elem elem;
  __shared__ Slots slots;
  const NormArgs& n = a.n;
  const Place<ONE, C> me(n.dim);
  const int first = me.worker * run, limit = group_limit(n.groups);
  const int last = limit - first < run ? limit : first + run;
  if (first >= last) return;  // (the whole worker)
  const float inv_dim = 1.0f / (float)n.dim;
  const bool layer = n.norm == BSQ_NORM_LAYER, post_layer = n.post == BSQ_NORM_LAYER;
  const bool normed = n.norm != BSQ_NORM_NONE;
  float sums[3][C][8];
#pragma unroll
  for (int k = 0; k < C; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) sums[0][k][e] = sums[1][k][e] = sums[2][k][e] = 0.0f;
  auto flush = [&](int g) {
    float* to = part_sums + (int64_t)(me.worker + g) * 3 * n.dim;
#pragma unroll
    for (int q = 0; q < 3; ++q)
#pragma unroll
      for (int k = 0; k < C; ++k) {
        if ((need >> q & 1) && me.has[k]) store8<Fp32>(to + (int64_t)q * n.dim + me.at[k], sums[q][k]);
#pragma unroll
        for (int e = 0; e < 8; ++e) sums[q][k][e] = 0.0f;
      }
  };
  constexpr bool kHold = C * sizeof(elem) <= 8, kAhead = kHold && (!POST || C == 1);  // (as registers allow)
  struct Row {
    Chunk<E> x[C], dy[C], dx[C], h[C];
  } now, next;
  auto load_row = [&](Row& r, int row) {
    me.load(r.x, normed ? row_of<E>(a.x_out, row) : nullptr);
    me.load(r.dy, normed ? row_of<E>(a.dy, row) : nullptr);
    me.load(r.h, row_of<E>(a.branch, row));
    me.load(r.dx, row_of<E>(a.dx_out, row));
  };
  Vector<E, C, kHold && !GROUPED> weight, pw;
  Vector<E, C, kHold && GROUPED> scale, gate;
  if constexpr (kAhead) load_row(next, first);
  weight.set(me, row_of<E>(n.weight));
  pw.set(me, row_of<E>(n.post_weight));
  int g = GROUPED ? -1 : 0, end = first;  // (without vectors of groups all rows count as one's)
  for (int row = first; row < last; ++row) {
    if (GROUPED && row >= end) {
      if (g >= 0 && need) flush(g);
      g = group_of_wave(n.groups, row, me.lane);
      end = group_end(n.groups, g);
      scale.set(me, row_of<E>(n.scale, g));
      gate.set(me, row_of<E>(n.gate, g));
    }
    if constexpr (kAhead) {
      now = next;
      if (row + 1 < last) load_row(next, row + 1);
    } else {
      load_row(now, row);
    }
    RowSums<ONE> rs{&slots, me.part, me.parts, me.lane, row, 0};
    // dy (1 + scale) weight of chunk k
    auto scaled = [&](int k, const float (&dy)[8], float (&d)[8]) {
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] = dy[e];
      float w[8];
      if (GROUPED && scale.p) {
        scale.get(me, k, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = fmaf(d[e], w[e], d[e]);
      }
      if (weight.p) {
        weight.get(me, k, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] *= w[e];
      }
    };
    // A
    float mean = 0.0f, post_mean = 0.0f;
    if (layer || (POST && post_layer)) {
      float t[2] = {0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < C; ++k) {
        float f[8];
        if (layer) {
          now.x[k].get(f);
#pragma unroll
          for (int e = 0; e < 8; ++e) t[0] += f[e];
        }
        if (POST && post_layer) {
          now.h[k].get(f);
#pragma unroll
          for (int e = 0; e < 8; ++e) t[1] += f[e];
        }
      }
      rs.sum(t);
      mean = t[0] * inv_dim;
      post_mean = t[1] * inv_dim;
    }
    // B
    float r = 0.0f, along = 0.0f, level = 0.0f, hr = 1.0f;
    if (normed || POST) {
      float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int k = 0; k < C; ++k) {
        if (!me.has[k]) continue;
        float f[8], d[8];
        if (normed) {
          now.x[k].get(f);
          float dy[8];
          now.dy[k].get(dy);
          scaled(k, dy, d);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float v = f[e] - mean;
            t[0] = fmaf(v, v, t[0]);
            t[1] = fmaf(d[e], v, t[1]);
            t[2] += d[e];
          }
        }
        if constexpr (POST) {
          now.h[k].get(f);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float v = f[e] - post_mean;
            t[3] = fmaf(v, v, t[3]);
          }
        }
      }
      rs.sum(t);
      r = normed ? 1.0f / sqrtf(t[0] * inv_dim + n.eps) : 0.0f;
      along = t[1] * r * inv_dim;
      level = layer ? t[2] * inv_dim : 0.0f;
      if constexpr (POST) hr = 1.0f / sqrtf(t[3] * inv_dim + n.post_eps);
    }
    // C
    float o[POST ? C : 1][8], hn[POST ? C : 1][8];
    float t[2] = {0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < C; ++k) {
      if (!me.has[k]) continue;
      float c[8], f[8], w[8];
      now.dx[k].get(c);
      if (normed) {
        float dy[8], d[8];
        now.x[k].get(f);
        now.dy[k].get(dy);
        scaled(k, dy, d);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float v = (f[e] - mean) * r;
          c[e] = fmaf(r, fmaf(-v, along, d[e] - level), c[e]);
          sums[0][k][e] = fmaf(dy[e], v, sums[0][k][e]);
          sums[1][k][e] += dy[e];
        }
      }
      if (a.dx.p) store8<E>(out_of<E>(a.dx, row) + me.at[k], c);
      now.h[k].get(f);  // (0 without a branch)
      if constexpr (POST) {
#pragma unroll
        for (int e = 0; e < 8; ++e) hn[k][e] = f[e] = (f[e] - post_mean) * hr;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sums[2][k][e] = fmaf(c[e], f[e], sums[2][k][e]);
      if (!a.dbranch.p) continue;
      if (GROUPED && gate.p) {
        gate.get(me, k, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) c[e] *= w[e];
      }
      if constexpr (POST) {
        if (pw.p) {
          pw.get(me, k, w);
#pragma unroll
          for (int e = 0; e < 8; ++e) c[e] *= w[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          o[k][e] = c[e];
          t[0] = fmaf(c[e], f[e], t[0]);
          t[1] += c[e];
        }
      } else {
        store8<E>(out_of<E>(a.dbranch, row) + me.at[k], c);
      }
    }
    // D
    if (POST && a.dbranch.p) {
      rs.sum(t);
      const float post_along = t[0] * inv_dim, post_level = post_layer ? t[1] * inv_dim : 0.0f;
#pragma unroll
      for (int k = 0; k < (POST ? C : 0); ++k) {
        if (!me.has[k]) continue;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[k][e] = hr * fmaf(-hn[k][e], post_along, o[k][e] - post_level);
        store8<E>(out_of<E>(a.dbranch, row) + me.at[k], o[k]);
      }
    }
  }
  if (need) flush(g);
}

template <class E>
__device__ __forceinline__ float one(const void* p, int64_t at) {
  if constexpr (sizeof(typename E::elem) == 4) return static_cast<const float*>(p)[at];
  else return E::up(static_cast<const uint16_t*>(p)[at]);
}
// Columns are taken four at a time, by 8 x 8 lanes of a wave (quadruple, share) and W waves: with 16 of them 128 threads
// share the sum of a column, so that a few hundred slots are a few loads each (1001 x 1536 fp32, 48 workgroups: 6.4 us, with
// eight 8.2, with four 10.8); eight where there is more than a workgroup a compute unit (4608 x 2560 in five groups, 400
// workgroups: 9.2 us, with sixteen 12.2, with four 12.7); one wave where groups have few slots on average, since the starts
// are on the device (16384 x 512 in 200 groups: even ones 31.6 us for the whole gradient, one with all but 199 rows 258).
constexpr int kCols = 8;

__device__ __forceinline__ void add4(float4& a, float4 b) { a = make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w); }
// sums[q] over the threads of a column: whole in the first 8 threads of the workgroup
template <int W>
struct ColumnSlots {
  float4 s[3][W][kCols];
};
template <int W>
__device__ __forceinline__ void column_sums(float4 (&v)[3], int need, ColumnSlots<W>& slots) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
  for (int q = 0; q < 3; ++q) {
    if (!(need >> q & 1)) continue;
#pragma unroll
    for (int off = 8; off <= 32; off <<= 1)
      add4(v[q], make_float4(__shfl_xor(v[q].x, off, 64), __shfl_xor(v[q].y, off, 64), __shfl_xor(v[q].z, off, 64),
                             __shfl_xor(v[q].w, off, 64)));
    if (lane < kCols) slots.s[q][wave][lane] = v[q];
  }
  __syncthreads();
  if (threadIdx.x < kCols) {
#pragma unroll
    for (int q = 0; q < 3; ++q) {
      if (!(need >> q & 1)) continue;
      v[q] = slots.s[q][0][threadIdx.x];
#pragma unroll
      for (int w = 1; w < W; ++w) add4(v[q], slots.s[q][w][threadIdx.x]);
    }
  }
  __syncthreads();  // (the slots are free again)
}
__device__ __forceinline__ float4 fma4(float4 a, float4 b, float4 c) {
  return make_float4(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y), fmaf(a.z, b.z, c.z), fmaf(a.w, b.w, c.w));
}
template <class E>
__device__ __forceinline__ float4 four(const void* p, int64_t at) {
  return make_float4(one<E>(p, at), one<E>(p, at + 1), one<E>(p, at + 2), one<E>(p, at + 3));
}
__device__ __forceinline__ void put4(float* p, int64_t at, float4 v) {  // (gradients are 4-byte aligned)
  p[at] = v.x; p[at + 1] = v.y; p[at + 2] = v.z; p[at + 3] = v.w;
}

// the gradients that all groups share, from the sums of one group (or of all)
template <class E>
__device__ __forceinline__ void add_shared(const NormBackward& a, int g, int col, const float4 (&s)[3], float4 (&t)[3]) {
  float4 m = make_float4(1, 1, 1, 1), k = m;
  if (a.n.scale.p) add4(m, four<E>(a.n.scale.p, (int64_t)g * a.n.scale.stride + col));
  if (a.n.gate.p) k = four<E>(a.n.gate.p, (int64_t)g * a.n.gate.stride + col);
  t[0] = fma4(m, s[0], t[0]);
  t[1] = fma4(m, s[1], t[1]);
  t[2] = fma4(k, s[2], t[2]);
}
__device__ __forceinline__ void put_shared(const NormBackward& a, int col, const float4 (&t)[3]) {
  if (a.dweight) put4(a.dweight, col, t[0]);
  if (a.dbias) put4(a.dbias, col, t[1]);
  if (a.dpost_weight) put4(a.dpost_weight, col, t[2]);
}

// the workers of group g's rows: first to last (none: last < first); whether it has rows
__device__ __forceinline__ bool workers_of_group(const RowGroups& rg, int g, int run, int& first, int& last) {
  int r0, r1;
  if (rg.starts) {
    const int limit = group_limit(rg);  // (the first group starts at 0, the last one ends there)
    r0 = g == 0 ? 0 : rg.starts[g];
    r1 = g == rg.groups - 1 ? limit : rg.starts[g + 1];
    r0 = r0 < 0 ? 0 : r0;
    r1 = r1 < limit ? r1 : limit;
  } else {
    r0 = g * rg.per;
    r1 = r0 + rg.per;
  }
  first = r1 > r0 ? r0 / run : 0;
  last = r1 > r0 ? (r1 - 1) / run : -1;
  return r1 > r0;
}
// this thread's share of group g's slots, four columns of each sum; whether the group has rows (the vectors of one
// without may hold anything, NaN too, and do not count)
__device__ __forceinline__ bool slot_share(const NormBackward& a, int g, int run, int need, const float* part_sums,
                                           int col, int share, int shares, float4 (&s)[3]) {
  int w, last;
  const bool any = workers_of_group(a.n.groups, g, run, w, last);
#pragma unroll 4
  for (w += share; w <= last; w += shares) {
    const float* p = part_sums + (int64_t)(w + g) * 3 * a.n.dim + col;
#pragma unroll
    for (int q = 0; q < 3; ++q)
      if (need >> q & 1) add4(s[q], *reinterpret_cast<const float4*>(p + (int64_t)q * a.n.dim));
  }
  return any;
}

// The sums of the slots: grid.x over columns, grid.y (striding) over groups, starting with `from`, for the gradients that
// each has of its own and, for `shared`, one more for those that all share. With `group_sums` [groups][3][dim] the groups'
// sums go there too, for norm_shared_sums.
template <class E, int W>
__global__ __launch_bounds__(64 * W) void norm_group_sums(NormBackward a, int run, int need, int from,
                                                           int shared, const float* part_sums, float* group_sums) {
  __shared__ ColumnSlots<W> slots;
  const int share = threadIdx.x / kCols, col = 4 * (int)(blockIdx.x * kCols + threadIdx.x % kCols);
  const bool live = col < a.n.dim;
  const int groups = a.n.groups.groups;
  for (int g = from + blockIdx.y; g < groups + shared; g += gridDim.y) {
    float4 s[3] = {};
    bool any = false;
    if (g == groups) {
      for (int o = 0; o < groups && live; ++o) {
        float4 t[3] = {};
        if (slot_share(a, o, run, need, part_sums, col, share, 8 * W, t)) add_shared<E>(a, o, col, t, s);
      }
    } else if (live) {
      any = slot_share(a, g, run, need, part_sums, col, share, 8 * W, s);
    }
    column_sums(s, need, slots);
    if (!live || share != 0) continue;
    if (g == groups) {
      put_shared(a, col, s);
      continue;
    }
    const int64_t at = (int64_t)g * a.n.dim + col;
    if (a.dscale) {
      float4 d = s[0];
      const float4 zero = make_float4(0, 0, 0, 0);
      if (any && a.n.weight) d = fma4(d, four<E>(a.n.weight, col), zero);
      if (any && a.n.bias) d = fma4(four<E>(a.n.bias, col), s[1], d);
      put4(a.dscale, at, d);
    }
    if (a.dshift) put4(a.dshift, at, s[1]);
    if (a.dgate)
      put4(a.dgate, at,
           any && a.n.post_weight ? fma4(s[2], four<E>(a.n.post_weight, col), make_float4(0, 0, 0, 0)) : s[2]);
    if (group_sums) {
#pragma unroll
      for (int q = 0; q < 3; ++q) put4(group_sums, ((int64_t)g * 3 + q) * a.n.dim + col, s[q]);
    }
  }
}

template <class E, int W>
__global__ __launch_bounds__(64 * W) void norm_shared_sums(NormBackward a, int run, const float* group_sums) {
  __shared__ ColumnSlots<W> slots;
  const int share = threadIdx.x / kCols, col = 4 * (int)(blockIdx.x * kCols + threadIdx.x % kCols);
  const bool live = col < a.n.dim;
  float4 t[3] = {};
  if (live) {
    for (int g = share; g < a.n.groups.groups; g += 8 * W) {
      int w, last;
      if (!workers_of_group(a.n.groups, g, run, w, last)) continue;
      float4 s[3];
#pragma unroll
      for (int q = 0; q < 3; ++q)
        s[q] = *reinterpret_cast<const float4*>(group_sums + ((int64_t)g * 3 + q) * a.n.dim + col);
      add_shared<E>(a, g, col, s, t);
    }
  }
  column_sums(t, 7, slots);
  if (live && share == 0) put_shared(a, col, t);
}

// a call without rows: the gradients of the vectors are sums over nothing
__global__ __launch_bounds__(256) void zero(float* p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) p[i] = 0.0f;
}

// One chunk a lane up to here in the forward pass, two beyond (8192 x 5120 bf16 into fp8r: 65 us against 77 with one).
constexpr int kForwardOne = 2048;
// Waves a compute unit and least rows a worker in the backward pass. 4608 x 2560 bf16: 12 waves 47 us, 8 waves 70, 16 and
// 20 waves 54 and 65 (workers of five waves do not share out evenly over four SIMDs); a worker of fewer rows writes
// sums for fewer (1001 x 1536 fp32: 4 rows 24 us, 2 rows 31, 1 row 59).
constexpr int kBackwardWaves = 12, kBackwardRows = 4;
constexpr int kGroupsAlong = 64;  // up to here the sums that all groups share are taken along with the groups' own

// ---- launches -----------------------------------------------------------------------

// f(whether a worker is one wave, chunks of a lane, whether groups have vectors); waves of a worker
template <class F>
hipError_t with_groups(const NormArgs& n, F f) {
  return n.scale.p || n.shift.p || n.gate.p ? f(std::true_type{}) : f(std::false_type{});
}
template <int C>
using chunks_t = std::integral_constant<int, C>;
int waves_of(int64_t dim, int chunks) { return (int)((dim + 512 * chunks - 1) / (512 * chunks)); }

template <class E>
hipError_t forward(const NormForward& a, hipStream_t s) {
  return with_groups(a.n, [&](auto grouped) {
    constexpr bool G = decltype(grouped)::value;
    const unsigned rows = (unsigned)a.n.rows;
    if (a.n.dim <= 512)
      hipLaunchKernelGGL((block_norm<E, true, 1, G>), dim3((rows + 3) / 4), dim3(256), 0, s, a);
    else if (a.n.dim <= kForwardOne)
      hipLaunchKernelGGL((block_norm<E, false, 1, G>), dim3(rows), dim3(64 * waves_of(a.n.dim, 1)), 0, s, a);
    else
      hipLaunchKernelGGL((block_norm<E, false, 2, G>), dim3(rows), dim3(64 * waves_of(a.n.dim, 2)), 0, s, a);
    return hipGetLastError();
  });
}

int backward_chunks(int64_t dim) { return dim <= 4096 ? 1 : dim <= 8192 ? 2 : dim <= 12288 ? 3 : 4; }
// Rows of a worker: so many that the workers fill the 256 compute units once, kBackwardWaves on each, and at least
// kBackwardRows, since each worker's sums are written once and read once
int backward_run(int64_t rows, int64_t dim) {
  const int w = waves_of(dim, backward_chunks(dim));
  const int64_t workers = 256 * (int64_t)(kBackwardWaves / w > 0 ? kBackwardWaves / w : 1);
  const int64_t n = (rows + workers - 1) / workers;
  return (int)(n < kBackwardRows ? kBackwardRows : n);
}
size_t pad256(size_t n) { return (n + 255) & ~(size_t)255; }
size_t slot_bytes(int64_t rows, int64_t dim, int64_t groups) {
  const int run = backward_run(rows, dim);
  return pad256((size_t)((rows + run - 1) / run + groups) * 3 * (size_t)dim * 4);
}

template <class E>
hipError_t backward(const NormBackward& a, void* workspace, hipStream_t s) {
  if (a.n.rows == 0) {
    const int64_t all = (int64_t)a.n.groups.end * a.n.dim;
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
  const int run = backward_run(a.n.rows, a.n.dim), workers = (a.n.rows + run - 1) / run, groups = a.n.groups.groups;
  const int need = (a.dscale || a.dweight ? kSumScale : 0) |
                   (a.dshift || a.dbias || (a.dscale && a.n.bias) ? kSumShift : 0) |
                   (a.dgate || a.dpost_weight ? kSumGate : 0);
  float* parts = static_cast<float*>(workspace);
  hipError_t e = with_groups(a.n, [&](auto grouped) {
    constexpr bool G = decltype(grouped)::value;
    const int chunks = backward_chunks(a.n.dim);
    const bool one = a.n.dim <= 512;
    const unsigned blocks = one ? (workers + 3) / 4 : workers, threads = one ? 256u : 64u * waves_of(a.n.dim, chunks);
    auto go = [&](auto o, auto c) {
      constexpr bool ONE = decltype(o)::value;
      constexpr int C = decltype(c)::value;
      if (a.branch.p && a.n.post != BSQ_NORM_NONE)
        hipLaunchKernelGGL((block_norm_backward<E, ONE, C, G, true>), dim3(blocks), dim3(threads), 0, s, a, run, need,
                           parts);
      else
        hipLaunchKernelGGL((block_norm_backward<E, ONE, C, G, false>), dim3(blocks), dim3(threads), 0, s, a, run, need,
                           parts);
      return hipGetLastError();
    };
    if (one) return go(std::true_type{}, chunks_t<1>{});
    if (chunks == 1) return go(std::false_type{}, chunks_t<1>{});
    if (chunks == 2) return go(std::false_type{}, chunks_t<2>{});
    if (chunks == 3) return go(std::false_type{}, chunks_t<3>{});
    return go(std::false_type{}, chunks_t<4>{});
  });
  if (e != hipSuccess || !need) return e;
  // what all groups share: along with the groups' own, or after them where there are many
  const bool shared = a.dweight || a.dbias || a.dpost_weight, own = a.dscale || a.dshift || a.dgate;
  float* sums = nullptr;
  if (shared && groups > kGroupsAlong)
    sums = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + slot_bytes(a.n.rows, a.n.dim, groups));
  const int along = shared && !sums ? 1 : 0, from = own || sums ? 0 : groups, jobs = groups + along - from;
  const unsigned cols = (unsigned)((a.n.dim + 4 * kCols - 1) / (4 * kCols));
  const dim3 grid(cols, (unsigned)(jobs < 65535 ? jobs : 65535));
  if (workers / groups < 16 && (!along || workers < 64))
    hipLaunchKernelGGL((norm_group_sums<E, 1>), grid, dim3(64), 0, s, a, run, need, from, along, parts, sums);
  else if ((int64_t)cols * grid.y > 256)
    hipLaunchKernelGGL((norm_group_sums<E, 8>), grid, dim3(512), 0, s, a, run, need, from, along, parts, sums);
  else
    hipLaunchKernelGGL((norm_group_sums<E, 16>), grid, dim3(1024), 0, s, a, run, need, from, along, parts, sums);
  if ((e = hipGetLastError()) != hipSuccess || !sums) return e;
  hipLaunchKernelGGL((norm_shared_sums<E, 16>), dim3(cols), dim3(1024), 0, s, a, run, sums);
  return hipGetLastError();
}

}  // namespace

size_t block_norm_workspace(int64_t rows, int64_t dim, int64_t groups) {
  return slot_bytes(rows, dim, groups) + (groups > kGroupsAlong ? (size_t)groups * 3 * (size_t)dim * 4 : 0);
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
