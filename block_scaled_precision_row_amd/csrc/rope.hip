// Rotary positions: y = f * R(+-p w_i) x over pairs of a head's first `rot` elements.
//
// Bound by memory: every element is read and written once; an angle costs some 55 instructions
// and serves all heads of its token, so a workgroup first puts the cosines and sines of its tokens
// into LDS and then streams the tokens' heads, 16 bytes of each half of eight pairs (four of fp32) a thread and step.
// 8192 tokens of 40 heads of 128, fp16: 168 MB in 32.8 us, 5.1 TB/s, what a copy reaches; 48 tokens of 40 heads 3.1 us, a launch.
//
// With several axes (bsq_rope_axes) the angles take their pair's axis' position, and nothing else changes: 14400 tokens
// of 48 heads of 128, bf16, three axes: 354 MB in 65 us, 5.4 TB/s.
#include "block_launch.hpp"
#include "serve_device.hpp"

namespace bsq {

namespace {

struct RopeArgs {
  const void* x;
  void* y;
  int64_t xt, xh, yt, yh;
  const int64_t* pos;
  const float* inv_freq;
  float factor;
  int rot;
  int64_t T;
  int H, D;
  int tokens, heads;  // per workgroup
};

struct OneAxis {
  __device__ __forceinline__ int64_t position(const int64_t* pos, int64_t t, int) const { return pos[t]; }
};
struct Axes {
  RopeAxes a;
  __device__ __forceinline__ int64_t position(const int64_t* pos, int64_t t, int pair) const {
    int c;
    if (a.cycled) {
      const int turn = pair / a.axes;
      c = pair - turn * a.axes;
      const int has = c == 0 ? a.sections[0] : c == 1 ? a.sections[1] : c == 2 ? a.sections[2] : a.sections[3];
      if (turn >= has) c = 0;
    } else {  // (sections past the last axis are 0 and the pairs before it fewer than all)
      int end = a.sections[0];
      c = 0;
#pragma unroll
      for (int i = 1; i < 4; ++i) {
        c += i < a.axes && pair >= end ? 1 : 0;
        end += a.sections[i];
      }
    }
    return pos[t * a.pos_t + c * a.pos_a];
  }
};

// P pairs per thread and step, in two 16-byte accesses: eight pairs, four of fp32 (with eight, whose lanes are 64 bytes
// apart, the fp32 gradient of 5001 x 24 x 128 took 32 us); rot % 16 == 0, D % 16 == 0
template <class E>
constexpr int pairs_of() { return sizeof(typename E::elem) == 4 ? 4 : 8; }
template <class E>
__device__ __forceinline__ void load_step(const typename E::elem* p, float (&f)[pairs_of<E>()]) { load8<E>(p, f); }
template <>
__device__ __forceinline__ void load_step<Fp32>(const float* p, float (&f)[4]) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
}
template <class E>
__device__ __forceinline__ void store_step(typename E::elem* p, const float (&f)[pairs_of<E>()]) { store8<E>(p, f); }
template <>
__device__ __forceinline__ void store_step<Fp32>(float* p, const float (&f)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
}

template <class E, bool INTER, bool BACK, class X>
__global__ __launch_bounds__(256) void rope_vec(RopeArgs a, X axes) {
  extern __shared__ float2 cs[];  // [tokens][rot / 2]
  typedef typename E::elem elem;
  const int64_t t0 = (int64_t)blockIdx.x * a.tokens;
  const int h0 = blockIdx.y * a.heads;
  const int nt = (int)(a.T - t0 < a.tokens ? a.T - t0 : a.tokens);
  const int nh = a.H - h0 < a.heads ? a.H - h0 : a.heads;
  const int half = a.rot >> 1;
  for (int i = threadIdx.x; i < nt * half; i += 256) {
    const int t = i / half;
    float2 v = rope_angle((double)axes.position(a.pos, t0 + t, i - t * half), a.inv_freq[i - t * half], a.factor);
    if (BACK) v.y = -v.y;
    cs[i] = v;
  }
  __syncthreads();
  constexpr int P = pairs_of<E>();
  const int units = a.D / (2 * P);
  const int per_token = nh * units;
  for (int i = threadIdx.x; i < nt * per_token; i += 256) {
    const int t = i / per_token, r = i - t * per_token, h = r / units, u = r - h * units;
    const elem* x = static_cast<const elem*>(a.x) + (t0 + t) * a.xt + (int64_t)(h0 + h) * a.xh;
    elem* y = static_cast<elem*>(a.y) + (t0 + t) * a.yt + (int64_t)(h0 + h) * a.yh;
    const bool turned = 2 * P * u < a.rot;
    const int e0 = turned && !INTER ? P * u : 2 * P * u;
    const int e1 = turned && !INTER ? P * u + half : 2 * P * u + P;
    float p[P], q[P];
    load_step<E>(x + e0, p);
    load_step<E>(x + e1, q);
    if (turned) {
      const float2* c = cs + t * half + P * u;
      if (INTER) {
#pragma unroll
        for (int j = 0; j < P / 2; ++j) {
          const float2 c0 = c[j], c1 = c[j + P / 2];
          const float a0 = p[2 * j], b0 = p[2 * j + 1], a1 = q[2 * j], b1 = q[2 * j + 1];
          p[2 * j] = a0 * c0.x - b0 * c0.y;
          p[2 * j + 1] = b0 * c0.x + a0 * c0.y;
          q[2 * j] = a1 * c1.x - b1 * c1.y;
          q[2 * j + 1] = b1 * c1.x + a1 * c1.y;
        }
      } else {
#pragma unroll
        for (int j = 0; j < P; ++j) {
          const float2 v = c[j];
          const float b = q[j];
          q[j] = b * v.x + p[j] * v.y;
          p[j] = p[j] * v.x - b * v.y;
        }
      }
    }
    store_step<E>(y + e0, p);
    store_step<E>(y + e1, q);
  }
}

template <class E>
__device__ __forceinline__ float load1(const typename E::elem* p) { return E::up(*p); }
template <>
__device__ __forceinline__ float load1<Fp32>(const float* p) { return *p; }
template <class E>
__device__ __forceinline__ void store1(typename E::elem* p, float v) { *p = (uint16_t)E::pack(v, 0.0f); }
template <>
__device__ __forceinline__ void store1<Fp32>(float* p, float v) { *p = v; }

// any rot, D, strides and alignment: a pair or a copied element per thread and step, the angle
// formed by each thread
template <class E, class X>
__global__ __launch_bounds__(256) void rope_any(RopeArgs a, X axes, bool inter, bool back) {
  typedef typename E::elem elem;
  const int half = a.rot >> 1, work = half + a.D - a.rot;
  const int64_t n = a.T * a.H * work;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int64_t th = i / work, t = th / a.H;
    const int u = (int)(i - th * work), h = (int)(th - t * a.H);
    const elem* x = static_cast<const elem*>(a.x) + t * a.xt + (int64_t)h * a.xh;
    elem* y = static_cast<elem*>(a.y) + t * a.yt + (int64_t)h * a.yh;
    if (u >= half) {
      y[u + half] = x[u + half];
      continue;
    }
    float2 v = rope_angle((double)axes.position(a.pos, t, u), a.inv_freq[u], a.factor);
    if (back) v.y = -v.y;
    const int e0 = inter ? 2 * u : u, e1 = inter ? 2 * u + 1 : u + half;
    const float p = load1<E>(x + e0), q = load1<E>(x + e1);
    store1<E>(y + e0, p * v.x - q * v.y);
    store1<E>(y + e1, q * v.x + p * v.y);
  }
}

template <class E, class X>
hipError_t launch(RopeArgs& a, const X& x, bool inter, bool back, bool vec, hipStream_t s) {
  if (!vec) {
    const int64_t n = a.T * a.H * (a.D - a.rot / 2);
    const int64_t blocks = (n + 255) / 256;
    hipLaunchKernelGGL((rope_any<E, X>), dim3((unsigned)(blocks < 16384 ? blocks : 16384)), dim3(256), 0, s, a, x, inter,
                       back);
    return hipGetLastError();
  }
  const dim3 grid((unsigned)((a.T + a.tokens - 1) / a.tokens), (unsigned)((a.H + a.heads - 1) / a.heads));
  const size_t lds = (size_t)a.tokens * (a.rot / 2) * sizeof(float2);
  if (inter && back) hipLaunchKernelGGL((rope_vec<E, true, true, X>), grid, dim3(256), lds, s, a, x);
  else if (inter) hipLaunchKernelGGL((rope_vec<E, true, false, X>), grid, dim3(256), lds, s, a, x);
  else if (back) hipLaunchKernelGGL((rope_vec<E, false, true, X>), grid, dim3(256), lds, s, a, x);
  else hipLaunchKernelGGL((rope_vec<E, false, false, X>), grid, dim3(256), lds, s, a, x);
  return hipGetLastError();
}

bool wide(const Strided& t, int bytes) {  // 16-byte accesses to every row
  const int per = 16 / bytes;
  return (reinterpret_cast<uintptr_t>(t.p) & 15) == 0 && t.st % per == 0 && t.sh % per == 0;
}

template <class X>
hipError_t launch_any(bsq_dtype dt, Strided x, const int64_t* positions, const X& axes, Rotation r, bool backward,
                      Strided y, int64_t T, int H, int D, hipStream_t s) {
  RopeArgs a{x.p, const_cast<void*>(y.p), x.st, x.sh, y.st, y.sh, positions, r.inv_freq, r.factor, r.rot, T, H, D, 1, H};
  const int bytes = dt == BSQ_FP32 ? 4 : 2;
  // (2^23 workgroups of 256 threads: the most that one dimension of a grid takes)
  const bool vec = r.rot % 16 == 0 && D % 16 == 0 && wide(x, bytes) && wide(y, bytes) && T < (int64_t)1 << 23;
  if (vec) {
    // about 512 steps to a workgroup where there are tokens enough, and otherwise
    // the heads spread so that a thread has one step
    const int per_head = D / (dt == BSQ_FP32 ? 8 : 16);
    const int64_t steps = (int64_t)H * per_head;
    if (T * steps >= (int64_t)1024 * 512) {
      int64_t n = 512 / steps;
      const int64_t fit = 32768 / (r.rot * 4);  // 32 KB of angles
      n = n < 1 ? 1 : (n > fit ? fit : n);
      a.tokens = (int)n;
      const int64_t most = (512 + per_head - 1) / per_head;  // heads of a very wide token are spread too
      if (H > 4 * most) a.heads = (int)most;
    } else {
      const int least = (256 + per_head - 1) / per_head;
      a.heads = H < least ? H : least;
      int64_t n = 256 / ((int64_t)a.heads * per_head);
      a.tokens = (int)(n < 1 ? 1 : (n > 16 ? 16 : n));
    }
  }
  if (dt == BSQ_BF16) return launch<Bf16>(a, axes, r.interleaved, backward, vec, s);
  if (dt == BSQ_FP16) return launch<Fp16>(a, axes, r.interleaved, backward, vec, s);
  return launch<Fp32>(a, axes, r.interleaved, backward, vec, s);
}

}  // namespace

hipError_t launch_rope(bsq_dtype dt, Strided x, const int64_t* positions, Rotation r, bool backward, Strided y,
                       int64_t T, int H, int D, hipStream_t s) {
  return launch_any(dt, x, positions, OneAxis{}, r, backward, y, T, H, D, s);
}

hipError_t launch_rope_axes(bsq_dtype dt, Strided x, const int64_t* positions, const RopeAxes& axes, Rotation r,
                            bool backward, Strided y, int64_t T, int H, int D, hipStream_t s) {
  return launch_any(dt, x, positions, Axes{axes}, r, backward, y, T, H, D, s);
}

}  // namespace bsq
