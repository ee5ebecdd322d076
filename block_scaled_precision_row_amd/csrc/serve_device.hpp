// Device helpers of the token-serving kernels: the two 16-bit types, and the angles of a rotation.
#pragma once

#include "bsq_device.hpp"
#include "serve_launch.hpp"

namespace bsq {

struct Bf16 {
  typedef uint16_t elem;
  typedef v8bf vec8;
  typedef v2bf vec2;
  static constexpr bool is_half = false;
  static __device__ __forceinline__ float up(uint32_t bits) { return __uint_as_float(bits << 16); }
  static __device__ __forceinline__ float lo(uint32_t w) { return bf16_lo(w); }
  static __device__ __forceinline__ float hi(uint32_t w) { return bf16_hi(w); }
  static __device__ __forceinline__ uint32_t pack(float a, float b) { return pack_bf16x2(a, b); }
  static __device__ __forceinline__ v4f mfma(vec8 a, vec8 b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ v16f mfma32(vec8 a, vec8 b, v16f c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
  }
  // two E4M3 codes (half `h` of w) times 2^exponent(scale)
  template <bool h>
  static __device__ __forceinline__ vec2 dec(uint32_t w, float scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, scale, h);
  }
};
struct Fp16 {
  typedef uint16_t elem;
  typedef v8h vec8;
  typedef v2h vec2;
  static constexpr bool is_half = true;
  static __device__ __forceinline__ float up(uint32_t bits) {
    union { uint16_t u; _Float16 h; } c;
    c.u = (uint16_t)bits;
    return (float)c.h;
  }
  static __device__ __forceinline__ float lo(uint32_t w) { return up(w & 0xFFFFu); }
  static __device__ __forceinline__ float hi(uint32_t w) { return up(w >> 16); }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    union { v2h v; uint32_t u; } r;
    r.v = v2h{(_Float16)a, (_Float16)b};
    return r.u;
  }
  static __device__ __forceinline__ v4f mfma(vec8 a, vec8 b, v4f c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
  static __device__ __forceinline__ v16f mfma32(vec8 a, vec8 b, v16f c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
  }
  template <bool h>
  static __device__ __forceinline__ vec2 dec(uint32_t w, float scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w, scale, h);
  }
};
struct Fp32 {
  typedef float elem;
};

// eight consecutive elements as fp32, 16-byte (16-bit types) or 2 x 16-byte accesses
template <class T>
__device__ __forceinline__ void unpack8(uint4 v, float (&f)[8]) {
  f[0] = T::lo(v.x); f[1] = T::hi(v.x); f[2] = T::lo(v.y); f[3] = T::hi(v.y);
  f[4] = T::lo(v.z); f[5] = T::hi(v.z); f[6] = T::lo(v.w); f[7] = T::hi(v.w);
}
template <class T>
__device__ __forceinline__ void load8(const typename T::elem* p, float (&f)[8]) {
  unpack8<T>(*reinterpret_cast<const uint4*>(p), f);
}
template <>
__device__ __forceinline__ void load8<Fp32>(const float* p, float (&f)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
template <class T>
__device__ __forceinline__ void store8(typename T::elem* p, const float (&f)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(T::pack(f[0], f[1]), T::pack(f[2], f[3]), T::pack(f[4], f[5]), T::pack(f[6], f[7]));
}
template <>
__device__ __forceinline__ void store8<Fp32>(float* p, const float (&f)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// Cos and sin of position * w, times `factor`, in 64 bits (whose vector instructions take as long as those of 32
// here): the angle as a fraction of a turn, less whole quarters, and the Taylor series on what is left, at most pi / 4:
// the first terms left out are x^15 / 15! and x^14 / 14!, below 4e-13. The product of position and w and its part of a turn
// are formed with what their roundings leave (1 / 2 pi in two parts), so that the fraction is off by 2^-53 of a turn at
// any position below 2^53; without it by 2^-53 of all turns, 2^-22 at 2^31, of which one key's code in a million comes out
// wrong, and everything at 2^53.
struct Turn {
  double c, s;
};
__device__ __forceinline__ Turn rope_turn(double position, float w, float factor) {
  const double a0 = position * (double)w, a1 = fma(position, (double)w, -a0);
  constexpr double kTurn = 0.15915494309189535, kTurnRest = -9.839338337591243e-18;
  double t = a0 * kTurn;
  const double rest = fma(a0, kTurn, -t) + fma(a0, kTurnRest, a1 * kTurn);
  t = t - rint(t) + rest;
  const double quarter = rint(4.0 * t);
  const double x = fma(quarter, -0.25, t) * 6.283185307179586476925, z = x * x;
  double s = fma(z, 1.0 / 6227020800.0, -1.0 / 39916800.0), c = fma(z, 1.0 / 479001600.0, -1.0 / 3628800.0);
  s = fma(z, s, 1.0 / 362880.0);
  c = fma(z, c, 1.0 / 40320.0);
  s = fma(z, s, -1.0 / 5040.0);
  c = fma(z, c, -1.0 / 720.0);
  s = fma(z, s, 1.0 / 120.0);
  c = fma(z, c, 1.0 / 24.0);
  s = fma(z, s, -1.0 / 6.0);
  c = fma(z, c, -0.5);
  s = fma(x * z, s, x);
  c = fma(z, c, 1.0);
  const int q = (int)quarter & 3;
  double a = q & 1 ? s : c, b = q & 1 ? c : s;
  a = q == 1 || q == 2 ? -a : a;
  b = q >= 2 ? -b : b;
  return Turn{a * (double)factor, b * (double)factor};
}
__device__ __forceinline__ float2 rope_angle(double position, float w, float factor) {
  const Turn t = rope_turn(position, w, factor);
  return make_float2((float)t.c, (float)t.s);
}

// x in fp32 with the last bit set where that is not exact: a later rounding to fewer bits (after a power of two)
// then falls as it would from x itself
__device__ __forceinline__ float to_odd(double x) {
  const float f = (float)x;
  const double back = (double)f;
  uint32_t u = __float_as_uint(f);
  if (back != x) u = (fabs(back) > fabs(x) ? u - 1 : u) | 1u;
  return __uint_as_float(u);
}

}  // namespace bsq
