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

// cos and sin of position * w, times `factor`. The product is formed in 64 bits and reduced to a
// fraction of a turn there (a position of 10^6 keeps 10^-10 of a turn); the remaining angle,
// below half a turn, is rounded to fp32, an error of at most 2^-25 pi.
__device__ __forceinline__ float2 rope_angle(double position, float w, float factor) {
  double turns = position * (double)w * 0.15915494309189533577;
  turns -= rint(turns);
  float s, c;
  sincospif((float)(2.0 * turns), &s, &c);
  return make_float2(c * factor, s * factor);
}

}  // namespace bsq
