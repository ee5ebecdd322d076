// Few-token linears with 4-bit integer weights and group scales:
//   y[m][n] = sum_g s[n][g] * sum_{k in g} x[m][k] (c[n][k] - z[n][g]).
//
// 16 weight rows a workgroup, its waves taking every fourth stage of 128 K values; the products of
// 16 tokens run on 16x16x32 MFMA (A: x, B: W), 32 K values an instruction, so that a group's sum
// is complete in the accumulator before its scale is applied in fp32. A lane loads 16 bytes of a
// row (32 K values: whole 64-byte segments a row and stage); a 4 x 4 exchange of dwords between
// the four lanes of a row (four lane-swap instructions) then gives every lane eight values of each
// block of 32. Codes become 16-bit numbers by or-ing them into the mantissa of a power of two:
//   fp16: 1024 + c, from which a packed subtraction of 1024 + z leaves c - z exactly;
//   bf16 (no packed arithmetic): 128 + c stays, and the sum of x over the group, from one more
//   MFMA against ones, takes (128 + z) sum x away in fp32.
// The order of nibbles in a dword gives pairs (k, k + 4); x is put in the same order.
//
// Bound by memory: K / 2 bytes a row and its scales.
#include "serve_device.hpp"

namespace bsq {

namespace {

struct Args {
  const uint16_t* x;
  int64_t ldx;
  const uint8_t* w;
  const uint16_t* ws;
  const uint8_t* wz;
  uint16_t* y;
  int64_t ldy;
  int64_t M, N;
  int K;
};

template <class E>
union Frag {
  typename E::vec8 v;
  uint32_t u[4];
  uint4 q;
};

// dword e of lane group g becomes dword g of lane group e, over the four groups of 16 lanes
__device__ __forceinline__ void exchange(uint32_t (&d)[4]) {
  auto swap32 = [](uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    a = r[0];
    b = r[1];
  };
  auto swap16 = [](uint32_t& a, uint32_t& b) {
    const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    a = r[0];
    b = r[1];
  };
  swap32(d[0], d[2]);
  swap32(d[1], d[3]);
  swap16(d[0], d[1]);
  swap16(d[2], d[3]);
}

// the eight values of a dword as pairs (k, k + 4)
template <class E>
__device__ __forceinline__ typename E::vec8 codes8(uint32_t w, uint32_t minus) {
  constexpr uint32_t kMagic = E::is_half ? 0x64006400u : 0x43004300u;
  Frag<E> f;
#pragma unroll
  for (int i = 0; i < 4; ++i) f.u[i] = ((w >> (4 * i)) & 0x000F000Fu) | kMagic;
  if constexpr (E::is_half) {
    union { uint32_t u; v2h h; } c;
    c.u = minus;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      union { uint32_t u; v2h h; } t;
      t.u = f.u[i];
      t.h = t.h - c.h;
      f.u[i] = t.u;
    }
  }
  return f.v;
}
template <class E>
__device__ __forceinline__ typename E::vec8 paired(uint4 x) {
  Frag<E> f;
  f.u[0] = __builtin_amdgcn_perm(x.z, x.x, 0x05040100u);
  f.u[1] = __builtin_amdgcn_perm(x.z, x.x, 0x07060302u);
  f.u[2] = __builtin_amdgcn_perm(x.w, x.y, 0x05040100u);
  f.u[3] = __builtin_amdgcn_perm(x.w, x.y, 0x07060302u);
  return f.v;
}

template <class E, int TM, int GROUP>
__global__ __launch_bounds__(256) void int4_mfma(Args a) {
  __shared__ float sh[3][TM][64][4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, kq = lane >> 4;
  const int64_t n0 = (int64_t)blockIdx.x * 16, m0 = (int64_t)blockIdx.y * (16 * TM);
  const int64_t n = n0 + col < a.N ? n0 + col : a.N - 1;
  const int groups = a.K / GROUP;
  const uint8_t* wr = a.w + n * (a.K / 2);
  const uint16_t* sr = a.ws + n * groups;
  const uint8_t* zr = a.wz ? a.wz + n * groups : nullptr;
  const uint16_t* xr[TM];
  bool live[TM];
#pragma unroll
  for (int t = 0; t < TM; ++t) {
    const int64_t m = m0 + 16 * t + col;
    live[t] = m < a.M;
    xr[t] = a.x + (live[t] ? m : 0) * a.ldx + 8 * kq;
  }
  Frag<E> ones;
  ones.q = E::is_half ? make_uint4(0, 0, 0, 0) : make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
  v4f acc[TM];
#pragma unroll
  for (int t = 0; t < TM; ++t) acc[t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  for (int k0 = 128 * wave; k0 < a.K; k0 += 512) {
    uint4 wv = make_uint4(0, 0, 0, 0);
    if (k0 + 32 * kq < a.K) wv = *reinterpret_cast<const uint4*>(wr + (k0 >> 1) + 16 * kq);
    uint32_t d[4] = {wv.x, wv.y, wv.z, wv.w};
    exchange(d);
#pragma unroll
    for (int e0 = 0; e0 < 4; e0 += GROUP / 32) {
      if (k0 + 32 * e0 >= a.K) break;
      const int gi = (k0 + 32 * e0) / GROUP;
      const float s = E::up(sr[gi]);
      const float z = zr ? (float)zr[gi] : 8.0f;
      const uint32_t minus = E::pack(1024.0f + z, 1024.0f + z);
      v4f c[TM], cx[TM];
#pragma unroll
      for (int t = 0; t < TM; ++t) c[t] = cx[t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int e = e0; e < e0 + GROUP / 32; ++e) {
        const typename E::vec8 wf = codes8<E>(d[e], minus);
#pragma unroll
        for (int t = 0; t < TM; ++t) {
          const uint4 xv = live[t] ? *reinterpret_cast<const uint4*>(xr[t] + k0 + 32 * e) : make_uint4(0, 0, 0, 0);
          const typename E::vec8 xf = paired<E>(xv);
          c[t] = E::mfma(xf, wf, c[t]);
          if constexpr (!E::is_half) cx[t] = E::mfma(xf, ones.v, cx[t]);
        }
      }
#pragma unroll
      for (int t = 0; t < TM; ++t)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[t][r] += s * (E::is_half ? c[t][r] : c[t][r] - (128.0f + z) * cx[t][r]);
    }
  }
  if (wave > 0) {
#pragma unroll
    for (int t = 0; t < TM; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) sh[wave - 1][t][lane][r] = acc[t][r];
  }
  __syncthreads();
  if (wave > 0 || n0 + col >= a.N) return;
#pragma unroll
  for (int t = 0; t < TM; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int64_t m = m0 + 16 * t + 4 * kq + r;
      const float v = ((acc[t][r] + sh[0][t][lane][r]) + sh[1][t][lane][r]) + sh[2][t][lane][r];
      if (m < a.M) a.y[m * a.ldy + n0 + col] = (uint16_t)E::pack(v, 0.0f);
    }
}

template <class E, int TM>
hipError_t launch(const Args& a, int group, hipStream_t s) {
  const dim3 grid((unsigned)((a.N + 15) / 16), (unsigned)((a.M + 16 * TM - 1) / (16 * TM)));
  if (group == 32) hipLaunchKernelGGL((int4_mfma<E, TM, 32>), grid, dim3(256), 0, s, a);
  else if (group == 64) hipLaunchKernelGGL((int4_mfma<E, TM, 64>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((int4_mfma<E, TM, 128>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}
template <class E>
hipError_t launch_tokens(const Args& a, int group, hipStream_t s) {
  if (a.M <= 16) return launch<E, 1>(a, group, s);
  if (a.M <= 32) return launch<E, 2>(a, group, s);
  return launch<E, 4>(a, group, s);
}

}  // namespace

hipError_t launch_gemm_int4g(bsq_dtype dt, const Int4Args& p, hipStream_t s) {
  const Args a{static_cast<const uint16_t*>(p.x), p.ldx, p.w, static_cast<const uint16_t*>(p.ws), p.wz,
               static_cast<uint16_t*>(p.y), p.ldy, p.M, p.N, p.K};
  return dt == BSQ_FP16 ? launch_tokens<Fp16>(a, p.group, s) : launch_tokens<Bf16>(a, p.group, s);
}

}  // namespace bsq
