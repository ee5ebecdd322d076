// The epilogue of a linear: y = residual + gate * act(v + bias) on the scaled fp32 sums v.
//
// Activations are v / (1 + 2^q) with an odd q(v) = v p(v^2):
//   silu       p = -log2(e)
//   gelu_tanh  1/2 (1 + tanh u) = 1 / (1 + e^(-2u)): p = -2 log2(e) sqrt(2 / pi) (1 + 0.044715 v^2)
//   gelu       Phi(v) = 1 / (1 + (1 - Phi) / Phi), and log2((1 - Phi(v)) / Phi(v)) is odd because Phi(-v) = 1 - Phi(v):
//              p is the polynomial of degree 7 in v^2 that is nearest to it over |v| <= 5, weighted so that its worst
//              error of Phi(-v) relative to itself is least: 1.7e-5 (2^-15.9). Beyond, v^2 counts as 25 in p, so that
//              q stays linear in v and Phi goes on falling: off by less than 4e-7 of v there.
// One exp2, one reciprocal and 6 (gelu: 12) other instructions a value.
#pragma once

#include "block_launch.hpp"
#include "gemm_common.hpp"

namespace bsq {
namespace gemm {

// kinds of activation a kernel is built for: none, two coefficients of the launch, gelu's eight
enum ActKind { kActNone = 0, kActTwo = 1, kActGelu = 2 };
inline int act_kind(int act) { return act == BSQ_ACT_NONE ? kActNone : act == BSQ_ACT_GELU ? kActGelu : kActTwo; }

// gelu's p, from the constant term on
constexpr float kGelu[8] = {-2.30213666f, -0.10494373f, 0.000136703951f, 0.000154161346f,
                            -1.14962486e-05f, 4.40545364e-07f, -9.00572683e-09f, 7.73110395e-11f};

template <int ACT>
__device__ __forceinline__ float activate(float v, const Epilogue& e) {
  if constexpr (ACT == kActNone) return v;
  const float t = v * v;
  float p;
  if constexpr (ACT == kActTwo) {
    p = fmaf(fminf(t, 3e38f), e.c1, e.c0);  // (c1 may be 0, and t infinite)
  } else {
    const float u = fminf(t, 25.0f);
    p = kGelu[7];
    p = fmaf(u, p, kGelu[6]);
    p = fmaf(u, p, kGelu[5]);
    p = fmaf(u, p, kGelu[4]);
    p = fmaf(u, p, kGelu[3]);
    p = fmaf(u, p, kGelu[2]);
    p = fmaf(u, p, kGelu[1]);
    p = fmaf(u, p, kGelu[0]);
  }
  // (the hardware's exp2 and reciprocal, 1 ulp each: 2^-23 of itself; 2^q overflows to infinity, whose reciprocal is 0)
  return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * p));
}

__device__ __forceinline__ float bf16_at(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
// four bf16 of a row vector from element n on; elements past N read as zero. wide: 8-byte loads are aligned
__device__ __forceinline__ float4 bf16x4_at(const uint16_t* p, int n, int N, bool wide) {
  if (wide && n + 4 <= N) {
    const uint2 v = *reinterpret_cast<const uint2*>(p + n);
    return make_float4(bf16_lo(v.x), bf16_hi(v.x), bf16_lo(v.y), bf16_hi(v.y));
  }
  return make_float4(n < N ? bf16_at(p + n) : 0.0f, n + 1 < N ? bf16_at(p + n + 1) : 0.0f,
                     n + 2 < N ? bf16_at(p + n + 2) : 0.0f, n + 3 < N ? bf16_at(p + n + 3) : 0.0f);
}

// Residual rows [BM][BN] of a tile into LDS rows TROW bytes apart, 16 bytes a lane and step; past M or N nothing is
// read (and what LDS holds there only feeds outputs that are not stored)
template <int BM, int BN, int TROW>
__device__ __forceinline__ void load_tile_rows(uint8_t* tile, const uint16_t* r, int64_t ldr, int M, int N, int m0,
                                               int n0, int tid) {
  constexpr int CPR = BN / 8, IT = BM * CPR / kThreads;
  if (BM * CPR % kThreads == 0 && IT % 8 == 0 && (ldr & 7) == 0 && m0 + BM <= M && n0 + BN <= N) {
#pragma unroll
    for (int i0 = 0; i0 < IT; i0 += 8) {
      uint4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int idx = tid + (i0 + u) * kThreads, ml = idx / CPR, c = idx - ml * CPR;
        v[u] = *reinterpret_cast<const uint4*>(r + (int64_t)(m0 + ml) * ldr + n0 + 8 * c);
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int idx = tid + (i0 + u) * kThreads, ml = idx / CPR, c = idx - ml * CPR;
        *reinterpret_cast<uint4*>(tile + ml * TROW + c * 16) = v[u];
      }
    }
    return;
  }
  const bool wide = (ldr & 7) == 0;
  for (int idx = tid; idx < BM * CPR; idx += kThreads) {
    const int ml = idx / CPR, c = idx - ml * CPR;
    const int m = m0 + ml, n = n0 + 8 * c;
    if (m >= M) break;  // rows only grow with idx
    if (n >= N) continue;
    const uint16_t* src = r + (int64_t)m * ldr + n;
    uint4 v;
    if (n + 8 <= N && wide) {
      v = *reinterpret_cast<const uint4*>(src);
    } else {
      uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (n + e < N) w[e >> 1] |= (uint32_t)src[e] << (16 * (e & 1));
      v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    *reinterpret_cast<uint4*>(tile + ml * TROW + c * 16) = v;
  }
}

// The epilogue of a tile whose accumulators hold (n-tile i, m-tile j) as in gemm_common.hpp; nothing else uses `tile`
// (LDS) any more, which every wave of the workgroup knows. scaled(i, j, g) gives the four values of register group g, scaled. The residual
// comes through LDS: read in rows of 16 bytes a lane, taken by each lane at its own outputs' place and replaced there
// by the output, which leaves in rows again (so y may be the residual).
template <int BM, int BN, int TROW, int TN, int TM, int ACT, class Scaled>
__device__ __forceinline__ void epilogue_tile(uint8_t* tile, const Epilogue& e, uint16_t* y, int64_t ldy, int M, int N,
                                              int m0, int n0, int mw, int nw, int tid, bool stream, Scaled scaled) {
  const int lane = tid & 63, lr = lane & 31, lh = lane >> 5;
  const RowGroups& rg = e.groups;
  int first = 0, last = 0;
  if (e.gate) {
    M = group_limit(rg);
    if (rg.groups > 1 && rg.starts) {
      first = group_of_wave(rg, m0, lane);
      last = group_of_wave(rg, m0 + BM - 1, lane);
    }
  }
  const bool wide_gate = ((reinterpret_cast<uintptr_t>(e.gate) | (uintptr_t)(2 * e.gate_stride)) & 7) == 0;
  const bool wide_bias = (reinterpret_cast<uintptr_t>(e.bias) & 7) == 0;
  if (e.residual) {
    load_tile_rows<BM, BN, TROW>(tile, e.residual, e.residual_stride, M, N, m0, n0, tid);
    __syncthreads();
  }
#pragma unroll
  for (int j = 0; j < TM; ++j) {
    const int ml = mw + 32 * j + lr, m = m0 + ml;
    const uint16_t* gate = nullptr;
    if (e.gate) gate = e.gate + (int64_t)group_of_lane(rg, m < M ? m : m0, first, last) * e.gate_stride;
#pragma unroll
    for (int i = 0; i < TN; ++i) {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int nl = nw + 32 * i + 8 * g + 4 * lh, n = n0 + nl;
        float4 v = scaled(i, j, g);
        if (e.bias) {
          const float4 b = bf16x4_at(e.bias, n, N, wide_bias);
          v = make_float4(v.x + b.x, v.y + b.y, v.z + b.z, v.w + b.w);
        }
        v = make_float4(activate<ACT>(v.x, e), activate<ACT>(v.y, e), activate<ACT>(v.z, e), activate<ACT>(v.w, e));
        if (e.gate) {
          const float4 k = bf16x4_at(gate, n, N, wide_gate);
          v = make_float4(v.x * k.x, v.y * k.y, v.z * k.z, v.w * k.w);
        }
        uint2* at = reinterpret_cast<uint2*>(tile + ml * TROW + nl * 2);
        if (e.residual) {
          const uint2 r = *at;
          v = make_float4(bf16_lo(r.x) + v.x, bf16_hi(r.x) + v.y, bf16_lo(r.y) + v.z, bf16_hi(r.y) + v.w);
        }
        *at = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
      }
    }
  }
  __syncthreads();
  store_tile_rows<BM, BN, TROW>(tile, y, ldy, M, N, m0, n0, tid, stream);
}

// what the tiled kernels do with their scaled sums
template <int ACT>
struct TileEpilogue {
  static constexpr int act = ACT;
  Epilogue e;
  template <int BM, int BN, int TROW, int TN, int TM, class Scaled>
  __device__ __forceinline__ void tile(uint8_t* smem, uint16_t* y, int64_t ldy, int M, int N, int m0, int n0, int mw,
                                       int nw, int tid, bool stream, Scaled scaled) const {
    epilogue_tile<BM, BN, TROW, TN, TM, ACT>(smem, e, y, ldy, M, N, m0, n0, mw, nw, tid, stream, scaled);
  }
};

// what the few-token kernels do with theirs, value by value
template <int ACT>
struct ValueEpilogue {
  static constexpr int act = ACT;
  Epilogue e;
  __device__ __forceinline__ int rows(int M) const { return e.gate ? group_limit(e.groups) : M; }
  // the outputs of row m in columns n and (`two`) n + 1, n < N
  __device__ __forceinline__ void pair(float& a, float& b, int m, int n, bool two) const {
    const int o = two ? 1 : 0;
    if (e.bias) {
      a += bf16_at(e.bias + n);
      b += bf16_at(e.bias + n + o);
    }
    a = activate<ACT>(a, e);
    b = activate<ACT>(b, e);
    if (e.gate) {
      const uint16_t* gate = e.gate + (int64_t)group_of_lane(e.groups, m, 0, e.groups.groups - 1) * e.gate_stride + n;
      a *= bf16_at(gate);
      b *= bf16_at(gate + o);
    }
    if (e.residual) {
      const uint16_t* r = e.residual + (int64_t)m * e.residual_stride + n;
      a = bf16_at(r) + a;
      b = bf16_at(r + o) + b;
    }
  }
};

// f(the epilogue built for its kind of activation)
template <template <int> class E, class F>
hipError_t with_kind(const Epilogue& e, F f) {
  switch (act_kind(e.act)) {
    case kActNone: return f(E<kActNone>{e});
    case kActTwo: return f(E<kActTwo>{e});
    default: return f(E<kActGelu>{e});
  }
}
}  // namespace gemm
}  // namespace bsq
