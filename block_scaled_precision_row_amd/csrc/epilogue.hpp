// The epilogue of a linear: y = residual + gate * act(v + bias) on the scaled fp32 sums v.
//
// Activations are v / (1 + 2^q) with an odd q(v) = v p(v^2):
//   silu       p = -log2(e)
//   gelu_tanh  1/2 (1 + tanh u) = 1 / (1 + e^(-2u)): p = -2 log2(e) sqrt(2 / pi) (1 + 0.044715 v^2)
//   gelu       Phi(v) = 1 / (1 + (1 - Phi) / Phi), and log2((1 - Phi(v)) / Phi(v)) is odd because Phi(-v) = 1 - Phi(v):
//              p is the polynomial of degree 7 in v^2 that is nearest to it over |v| <= 5, weighted so that its worst
//              error of Phi(-v) relative to itself is least: 1.7e-5 (2^-15.9). Beyond, v^2 counts as 25 in p, so that
//              q stays linear in v and Phi goes on falling: off by less than 4e-7 of v there.
// One exp2, one reciprocal and 3 (silu), 5 (gelu_tanh) or 12 (gelu) other instructions a value: 4096 x 10240 x 2560
// fp8r takes 128 us with gelu_tanh and 127 without an epilogue.
#pragma once

#include "block_launch.hpp"
#include "gemm_common.hpp"

namespace bsq {
namespace gemm {

// gelu's p, from the constant term on
constexpr float kGelu[8] = {-2.30213666f, -0.10494373f, 0.000136703951f, 0.000154161346f,
                            -1.14962486e-05f, 4.40545364e-07f, -9.00572683e-09f, 7.73110395e-11f};

template <int ACT>  // a bsq_act
__device__ __forceinline__ float activate(float v) {
  if constexpr (ACT == BSQ_ACT_NONE) return v;
  constexpr double kLog2e = 1.4426950408889634, kTanh = -2.0 * kLog2e * 0.7978845608028654;
  float p;
  if constexpr (ACT == BSQ_ACT_SILU) {
    p = (float)-kLog2e;
  } else if constexpr (ACT == BSQ_ACT_GELU_TANH) {
    p = fmaf(v * v, (float)(kTanh * 0.044715), (float)kTanh);
  } else {
    const float u = fminf(v * v, 25.0f);
    p = kGelu[7];
#pragma unroll
    for (int i = 6; i >= 0; --i) p = fmaf(u, p, kGelu[i]);
  }
  // (the hardware's exp2 and reciprocal, 1 ulp each: 2^-23 of itself; 2^q overflows to infinity, whose reciprocal is 0)
  return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * p));
}

__device__ __forceinline__ float bf16_at(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
// four bf16 of a row vector from element n on; elements past N read as zero
__device__ __forceinline__ float4 bf16x4_at(const uint16_t* p, int n, int N) {
  return make_float4(n < N ? bf16_at(p + n) : 0.0f, n + 1 < N ? bf16_at(p + n + 1) : 0.0f,
                     n + 2 < N ? bf16_at(p + n + 2) : 0.0f, n + 3 < N ? bf16_at(p + n + 3) : 0.0f);
}

// eight bf16 at any even address (the memory takes 16-byte accesses there)
struct __attribute__((packed, aligned(2))) Eight {
  uint32_t w[4];
};
// chunk of eight of a row from column n on, n < N: columns past N read as zero, and are not written
__device__ __forceinline__ uint4 load_chunk(const uint16_t* p, int n, int N) {
  if (n + 8 <= N) {
    const Eight v = *reinterpret_cast<const Eight*>(p);
    return make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
  }
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (n + e < N) w[e >> 1] |= (uint32_t)p[e] << (16 * (e & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void store_chunk(uint16_t* p, uint4 v, int n, int N) {
  if (n + 8 <= N) {
    *reinterpret_cast<Eight*>(p) = Eight{{v.x, v.y, v.z, v.w}};
    return;
  }
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (n + e < N) p[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
}

// The residual's rows of a tile into LDS rows TROW bytes apart, 16 bytes a lane and step, up to 16 of them under way;
// past M or N nothing is read (and what LDS holds there only feeds outputs that are not stored)
template <int BM, int BN, int TROW>
__device__ __forceinline__ void load_tile_rows(uint8_t* tile, const uint16_t* r, int64_t ldr, int M, int N, int m0,
                                               int n0, int tid) {
  constexpr int CPR = BN / 8, IT = BM * CPR / kThreads;
  constexpr int U = IT % 16 == 0 ? 16 : IT % 12 == 0 ? 12 : IT % 8 == 0 ? 8 : IT;
  static_assert(BM * CPR % kThreads == 0 && IT % U == 0, "whole steps");
#pragma unroll
  for (int i0 = 0; i0 < IT; i0 += U) {
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int idx = tid + (i0 + u) * kThreads, ml = idx / CPR, c = idx - ml * CPR, n = n0 + 8 * c;
      v[u] = make_uint4(0, 0, 0, 0);
      if (m0 + ml < M && n < N) v[u] = load_chunk(r + (int64_t)(m0 + ml) * ldr + n, n, N);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int idx = tid + (i0 + u) * kThreads, ml = idx / CPR, c = idx - ml * CPR;
      *reinterpret_cast<uint4*>(tile + ml * TROW + c * 16) = v[u];
    }
  }
}
// and a tile's rows out of LDS
template <int BM, int BN, int TROW>
__device__ __forceinline__ void put_tile_rows(const uint8_t* tile, uint16_t* y, int64_t ldy, int M, int N, int m0, int n0,
                                              int tid, bool stream) {
  constexpr int CPR = BN / 8;
  if ((ldy & 7) == 0 && m0 + BM <= M && n0 + BN <= N) {
    store_tile_rows<BM, BN, TROW>(tile, y, ldy, M, N, m0, n0, tid, stream);
    return;
  }
  for (int idx = tid; idx < BM * CPR; idx += kThreads) {
    const int ml = idx / CPR, c = idx - ml * CPR, n = n0 + 8 * c;
    if (m0 + ml >= M) break;  // rows only grow with idx
    const uint4 v = *reinterpret_cast<const uint4*>(tile + ml * TROW + c * 16);
    if (n < N) store_chunk(y + (int64_t)(m0 + ml) * ldy + n, v, n, N);
  }
}

// The epilogue of a tile whose accumulators hold (n-tile i, m-tile j) as in gemm_common.hpp; nothing else uses `tile`
// (LDS) any more, which every wave of the workgroup knows. scaled(i, j, g, bias) gives the four values of register group
// g, scaled, plus the bias (null: without). Bias, the gates of up to four groups and the residual come through LDS, all
// under way together; each lane takes the residual at its own outputs' place and puts the output there, which
// leaves in rows again (so y may be the residual).
constexpr int kGateRows = 4;  // groups of a tile whose gates LDS holds; with more of them lanes read their own from memory
template <int BM, int BN, int TROW, int TN, int TM, int ACT, class Scaled>
__device__ __forceinline__ void epilogue_tile(uint8_t* tile, const Epilogue& e, uint16_t* y, int64_t ldy, int M, int N,
                                              int m0, int n0, int mw, int nw, int tid, bool stream, Scaled scaled) {
  __shared__ __attribute__((aligned(16))) float vectors[1 + kGateRows][BN];
  const int lane = tid & 63, lr = lane & 31, lh = lane >> 5;
  const RowGroups& rg = e.groups;
  int first = 0, last = 0;
  if (e.gate) {
    M = group_limit(rg);
    if (rg.groups > 1) {
      first = group_of_wave(rg, m0, lane);
      last = group_of_wave(rg, m0 + BM < M ? m0 + BM - 1 : (M > m0 ? M - 1 : m0), lane);
    }
  }
  const bool held = last - first < kGateRows;
  if (tid < BN) {
    const int n = n0 + tid;
    if (e.bias) vectors[0][tid] = n < N ? bf16_at(e.bias + n) : 0.0f;
    if (e.gate && held) {
#pragma unroll
      for (int k = 0; k < kGateRows; ++k)
        if (first + k <= last) vectors[1 + k][tid] = n < N ? bf16_at(e.gate + (int64_t)(first + k) * e.gate_stride + n) : 0.0f;
    }
  }
  if (e.residual) load_tile_rows<BM, BN, TROW>(tile, e.residual, e.residual_stride, M, N, m0, n0, tid);
  __syncthreads();
#pragma unroll
  for (int j = 0; j < TM; ++j) {
    const int ml = mw + 32 * j + lr, m = m0 + ml;
    const int mine = e.gate ? group_of_lane(rg, m < M ? m : m0, first, last) : 0;
    int row = mine - first;  // of the gates that LDS holds (starts out of order could lead outside them)
    row = row < 0 ? 0 : (row < kGateRows ? row : kGateRows - 1);
    const float* gates = vectors[1 + row];
#pragma unroll
    for (int i = 0; i < TN; ++i) {
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int nl = nw + 32 * i + 8 * g + 4 * lh;
        float4 v = scaled(i, j, g, e.bias ? reinterpret_cast<const float4*>(&vectors[0][nl]) : nullptr);
        v = make_float4(activate<ACT>(v.x), activate<ACT>(v.y), activate<ACT>(v.z), activate<ACT>(v.w));
        if (e.gate) {
          const float4 k = held ? *reinterpret_cast<const float4*>(gates + nl)
                                : bf16x4_at(e.gate + (int64_t)mine * e.gate_stride, n0 + nl, N);
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
  put_tile_rows<BM, BN, TROW>(tile, y, ldy, M, N, m0, n0, tid, stream);
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
    a = activate<ACT>(a);
    b = activate<ACT>(b);
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

// f(the epilogue built for its activation)
template <template <int> class E, class F>
hipError_t with_kind(const Epilogue& e, F f) {
  switch (e.act) {
    case BSQ_ACT_NONE: return f(E<BSQ_ACT_NONE>{e});
    case BSQ_ACT_SILU: return f(E<BSQ_ACT_SILU>{e});
    case BSQ_ACT_GELU_TANH: return f(E<BSQ_ACT_GELU_TANH>{e});
    default: return f(E<BSQ_ACT_GELU>{e});
  }
}

}  // namespace gemm
}  // namespace bsq
