// The output tile of the nvfp4 W4A4 GEMM, shared by its launches (gemm_w4a4.hip) and by those with an epilogue
// (gemm_w4a4_epilogue.hip). The K loop's design is described in gemm_w4a4.hip.
#pragma once

#include <type_traits>

#include "gemm_common.hpp"
#include "bsq_launch.hpp"

namespace bsq {
namespace w4a4 {

using namespace gemm;

constexpr int kStageK = 256;  // K values per stage

// packed operand bytes of one K group for one lane: 32 E2M1 values (4 dwords)
struct Raw {
  uint4 q;
};

// packed bytes of K group q (0..3) of a stage for this lane: chunk 4h + q of the row
template <int TN, int TM>
__device__ __forceinline__ void read_raw(const uint8_t* st, int a_off, int b_off, int rowa, int rowb, int lh, int q,
                                         Raw (&ra)[TN], Raw (&rb)[TM]) {
#pragma unroll
  for (int i = 0; i < TN; ++i)
    ra[i].q = *reinterpret_cast<const uint4*>(st + a_off + swz_off<128>(rowa + i * 32, 4 * lh + q));
#pragma unroll
  for (int j = 0; j < TM; ++j)
    rb[j].q = *reinterpret_cast<const uint4*>(st + b_off + swz_off<128>(rowb + j * 32, 4 * lh + q));
}

// this lane's 8 block scales of a stage (blocks 8h .. 8h + 7 of the row)
template <int TN, int TM>
__device__ __forceinline__ void read_scales(const uint8_t* st, int sa_off, int sb_off, int rowa, int rowb, int lh,
                                            uint2 (&sa)[TN], uint2 (&sb)[TM]) {
#pragma unroll
  for (int i = 0; i < TN; ++i) sa[i] = *reinterpret_cast<const uint2*>(st + sa_off + (rowa + i * 32) * 16 + 8 * lh);
#pragma unroll
  for (int j = 0; j < TM; ++j) sb[j] = *reinterpret_cast<const uint2*>(st + sb_off + (rowb + j * 32) * 16 + 8 * lh);
}

// block scale bytes 2 hi and 2 hi + 1 of `s` as f16 (E4M3 -> f16 is exact)
__device__ __forceinline__ v2h scale_pairs(uint32_t s, int hi) {
  return hi ? __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(s, 1.0f, true)
            : __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(s, 1.0f, false);
}

__device__ __forceinline__ uint32_t h2u(v2h v) {
  union { v2h h; uint32_t u; } c;
  c.h = v;
  return c.u;
}

// decode the 8 values of K step t (dword t of the packed chunk) times its block scale
__device__ __forceinline__ v8h decode8(uint32_t w, v2h s) {
  union { uint4 u; v8h h; } r;
  r.u = make_uint4(h2u(dec_e2m1x2_f16<0>(w) * s), h2u(dec_e2m1x2_f16<1>(w) * s),
                   h2u(dec_e2m1x2_f16<2>(w) * s), h2u(dec_e2m1x2_f16<3>(w) * s));
  return r.h;
}

template <int T>
__device__ __forceinline__ uint32_t dword_of(const uint4& q) {
  return T == 0 ? q.x : T == 1 ? q.y : T == 2 ? q.z : q.w;
}

// The block scales of a stage, for any K (scale_row_load of gemm_tiles.hpp): 16 bytes of each W and Xq row into registers, at
// any even address, and from there to LDS. Scales past K and rows past the matrix are 0 (the codes there are read as 0; a
// scale's NaN must not meet them).
template <int BM, int BN>
struct ScaleRows {
  static constexpr int N = (BM + BN + kThreads - 1) / kThreads;
  struct __attribute__((packed, aligned(2))) Any {
    uint32_t w[4];
  };
  uint4 v[N];
  __device__ __forceinline__ void load(const DecArgs& a, int m0, int n0, int kt, int tid) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const ScaleRowLoad l = scale_row_load<BM, BN>(tid + j * kThreads, kt, m0, n0, (int)a.M, (int)a.N, (int)a.K);
      v[j] = make_uint4(0, 0, 0, 0);
      if (l.left == 0) continue;
      const uint8_t* p = (l.w ? a.ws : a.xs) + l.from;
      if (l.left >= 16) {
        const Any x = *reinterpret_cast<const Any*>(p);
        v[j] = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
      } else {  // (an even number of them: K % 32 == 0)
        uint32_t x[4] = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (2 * e < l.left) x[e >> 1] |= (uint32_t) reinterpret_cast<const uint16_t*>(p)[e] << (16 * (e & 1));
        v[j] = make_uint4(x[0], x[1], x[2], x[3]);
      }
    }
  }
  __device__ __forceinline__ void store(uint8_t* stage, int tid) const {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int at = scale_row_load<BM, BN>(tid + j * kThreads, 0, 0, 0, 0, 0, 0).lds;
      if (at >= 0) *reinterpret_cast<uint4*>(stage + at) = v[j];
    }
  }
};

// Finish: what becomes of the scaled sums (TileEpilogue of epilogue.hpp); NoFinish: y is their bf16. ANYK: K % 256 != 0.
// One output tile: workgroup `bid` of the grid of BM x BN tiles over M x N.
template <int BM, int BN, bool LORA, class Finish = NoFinish, bool ANYK = false>
__device__ __forceinline__ void w4a4_tile(const DecArgs& a, int bid, const Finish& finish = Finish{}) {
  constexpr bool kFinish = !std::is_same<Finish, NoFinish>::value;
  using C = W4Cfg<BM, BN>;
  constexpr int TN = C::TN, TM = C::TM;
  __shared__ __attribute__((aligned(16))) uint8_t smem[C::LDS];
  __shared__ __attribute__((aligned(16))) float s_g[2][64];  // gx, gw (lane 0 of two dword DMAs)

  const int M = (int)a.M, N = (int)a.N, K = (int)a.K;
  int m0, n0;
  tile_of_id(bid, M, N, BM, BN, m0, n0);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave & 1, wn = wave >> 1;

  const int rows_x = M - m0 < BM ? M - m0 : BM, rows_w = N - n0 < BN ? N - n0 : BN;
  const int kp = K >> 1, ks = K >> 4;  // packed bytes and scale bytes per row
  const v4i rxq = buffer_rsrc(a.xq + (int64_t)m0 * kp, (uint32_t)(rows_x * kp));
  const v4i rwq = buffer_rsrc(a.w + (int64_t)n0 * kp, (uint32_t)(rows_w * kp));
  const v4i rxs = buffer_rsrc(a.xs + (int64_t)m0 * ks, (uint32_t)(rows_x * ks));
  const v4i rws = buffer_rsrc(a.ws + (int64_t)n0 * ks, (uint32_t)(rows_w * ks));
  const uint32_t lds0 = lds_offset(smem);
  // the two global scales, by dword LDS DMA ahead of the first stage (older than every stage
  // load, so the prologue's wait covers them): the last stage scales the accumulators in the loop
  if (wave == 0) {
    dma4(buffer_rsrc(a.gx, 4u), lds_offset(s_g[0]), lane == 0 ? 0 : kOutOfRange, 0);
    dma4(buffer_rsrc(a.gw, 4u), lds_offset(s_g[1]), lane == 0 ? 0 : kOutOfRange, 0);
  }

  // fetch stage kt into buffer kt % 2 (stages past K read as zeros)
  ScaleRows<BM, BN> scale_rows;  // (ANYK)
  auto issue_stage = [&](int kt) {
    const int kb = kt * kStageK;
    const uint32_t base = lds0 + (uint32_t)((kt & 1) * C::STAGE);
    dma_region<typename C::RA>(rwq, base + C::A_OFF, wave, lane, kp, kb >> 1, kb, K);
    dma_region<typename C::RB>(rxq, base + C::B_OFF, wave, lane, kp, kb >> 1, kb, K);
    if constexpr (ANYK) {
      scale_rows.load(a, m0, n0, kt, tid);
    } else {
      dma_region<typename C::SA>(rws, base + C::SA_OFF, wave, lane, ks, kb >> 4, kb, K);
      dma_region<typename C::SB>(rxs, base + C::SB_OFF, wave, lane, ks, kb >> 4, kb, K);
    }
  };

  v16f acc[TN][TM];
#pragma unroll
  for (int i = 0; i < TN; ++i)
#pragma unroll
    for (int j = 0; j < TM; ++j) acc[i][j] = v16f{};

  const int lr = lane & 31, lh = lane >> 5;
  const int rowa = wn * C::WN + lr, rowb = wm * C::WM + lr;  // region-local rows
  const int nk = ANYK ? (K + kStageK - 1) / kStageK : K / kStageK;

  Raw r0a[TN], r0b[TM], r1a[TN], r1b[TM];  // packed operands of the current / next K group
  uint2 s0a[TN], s0b[TM], s1a[TN], s1b[TM];  // block scales of the current / next stage
  v8h d0a[TN], d0b[TM], d1a[TN], d1b[TM];  // decoded operands of two consecutive K steps
  v2h spa[TN][2], spb[TM][2];              // block-scale pairs of the K group being decoded

  // scale pairs of K group q from the stage's scale bytes (bytes 2q, 2q + 1 of the lane's 8)
  // (one conversion gives both scales of the group; the multiplies broadcast one half of it)
  auto scales_of = [&](const uint2 (&sa)[TN], const uint2 (&sb)[TM], int q) {
#pragma unroll
    for (int i = 0; i < TN; ++i) {
      const v2h p = scale_pairs(q < 2 ? sa[i].x : sa[i].y, q & 1);
      spa[i][0] = v2h{p.x, p.x};
      spa[i][1] = v2h{p.y, p.y};
    }
#pragma unroll
    for (int j = 0; j < TM; ++j) {
      const v2h p = scale_pairs(q < 2 ? sb[j].x : sb[j].y, q & 1);
      spb[j][0] = v2h{p.x, p.x};
      spb[j][1] = v2h{p.y, p.y};
    }
  };
  auto decode_step = [&](auto tc, const Raw (&ra)[TN], const Raw (&rb)[TM], v8h (&da)[TN], v8h (&db)[TM]) {
    constexpr int T = decltype(tc)::value;
#pragma unroll
    for (int i = 0; i < TN; ++i) da[i] = decode8(dword_of<T>(ra[i].q), spa[i][T >> 1]);
#pragma unroll
    for (int j = 0; j < TM; ++j) db[j] = decode8(dword_of<T>(rb[j].q), spb[j][T >> 1]);
  };
  auto mfmas = [&](const v8h (&da)[TN], const v8h (&db)[TM]) {
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(da[i], db[j], acc[i][j], 0, 0, 0);
  };
  // one K step's MFMAs with the next step's decode (VALU) and LDS reads issued between them
  auto pipeline = [&](auto vc, auto dc) {
    constexpr int NV = decltype(vc)::value, ND = decltype(dc)::value;
#pragma unroll
    for (int i = 0; i < TN * TM; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x002, NV, 0);
      if (ND) __builtin_amdgcn_sched_group_barrier(0x100, ND, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  using I2 = std::integral_constant<int, 2>;
  using I3 = std::integral_constant<int, 3>;
  using NV = std::integral_constant<int, 8 * (TN + TM) / (TN * TM) + 1>;  // decode VALU per MFMA
  using NV2 = std::integral_constant<int, 8 * (TN + TM) / (TN * TM) + 3>;

  // the epilogue's scaling by gx gw and bf16 conversion of accumulator tile t into the LDS copy
  // of the output tile [BM][BN]
  auto tile_out = [&](int t, float alpha) {
    const int i = t / TM, j = t % TM;
    const int ml = wm * C::WM + j * 32 + lr;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int nl = wn * C::WN + i * 32 + 8 * g + 4 * lh;
      const v16f& A = acc[i][j];
      *reinterpret_cast<uint2*>(smem + ml * C::TROW + nl * 2) =
          make_uint2(pack_bf16x2(A[4 * g + 0] * alpha, A[4 * g + 1] * alpha),
                     pack_bf16x2(A[4 * g + 2] * alpha, A[4 * g + 3] * alpha));
    }
  };

  // K group q of a stage: operands in ca/cb (K step 0 decoded in d0, scale pairs of the group
  // in spa/spb); the next group's packed bytes are read into na/nb from `nst` (group nq, whose
  // scales are in nsa/nsb) and its K step 0 decoded into d0. The last group of the last stage
  // (LG) reads nothing ahead; once every wave has passed the last stage's barrier no stage
  // buffer is read any more, so each accumulator tile is scaled and written to the output copy
  // while the next tile's last MFMA runs.
  auto group = [&](const Raw (&ca)[TN], const Raw (&cb)[TM], Raw (&na)[TN], Raw (&nb)[TM], const uint8_t* nst,
                   int nq, const uint2 (&nsa)[TN], const uint2 (&nsb)[TM], auto lg) {
    constexpr bool LG = decltype(lg)::value;
    if constexpr (!LG) read_raw<TN, TM>(nst, C::A_OFF, C::B_OFF, rowa, rowb, lh, nq, na, nb);
    decode_step(I1{}, ca, cb, d1a, d1b);
    mfmas(d0a, d0b);
    pipeline(NV{}, std::integral_constant<int, LG ? 0 : 1>{});
    decode_step(I2{}, ca, cb, d0a, d0b);
    mfmas(d1a, d1b);
    pipeline(NV{}, I0{});
    decode_step(I3{}, ca, cb, d1a, d1b);
    if constexpr (!LG) scales_of(nsa, nsb, nq);
    mfmas(d0a, d0b);
    pipeline(NV2{}, I0{});
    if constexpr (LG) {
      const float alpha = s_g[0][0] * s_g[1][0];
#pragma unroll
      for (int k = 0; k < TN * TM; ++k) {
        const int i = k / TM, j = k % TM;
        acc[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_f16(d1a[i], d1b[j], acc[i][j], 0, 0, 0);
        if (k > 0) tile_out(k - 1, alpha);
      }
      tile_out(TN * TM - 1, alpha);
    } else {
      decode_step(I0{}, na, nb, d0a, d0b);
      mfmas(d1a, d1b);
      pipeline(NV{}, I0{});
    }
  };

  if constexpr (LORA) {
    // low-rank adapter: the accumulators start at T' B^T with T' = T / (gx gw) (the down
    // projection divides), so the epilogue's scaling by gx gw leaves y = bf16(base + T B^T).
    // Its first 64 rank values are loaded alongside the first stage; larger ranks follow.
    const rsrc_t rt = make_rsrc(a.lt, (uint32_t)M * (uint32_t)a.rank * 2u);
    const rsrc_t rb = make_rsrc(a.lb, (uint32_t)N * (uint32_t)a.rank * 2u);
    const int nw0 = n0 + wn * C::WN, mw0 = m0 + wm * C::WM;
    LoraRegs<TN, TM, 4> lo;
    lora_load(lo, rt, rb, 0, a.rank, nw0, mw0, lane);
    issue_stage(0);
    // both sets of loads are in flight before anything waits (the scheduler would otherwise
    // hoist the adapter MFMAs, and their wait, above the stage's DMA)
    __builtin_amdgcn_sched_barrier(0);
    wait_vmcnt<0>();
    lora_mfma(acc, lo, 0, a.rank);
    for (int k0 = 64; k0 < a.rank; k0 += 64) {
      lora_load(lo, rt, rb, k0, a.rank, nw0, mw0, lane);
      lora_mfma(acc, lo, k0, a.rank);
    }
  } else {
    issue_stage(0);
    wait_vmcnt<0>();
  }
  if constexpr (ANYK) scale_rows.store(smem, tid);
  __syncthreads();
  issue_stage(1);
  read_raw<TN, TM>(smem, C::A_OFF, C::B_OFF, rowa, rowb, lh, 0, r0a, r0b);
  read_scales<TN, TM>(smem, C::SA_OFF, C::SB_OFF, rowa, rowb, lh, s0a, s0b);
  scales_of(s0a, s0b, 0);
  decode_step(I0{}, r0a, r0b, d0a, d0b);

  // Stage s sits in buffer s % 2 and stage s + 1 is in flight into the other one. Before the
  // last K group reads ahead into stage s + 1, every wave waits for its share of stage s + 1,
  // the barrier publishes it (and ends all reads of stage s), and stage s + 2 (if there is one)
  // is fetched into buffer s % 2. Past the second-to-last stage the read-ahead sees a stale
  // buffer and goes unused; the last stage reads nothing ahead.
  using F = std::false_type;
  auto stage = [&](int s, const uint2 (&csa)[TN], const uint2 (&csb)[TM], uint2 (&nsa)[TN], uint2 (&nsb)[TM],
                   auto last) {
    constexpr bool LAST = decltype(last)::value;
    const uint8_t* cur = smem + (s & 1) * C::STAGE;
    const uint8_t* nxt = smem + ((s + 1) & 1) * C::STAGE;
    group(r0a, r0b, r1a, r1b, cur, 1, csa, csb, F{});
    group(r1a, r1b, r0a, r0b, cur, 2, csa, csb, F{});
    group(r0a, r0b, r1a, r1b, cur, 3, csa, csb, F{});
    wait_vmcnt<0>();
    if constexpr (ANYK) scale_rows.store(smem + ((s + 1) & 1) * C::STAGE, tid);
    __syncthreads();
    if (s + 2 < nk) issue_stage(s + 2);
    if constexpr (!LAST) read_scales<TN, TM>(nxt, C::SA_OFF, C::SB_OFF, rowa, rowb, lh, nsa, nsb);
    group(r1a, r1b, r0a, r0b, nxt, 0, nsa, nsb, last);
  };
  int s = 0;
  for (; s + 2 < nk; s += 2) {
    stage(s, s0a, s0b, s1a, s1b, F{});
    stage(s + 1, s1a, s1b, s0a, s0b, F{});
  }
  if (s + 2 == nk) {
    stage(s, s0a, s0b, s1a, s1b, F{});
#pragma unroll
    for (int i = 0; i < TN; ++i) s0a[i] = s1a[i];
#pragma unroll
    for (int j = 0; j < TM; ++j) s0b[j] = s1b[j];
    ++s;
  }
  stage(s, s0a, s0b, s1a, s1b, std::integral_constant<bool, !kFinish>{});

  if constexpr (kFinish) {
    static_assert(!LORA, "an adapter's linear has no epilogue");
    __syncthreads();  // no stage buffer is read any more
    const float alpha = s_g[0][0] * s_g[1][0];
    auto scaled = [&](int i, int j, int g, const float4* bias) {
      const v16f& A = acc[i][j];
      if (!bias) return make_float4(A[4 * g] * alpha, A[4 * g + 1] * alpha, A[4 * g + 2] * alpha, A[4 * g + 3] * alpha);
      const float4 b = *bias;
      return make_float4(fmaf(A[4 * g], alpha, b.x), fmaf(A[4 * g + 1], alpha, b.y), fmaf(A[4 * g + 2], alpha, b.z),
                         fmaf(A[4 * g + 3], alpha, b.w));
    };
    finish.template tile<BM, BN, C::TROW, TN, TM>(smem, a.y, a.ldy, M, N, m0, n0, wm * C::WM, wn * C::WN, tid,
                                                  a.stream_y != 0, scaled);
    return;
  }
  // ---- epilogue: y = bf16(acc * gx * gw), written to the LDS copy of the tile [BM][BN] by the
  // last stage above, then stored
  __syncthreads();
  if (a.y) store_tile_rows<BM, BN, C::TROW>(smem, a.y, a.ldy, M, N, m0, n0, tid, a.stream_y != 0);
  // optionally the nvfp4 encoding of Y for the next linear ("BFL (fp8r / nvfp4)": every
  // quantized linear quantizes its input at run time); its 16-blocks run along this N, inside
  // the tile
  if (a.yq) quant_tile_rows<BM, BN, C::TROW>(smem, a.yq, a.ys, 1.0f / a.gy[0], M, N, m0, n0, tid);
  // or the row maxima of an fp8r encoding, whose per-row scale spans every tile of the row
  if (a.ypmax) rowmax_tile<BM, BN, C::TROW>(smem, a.ypmax, M, N, m0, n0, tid);
}

}  // namespace w4a4
}  // namespace bsq
