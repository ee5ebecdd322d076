// fp8r W8A8 GEMM on the gfx950 FP8 matrix cores.
//
// "BFL (fp8r / nvfp4)", "Kernels" table: the fp8r scheme multiplies E4M3
// activations (quantized per row at run time) by E4M3 weights and applies the
// two row-wise scale vectors to the fp32 result:
//   y[m][n] = bf16( (sum_k e4m3(xq[m][k]) * e4m3(w[n][k])) * sx[m] * sw[n] ).
// Both scale vectors are rank-1 over (m, n), so they are applied once in the
// epilogue; the K loop is a plain E4M3 x E4M3 -> fp32 contraction on
// v_mfma_f32_32x32x64_f8f6f4 (no per-block scaling inside the loop).
//
// Pipeline (layout conventions in gemm_common.hpp): each stage is 128 K
// values = 128 bytes (one full cache line) of every W row and every Xq row,
// fetched by LDS DMA into a ring of NS stage buffers; full-line rows halve
// the number of memory requests against 64-byte stages. A stage is two
// 64-deep MFMA K steps. Iteration s reads step 1 of stage s into registers
// while the MFMAs of step 0 run, waits until stage s + 1 has landed, and at
// the barrier that follows no wave reads stage s any more, so its buffer is
// refilled with stage s + NS at once; step 0 of stage s + 1 is then read
// while the MFMAs of step 1 run. NS - 1 stages are in flight behind the one
// being multiplied.
// K permutation: in step t of a stage, lane half h of an MFMA operand holds
// the 32 bytes [64 h + 32 t, 64 h + 32 t + 32) of its row -- the same for W
// and Xq, so every product pairs equal K indices.
// The epilogue scales the accumulators, converts them to bf16 into an LDS
// copy of the output tile, and writes the tile back in 16-byte row chunks.
#include <cmath>

#include "gemm_fp8_tile.hpp"

namespace bsq {

namespace {

using namespace gemm;
using namespace fp8;

template <int BM, int BN, int NS, bool LORA, int OQ = 0, bool HS = false, int LL = kLoraGlobal, int WPE = 1>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(WPE, WPE)))
void gemm_fp8_kernel(const uint8_t* __restrict__ xq, const float* __restrict__ sx,
                     const uint8_t* __restrict__ w, const float* __restrict__ sw,
                     uint16_t* __restrict__ y, int64_t ldy, int M, int N, int K, const uint16_t* lt,
                     const uint16_t* lb, int rank, int stream_y, YQuant q) {
  fp8_tile<BM, BN, NS, LORA, OQ, HS, LL>(xq, sx, w, sw, y, ldy, M, N, K, lt, lb, rank, stream_y, q, blockIdx.x);
}

// The tiles of several W8A8 GEMMs in one grid (hand-ordered loop, two stage buffers): the
// problem of each workgroup, then that problem's tile, exactly as its own launch would compute
// it (same tile shape, same bits).
struct Fp8Group {
  Fp8Problem p[kMaxGroup];
  int start[kMaxGroup + 1];
  int count;
};
template <int BM, int BN, int WPE>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(WPE, WPE)))
void gemm_fp8_grouped_kernel(Fp8Group g) {
  const int bid = blockIdx.x;
  const int p = group_problem(g.start, g.count, bid);
  const Fp8Problem& q = g.p[p];
  fp8_tile<BM, BN, 2, false, 0, true, kLoraGlobal>(q.xq, q.sx, q.w, q.sw, q.y, q.ldy, q.M, q.N, q.K, nullptr,
                                                   nullptr, 0, q.stream_y, YQuant{}, bid - g.start[p]);
}

template <int BM, int BN, int NS, bool HS, int WPE = 1>
hipError_t launch_oq(int oq, int tiles, const uint8_t* xq, const float* sx, const uint8_t* w, const float* sw,
                     uint16_t* y, int64_t ldy, int64_t M, int64_t N, int64_t K, int st, const YQuant& qv,
                     hipStream_t s) {
  if (oq == 1)
    hipLaunchKernelGGL((gemm_fp8_kernel<BM, BN, NS, false, 1, HS, kLoraGlobal, WPE>), dim3(tiles), dim3(kThreads), 0,
                       s, xq, sx, w, sw, y, ldy, (int)M, (int)N, (int)K, nullptr, nullptr, 0, st, qv);
  else if (oq == 2)
    hipLaunchKernelGGL((gemm_fp8_kernel<BM, BN, NS, false, 2, HS, kLoraGlobal, WPE>), dim3(tiles), dim3(kThreads), 0,
                       s, xq, sx, w, sw, y, ldy, (int)M, (int)N, (int)K, nullptr, nullptr, 0, st, qv);
  else
    hipLaunchKernelGGL((gemm_fp8_kernel<BM, BN, NS, false, 0, HS, kLoraGlobal, WPE>), dim3(tiles), dim3(kThreads), 0,
                       s, xq, sx, w, sw, y, ldy, (int)M, (int)N, (int)K, nullptr, nullptr, 0, st, qv);
  return hipGetLastError();
}

// 128 x 128 tiles with two stage buffers and the hand-ordered loop, two workgroups per compute
// unit (65 KB of LDS and at most 256 registers a lane each), so one workgroup's barrier waits,
// prologue and output write overlap the other's K loop: 512 tiles a round
hipError_t run_pair(const uint8_t* xq, const float* sx, const uint8_t* w, const float* sw, uint16_t* y, int64_t ldy,
                    int64_t M, int64_t N, int64_t K, hipStream_t s, const YQuant* q) {
  const int tiles = (int)(((M + 127) / 128) * ((N + 127) / 128));
  const int st = (int)stream_output((M + N) * K, M, N);
  const YQuant qv = q ? *q : YQuant{};
  const int oq = qv.yq ? 1 : qv.pmax ? 2 : 0;
  return launch_oq<128, 128, 2, true, 2>(oq, tiles, xq, sx, w, sw, y, ldy, M, N, K, st, qv, s);
}

template <int BM, int BN, int NS>
hipError_t run(const uint8_t* xq, const float* sx, const uint8_t* w, const float* sw, uint16_t* y,
               int64_t ldy, int64_t M, int64_t N, int64_t K, const uint16_t* lt, const uint16_t* lb, int rank,
               hipStream_t s, const YQuant* q) {
  const int tiles = (int)(((M + BM - 1) / BM) * ((N + BN - 1) / BN));
  constexpr bool kAdapter = !(BM == 256 && BN == 256);  // the 256 x 256 tile never carries one (launch_gemm_fp8)
  const int st = (int)stream_output((M + N) * K, M, N);
  const YQuant qv = q ? *q : YQuant{};
  if (kAdapter && lt) {
    constexpr bool kHand = hand_ordered<NS>();
    constexpr int kAhead = kAdapter ? kLoraAhead : kLoraGlobal, kLate = kAdapter && kHand ? kLoraLate : kLoraGlobal,
                  kLate2 = kAdapter && kHand ? kLoraLate2 : kLoraGlobal;
    const bool hs = kHand && K % kStageK == 0;
    const int ll = lora_lds_host(rank, hs);
    if (hs && ll == kLoraAhead)
      hipLaunchKernelGGL((gemm_fp8_kernel<BM, BN, NS, kAdapter, 0, kHand, kAhead>), dim3(tiles), dim3(kThreads), 0, s,
                         xq, sx, w, sw, y, ldy, (int)M, (int)N, (int)K, lt, lb, rank, st, qv);
    else if (hs && ll == kLoraLate)
      hipLaunchKernelGGL((gemm_fp8_kernel<BM, BN, NS, kAdapter, 0, kHand, kLate>), dim3(tiles), dim3(kThreads), 0, s,
                         xq, sx, w, sw, y, ldy, (int)M, (int)N, (int)K, lt, lb, rank, st, qv);
    else if (hs && ll == kLoraLate2)
      hipLaunchKernelGGL((gemm_fp8_kernel<BM, BN, NS, kAdapter, 0, kHand, kLate2>), dim3(tiles), dim3(kThreads), 0, s,
                         xq, sx, w, sw, y, ldy, (int)M, (int)N, (int)K, lt, lb, rank, st, qv);
    else if (hs)
      hipLaunchKernelGGL((gemm_fp8_kernel<BM, BN, NS, kAdapter, 0, kHand>), dim3(tiles), dim3(kThreads), 0, s, xq, sx,
                         w, sw, y, ldy, (int)M, (int)N, (int)K, lt, lb, rank, st, qv);
    else if (ll == kLoraAhead)
      hipLaunchKernelGGL((gemm_fp8_kernel<BM, BN, NS, kAdapter, 0, false, kAhead>), dim3(tiles), dim3(kThreads), 0, s,
                         xq, sx, w, sw, y, ldy, (int)M, (int)N, (int)K, lt, lb, rank, st, qv);
    else
      hipLaunchKernelGGL((gemm_fp8_kernel<BM, BN, NS, kAdapter>), dim3(tiles), dim3(kThreads), 0, s, xq, sx, w, sw,
                         y, ldy, (int)M, (int)N, (int)K, lt, lb, rank, st, qv);
    return hipGetLastError();
  }
  const int oq = qv.yq ? 1 : qv.pmax ? 2 : 0;
  if (hand_ordered<NS>() && K % kStageK == 0)
    return launch_oq<BM, BN, NS, hand_ordered<NS>()>(oq, tiles, xq, sx, w, sw, y, ldy, M, N, K, st, qv, s);
  return launch_oq<BM, BN, NS, false>(oq, tiles, xq, sx, w, sw, y, ldy, M, N, K, st, qv, s);
}

}  // namespace

// Grouped W8A8: every problem on the hand-ordered loop (K % 128 == 0). Below three rounds of
// 256 x 192 tiles the group runs on 128 x 128 tiles two to a compute unit, once those fill one
// round of pairs (512 tiles); beyond, on the 256 x 256 or 256 x 192 tile of least expected time
// over whole rounds (each tile's time in proportion to its K; round times as for one GEMM, at
// K = 3072) when it fills two rounds. Smaller groups run one launch per problem, whose own tile
// choice fills the compute units. A joint block's four linears (qkv, proj, up, down; cold
// weights) as one grid against four launches, fp8r / nvfp4 (us): 384 tokens 96 / 102 vs 114 /
// 150, 512 tokens 104 / 111 vs 129 / 171, 768 tokens 104 / 158 vs 145 / 218, 1024 tokens 144 /
// 200 vs 156 / 242 (all on 128 x 128 pairs), 2048 tokens 221 / 356 vs 290 / 443 (256 x 192),
// 4096 tokens 410 / 672 vs 440 / 716 (256 x 256). On 128 x 128 pairs 2048 and 4096 tokens took
// 262 / 406 and 505 / 803 us; on 256-row tiles 512 tokens (288 tiles) took 145 / 196 us.
namespace {
struct GroupTile {
  int bm, bn, per_round, round_us;
};
constexpr GroupTile kFp8GroupTiles[3] = {{256, 256, 256, 92}, {256, 192, 256, 72}, {128, 128, 512, 52}};
// the group's tile (index into kFp8GroupTiles), or -1 when no tile fills two rounds
int fp8_group_tile(const Fp8Problem* p, int count) {
  auto tiles_of = [&](const GroupTile& c, double* work) {
    int64_t tiles = 0;
    double w = 0;  // tiles times K / 3072
    for (int i = 0; i < count; ++i) {
      const int64_t n = ((int64_t)(p[i].M + c.bm - 1) / c.bm) * ((p[i].N + c.bn - 1) / c.bn);
      tiles += n;
      w += (double)n * (double)p[i].K / 3072.0;
    }
    if (work) *work = w;
    return tiles;
  };
  // under three rounds of 256 x 192 tiles, 128 x 128 tiles two to a compute unit once they fill a
  // round of pairs (measured below); otherwise the 256-row tile of fewer whole rounds
  if (tiles_of(kFp8GroupTiles[1], nullptr) < 3 * 256) {
    const int64_t t = tiles_of(kFp8GroupTiles[2], nullptr);
    return t >= 512 && t < ((int64_t)1 << 31) ? 2 : -1;
  }
  int best = -1;
  double best_cost = 0;
  for (int t = 0; t < 2; ++t) {
    const GroupTile& c = kFp8GroupTiles[t];
    double work = 0;
    const int64_t tiles = tiles_of(c, &work);
    if (tiles < 2 * (int64_t)c.per_round || tiles >= ((int64_t)1 << 31)) continue;  // 32-bit workgroup ids
    const double cost = std::ceil(work / c.per_round - 1e-9) * c.round_us;
    if (best < 0 || cost < best_cost) best = t, best_cost = cost;
  }
  return best;
}
template <int BM, int BN, int WPE>
hipError_t run_fp8_group(const Fp8Problem* p, int count, hipStream_t s) {
  Fp8Group g{};
  g.count = count;
  int64_t total = 0;
  for (int i = 0; i < count; ++i) {
    g.p[i] = p[i];
    g.p[i].stream_y = (int)stream_output((int64_t)(p[i].M + p[i].N) * p[i].K, p[i].M, p[i].N);
    g.start[i] = (int)total;
    total += ((int64_t)(p[i].M + BM - 1) / BM) * ((p[i].N + BN - 1) / BN);
  }
  for (int i = count; i <= kMaxGroup; ++i) g.start[i] = (int)total;
  hipLaunchKernelGGL((gemm_fp8_grouped_kernel<BM, BN, WPE>), dim3((unsigned)total), dim3(kThreads), 0, s, g);
  return hipGetLastError();
}
}  // namespace

bool gemm_fp8_grouped_supported(const Fp8Problem* p, int count) {
  if (count < 2 || count > kMaxGroup) return false;
  for (int i = 0; i < count; ++i)
    if (p[i].K % kStageK != 0) return false;
  return fp8_group_tile(p, count) >= 0;
}

hipError_t launch_gemm_fp8_grouped(const Fp8Problem* p, int count, hipStream_t s) {
  switch (fp8_group_tile(p, count)) {
    case 0: return run_fp8_group<256, 256, 1>(p, count, s);
    case 1: return run_fp8_group<256, 192, 1>(p, count, s);
    default: return run_fp8_group<128, 128, 2>(p, count, s);
  }
}

hipError_t launch_gemm_fp8(const uint8_t* xq, const float* sx, const uint8_t* w, const float* sw,
                           uint16_t* y, int64_t ldy, int64_t M, int64_t N, int64_t K, const uint16_t* lt,
                           const uint16_t* lb, int rank, hipStream_t s, const YQuant* q) {
  // A grid of few tiles leaves compute units idle, and each busy unit is bound by the latency
  // of its own loads (three stages in flight); more, smaller tiles keep more loads in flight
  // across the chip. So while its grid fits one round on the 256 units, the smallest tile is
  // taken: 64 x 64 (its 64 KB of LDS lets two workgroups share a unit), then 64 tokens x 128
  // weight rows. Measured at K = 3072: 512 x 3072 14.8 -> 10.0 us, 320 x 3072 14.2 -> 8.4 us,
  // 512 x 3072 x 12288 46.4 -> 33.8 us.
  //
  // Larger grids take the tile of least expected time over whole rounds, with per-tile times
  // measured at K = 3072 with every unit busy: 256 x 256 46 us, 256 x 192 36 us, 128 x 128
  // 15.5 us. The square tile moves 12 % fewer operand bytes per flop through the L2 -> LDS
  // path that bounds this kernel, so it wins when the rounds come out even (16384 x 3072:
  // 7-11 % faster); the rounds decide elsewhere -- 3072 x 4096 78 -> 45.5 us on 256 x 256,
  // 3072 x 12288 131 -> 107 us on 256 x 192, 1024 x 3072 22 -> 14.7 us on 128 x 128. With an
  // adapter the square tile is left out (its epilogue does not fit the square tile's
  // registers). Every tile shape gives the same bits (the same MFMA sequence per output).
  const int64_t t64 = ((M + 63) / 64) * ((N + 63) / 64), t64x128 = ((M + 63) / 64) * ((N + 127) / 128);
  if (t64 <= 256) return run<64, 64, 4>(xq, sx, w, sw, y, ldy, M, N, K, lt, lb, rank, s, q);
  if (t64x128 <= 256) return run<64, 128, 4>(xq, sx, w, sw, y, ldy, M, N, K, lt, lb, rank, s, q);
  const int64_t c256 = lt ? INT64_MAX : rounds_cost(M, N, 256, 256, 92);
  const int64_t c192 = rounds_cost(M, N, 256, 192, 72), c128 = rounds_cost(M, N, 128, 128, 31);
  // 128 x 128 tiles two to a compute unit (no adapter, K % 128 == 0): 512 tiles a round at
  // about 26 us (K = 3072), which wins between 256 and 512 of them -- 2048 x 3072 28.3 -> 22.7 us,
  // 1536 x 3072 28.0 -> 21.7 us, 2048 x 4096 31.3 -> 26.6 us, 2500 x 3072 30.5 -> 25.7 us
  const int64_t t128 = ((M + 127) / 128) * ((N + 127) / 128);
  const int64_t c2 = lt || K % kStageK != 0 || t128 <= 256 ? INT64_MAX : (t128 + 511) / 512 * 52;
  if (c2 < c256 && c2 < c192 && c2 < c128) return run_pair(xq, sx, w, sw, y, ldy, M, N, K, s, q);
  if (c256 <= c192 && c256 <= c128) return run<256, 256, 2>(xq, sx, w, sw, y, ldy, M, N, K, lt, lb, rank, s, q);
  if (c192 <= c128) return run<256, 192, 2>(xq, sx, w, sw, y, ldy, M, N, K, lt, lb, rank, s, q);
  return run<128, 128, 4>(xq, sx, w, sw, y, ldy, M, N, K, lt, lb, rank, s, q);
}

}  // namespace bsq
