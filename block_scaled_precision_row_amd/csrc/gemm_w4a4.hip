// nvfp4 W4A4 GEMM: packed E2M1 operands decoded in registers, f16 matrix cores.
//
// "BFL (fp8r / nvfp4)", nvfp4 bullet: a value is e2m1 * e4m3(scale of its
// 16-element block) * global scale, and activations are quantized the same
// way with the calibrated input_scale before an fp4 GEMM ("Kernels" table):
//   y[m][n] = bf16( (sum_k xh[m][k] * wh[n][k]) * gx * gw ),
//   xh = e2m1(xq) * e4m3(sfx),  wh = e2m1(wq) * e4m3(sfw).
// An E2M1 value (2 significant bits) times an E4M3 scale (4 significant bits)
// has at most 6 significant bits and lies in [2^-10, 2688], so xh and wh are
// exact in f16; the contraction runs on v_mfma_f32_32x32x16_f16 with fp32
// accumulation and the two fp32 global scales go to the epilogue. (gfx950's
// block-scaled FP4 MFMA applies power-of-two scales per 32 elements, which
// cannot carry an E4M3 scale per 16.)
//
// Data movement (conventions in gemm_common.hpp): a stage is 256 K values
// of every W and Xq row -- 128 bytes of packed codes (one full cache line)
// plus 16 block-scale bytes -- copied to LDS as stored by LDS DMA into one of
// two stage buffers while the other is multiplied. Long stages keep the
// number of memory requests low (small per-row segments would cost one
// request each). Every wave reads its operands' packed bytes from LDS one
// 64-deep K group ahead and decodes them in registers right before the MFMAs
// of each 16-deep K step: per byte one v_cvt_scalef32_pk_f16_fp4 (exact
// E2M1 -> f16 pair) and one v_pk_mul_f16 by the block scale. LDS traffic
// stays at the packed size; the decode work (about 4 VALU per MFMA) issues
// under the MFMAs.
//
// K permutation: lane half h of an MFMA operand covers K values
// [128 h, 128 h + 128) of a stage -- 32 of them per 64-deep K group q, at
// [128 h + 32 q, 128 h + 32 q + 32), one 8-value group per K step -- for both
// operands alike, so every product pairs equal K indices. A lane's 8 block
// scales of a stage are then 8 consecutive bytes, read once per stage.
#include <cmath>

#include "gemm_w4a4_tile.hpp"

namespace bsq {

namespace {

using namespace gemm;
using namespace w4a4;

template <int BM, int BN, bool LORA, int WPE>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(WPE, WPE)))
void gemm_w4a4_kernel(DecArgs a) {
  w4a4_tile<BM, BN, LORA>(a, blockIdx.x);
}

// The tiles of several W4A4 GEMMs in one grid: the problem of each workgroup, then that
// problem's tile, exactly as its own launch would compute it (same tile shape, same bits).
struct W4Group {
  DecArgs p[kMaxGroup];
  int start[kMaxGroup + 1];
  int count;
};
template <int BM, int BN, int WPE>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(WPE, WPE)))
void gemm_w4a4_grouped_kernel(W4Group g) {
  const int bid = blockIdx.x;
  const int p = group_problem(g.start, g.count, bid);
  w4a4_tile<BM, BN, false>(g.p[p], bid - g.start[p]);
}

// WPE: waves per SIMD the registers are budgeted for. The 128 x 128 tile takes 72 KB of LDS, so
// two of its workgroups share a compute unit when each wave keeps to 256 registers; the decode
// VALU of one then overlaps the other's MFMAs.
template <int BM, int BN>
hipError_t run(const DecArgs& a, hipStream_t s) {
  constexpr int WPE = BM == 128 && BN == 128 ? 2 : 1;
  const int tiles = (int)(((a.M + BM - 1) / BM) * ((a.N + BN - 1) / BN));
  if (a.lt)
    hipLaunchKernelGGL((gemm_w4a4_kernel<BM, BN, true, WPE>), dim3(tiles), dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((gemm_w4a4_kernel<BM, BN, false, WPE>), dim3(tiles), dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace

bool gemm_w4a4_supported(const DecArgs& a) { return a.K % kStageK == 0; }

// Grouped W4A4: every problem with K % 256 == 0 and plain bf16 output (no adapter, no quantized
// output). The tile rule and its measurements are those of the grouped fp8r launch (128 x 128
// tiles two to a compute unit below three rounds of 256 x 192 tiles, else the 256 x 256 or
// 256 x 192 tile of least expected time over whole rounds), except that the decode-heavier W4A4
// tile already pays from 256 pair tiles (half a round): a joint block at 192 / 256 / 320 tokens
// as one grid 91.3 / 91.1 / 94.2 us against four launches 99.2 / 106.0 / 121.3 us, where the fp8r
// block lost (93.3 / 100.9 / 91.8 vs 76.6 / 83.3 / 86.7 us) and keeps the full round.
namespace {
struct GroupTile {
  int bm, bn, per_round, round_us;
};
constexpr GroupTile kW4GroupTiles[3] = {{256, 256, 256, 76}, {256, 192, 256, 60}, {128, 128, 512, 49}};
// the group's tile (index into kW4GroupTiles), or -1 when no tile fills two rounds
int w4a4_group_tile(const DecArgs* p, int count) {
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
  if (tiles_of(kW4GroupTiles[1], nullptr) < 3 * 256) {
    const int64_t t = tiles_of(kW4GroupTiles[2], nullptr);
    return t >= 256 && t < ((int64_t)1 << 31) ? 2 : -1;  // half a round of pairs already pays
  }
  int best = -1;
  double best_cost = 0;
  for (int t = 0; t < 2; ++t) {
    const GroupTile& c = kW4GroupTiles[t];
    double work = 0;
    const int64_t tiles = tiles_of(c, &work);
    if (tiles < 2 * (int64_t)c.per_round || tiles >= ((int64_t)1 << 31)) continue;  // 32-bit workgroup ids
    const double cost = std::ceil(work / c.per_round - 1e-9) * c.round_us;
    if (best < 0 || cost < best_cost) best = t, best_cost = cost;
  }
  return best;
}
template <int BM, int BN, int WPE>
hipError_t run_w4a4_group(const DecArgs* p, int count, hipStream_t s) {
  W4Group g{};
  g.count = count;
  int64_t total = 0;
  for (int i = 0; i < count; ++i) {
    g.p[i] = p[i];
    g.p[i].stream_y = stream_output((p[i].M + p[i].N) * (p[i].K / 2 + p[i].K / 16), p[i].M, p[i].N);
    g.start[i] = (int)total;
    total += ((p[i].M + BM - 1) / BM) * ((p[i].N + BN - 1) / BN);
  }
  for (int i = count; i <= kMaxGroup; ++i) g.start[i] = (int)total;
  hipLaunchKernelGGL((gemm_w4a4_grouped_kernel<BM, BN, WPE>), dim3((unsigned)total), dim3(kThreads), 0, s, g);
  return hipGetLastError();
}
}  // namespace

bool gemm_w4a4_grouped_supported(const DecArgs* p, int count) {
  if (count < 2 || count > kMaxGroup) return false;
  for (int i = 0; i < count; ++i)
    if (p[i].K % kStageK != 0 || p[i].lt || p[i].yq || p[i].ypmax || !p[i].y) return false;
  return w4a4_group_tile(p, count) >= 0;
}

hipError_t launch_gemm_w4a4_grouped(const DecArgs* p, int count, hipStream_t s) {
  switch (w4a4_group_tile(p, count)) {
    case 0: return run_w4a4_group<256, 256, 1>(p, count, s);
    case 1: return run_w4a4_group<256, 192, 1>(p, count, s);
    default: return run_w4a4_group<128, 128, 2>(p, count, s);
  }
}

bool lora_pre_scaled_w4a4(const DecArgs& a) { return gemm_w4a4_supported(a); }

hipError_t launch_gemm_w4a4(const DecArgs& args, hipStream_t s) {
  DecArgs a = args;
  a.stream_y = stream_output((a.M + a.N) * (a.K / 2 + a.K / 16), a.M, a.N);
  // While its grid fits one round on the 256 compute units, the smallest tile (64 x 64, then
  // 64 tokens x 128 weight rows): a grid of few large tiles leaves units idle while each busy
  // one waits on its own loads. Measured at K = 3072: 512 x 3072 26.6 -> 19.2 us, 256 x 3072
  // 27 -> 13.3 us, 64 x 12288 29 -> 14 us, 512 x 3072 x 12288 88 -> 64 us.
  //
  // Larger grids take the tile of least expected time over whole rounds, with round times
  // measured at K = 3072 with every unit busy: 256 x 256 76 us and 256 x 192 60 us for 256
  // tiles, 128 x 128 49 us for 512 (two workgroups a compute unit). The square tile does the
  // most work per operand byte and per decode, so it wins when the rounds come out even, as at
  // 4096 x 12288: 230 vs 240 us. Where they do not: 3072 x 3072 75 -> 53 us and 4096 x 6144
  // 136 -> 122 us on 256 x 192; 2048 x 3072 54 -> 43 us and 1536 x 3072 48 -> 41 us on
  // 128 x 128. Every tile shape gives the same bits.
  const int64_t t64 = ((a.M + 63) / 64) * ((a.N + 63) / 64), t64x128 = ((a.M + 63) / 64) * ((a.N + 127) / 128);
  if (t64 <= 256) return run<64, 64>(a, s);
  if (t64x128 <= 256) return run<64, 128>(a, s);
  const int64_t c256 = rounds_cost(a.M, a.N, 256, 256, 76), c192 = rounds_cost(a.M, a.N, 256, 192, 60);
  const int64_t c128 = ((a.M + 127) / 128 * ((a.N + 127) / 128) + 511) / 512 * 49;
  if (c256 <= c192 && c256 <= c128) return run<256, 256>(a, s);
  if (c192 <= c128) return run<256, 192>(a, s);
  return run<128, 128>(a, s);
}

}  // namespace bsq
