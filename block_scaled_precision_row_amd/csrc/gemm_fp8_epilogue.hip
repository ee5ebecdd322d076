// fp8r W8A8 GEMM with an epilogue (include/bsq_block.h): the tiles of gemm_fp8_tile.hpp, whose sums go through bias,
// activation, gate and residual (epilogue.hpp) before they are rounded.
//
// Bound by the matrix cores' feed, as without an epilogue: 4096 x 10240 x 2560 with gelu_tanh 128 us, 1.7 PFLOP/s (the plain
// linear 127). Forced onto other tiles: 256 x 256 145 us, 256 x 192 155, 128 x 128 alone with four buffers 191.
#include "epilogue.hpp"
#include "gemm_fp8_tile.hpp"

namespace bsq {

namespace {

using namespace gemm;
using namespace fp8;

template <int BM, int BN, int NS, bool HS, int WPE, int ACT>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(WPE, WPE)))
void gemm_fp8_epilogue_kernel(const uint8_t* __restrict__ xq, const float* __restrict__ sx,
                              const uint8_t* __restrict__ w, const float* __restrict__ sw, uint16_t* y, int64_t ldy,
                              int M, int N, int K, int stream_y, TileEpilogue<ACT> e) {
  fp8_tile<BM, BN, NS, false, 0, HS, kLoraGlobal>(xq, sx, w, sw, y, ldy, M, N, K, nullptr, nullptr, 0, stream_y,
                                                  YQuant{}, blockIdx.x, e);
}

template <int BM, int BN, int NS, bool HS, int WPE = 1>
hipError_t run(const DecArgs& a, const Epilogue& ep, hipStream_t s) {
  const int tiles = (int)(((a.M + BM - 1) / BM) * ((a.N + BN - 1) / BN));
  const int st = (int)stream_output((a.M + a.N) * a.K, a.M, a.N);
  return with_kind<TileEpilogue>(ep, [&](auto e) {
    hipLaunchKernelGGL((gemm_fp8_epilogue_kernel<BM, BN, NS, HS, WPE, decltype(e)::act>), dim3(tiles), dim3(kThreads),
                       0, s, a.xq, a.sx, a.w, a.sw, a.y, a.ldy, (int)a.M, (int)a.N, (int)a.K, st, e);
    return hipGetLastError();
  });
}

}  // namespace

// Tiles by the rules of gemm_fp8.hip, whose figures hold: the smallest while its grid fits one round, then the tile of
// least expected time over whole rounds. The hand-ordered loop takes any K here (a partial last stage's loads are made
// apart), so that no K leaves the large tiles.
hipError_t launch_gemm_fp8_epilogue(const DecArgs& a, const Epilogue& ep, hipStream_t s) {
  const int64_t t64 = ((a.M + 63) / 64) * ((a.N + 63) / 64), t64x128 = ((a.M + 63) / 64) * ((a.N + 127) / 128);
  if (t64 <= 256) return run<64, 64, 4, false>(a, ep, s);
  if (t64x128 <= 256) return run<64, 128, 4, false>(a, ep, s);
  const int64_t c256 = rounds_cost(a.M, a.N, 256, 256, 92), c192 = rounds_cost(a.M, a.N, 256, 192, 72);
  const int64_t c2 = (((a.M + 127) / 128) * ((a.N + 127) / 128) + 511) / 512 * 52;
  if (c2 <= c256 && c2 <= c192) return run<128, 128, 2, true, 2>(a, ep, s);
  if (c256 <= c192) return run<256, 256, 2, true>(a, ep, s);
  return run<256, 192, 2, true>(a, ep, s);
}

}  // namespace bsq
