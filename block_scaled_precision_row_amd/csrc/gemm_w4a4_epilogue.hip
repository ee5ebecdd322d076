// nvfp4 W4A4 GEMM with an epilogue (include/bsq_block.h): the tiles of gemm_w4a4_tile.hpp, whose sums go through bias,
// activation, gate and residual (epilogue.hpp) before they are rounded.
#include "epilogue.hpp"
#include "gemm_w4a4_tile.hpp"

namespace bsq {

namespace {

using namespace gemm;
using namespace w4a4;

template <int BM, int BN, int WPE, int ACT>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(WPE, WPE)))
void gemm_w4a4_epilogue_kernel(DecArgs a, TileEpilogue<ACT> e) {
  w4a4_tile<BM, BN, false>(a, blockIdx.x, e);
}

template <int BM, int BN>
hipError_t run(const DecArgs& a, const Epilogue& ep, hipStream_t s) {
  constexpr int WPE = BM == 128 && BN == 128 ? 2 : 1;
  const int tiles = (int)(((a.M + BM - 1) / BM) * ((a.N + BN - 1) / BN));
  return with_kind<TileEpilogue>(ep, [&](auto e) {
    hipLaunchKernelGGL((gemm_w4a4_epilogue_kernel<BM, BN, WPE, decltype(e)::act>), dim3(tiles), dim3(kThreads), 0, s,
                       a, e);
    return hipGetLastError();
  });
}

}  // namespace

hipError_t launch_gemm_w4a4_epilogue(const DecArgs& args, const Epilogue& ep, hipStream_t s) {
  DecArgs a = args;
  a.stream_y = stream_output((a.M + a.N) * (a.K / 2 + a.K / 16), a.M, a.N);
  const int64_t t64 = ((a.M + 63) / 64) * ((a.N + 63) / 64), t64x128 = ((a.M + 63) / 64) * ((a.N + 127) / 128);
  if (t64 <= 256) return run<64, 64>(a, ep, s);
  if (t64x128 <= 256) return run<64, 128>(a, ep, s);
  const int64_t c256 = rounds_cost(a.M, a.N, 256, 256, 76), c192 = rounds_cost(a.M, a.N, 256, 192, 60);
  const int64_t c128 = ((a.M + 127) / 128 * ((a.N + 127) / 128) + 511) / 512 * 49;
  if (c256 <= c192 && c256 <= c128) return run<256, 256>(a, ep, s);
  if (c192 <= c128) return run<256, 192>(a, ep, s);
  return run<128, 128>(a, ep, s);
}

}  // namespace bsq
