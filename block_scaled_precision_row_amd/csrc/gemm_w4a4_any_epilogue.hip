// nvfp4 W4A4 GEMM with an epilogue for K % 256 != 0: the tiles of gemm_w4a4_tile.hpp with their block scales by way of
// registers, loaded with the stage's codes and written to LDS in front of the barrier that publishes it: 360 x 89 x 6048
// with everything 28 us and 4501 x 792 x 1184 23 us (the dword-DMA tile of gemm_dec.hip, one stage in flight: 179 and
// 40). The tiles are those of gemm_w4a4.hip that cost least; its others differ by less than the partial stage costs.
#include "gemm_w4a4_epilogue.hpp"

namespace bsq {

hipError_t launch_gemm_w4a4_any_epilogue(const DecArgs& args, const Epilogue& ep, hipStream_t s) {
  DecArgs a = args;
  a.stream_y = stream_output((a.M + a.N) * (a.K / 2 + a.K / 16), a.M, a.N);
  if (((a.M + 63) / 64) * ((a.N + 63) / 64) <= 256) return run_w4a4_epilogue<64, 64, true>(a, ep, s);
  const int64_t c192 = rounds_cost(a.M, a.N, 256, 192, 60);
  const int64_t c128 = ((a.M + 127) / 128 * ((a.N + 127) / 128) + 511) / 512 * 49;
  if (c192 <= c128) return run_w4a4_epilogue<256, 192, true>(a, ep, s);
  return run_w4a4_epilogue<128, 128, true>(a, ep, s);
}

}  // namespace bsq
