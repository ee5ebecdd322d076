// nvfp4 W4A4 GEMM with an epilogue (include/bsq_block.h), K % 256 == 0: the tiles of gemm_w4a4_tile.hpp, whose sums go
// through bias, activation, gate and residual (epilogue.hpp) before they are rounded. Tiles by the rules of gemm_w4a4.hip,
// whose figures hold: 4608 x 2560 x 10240 with gates of five groups and a residual 198 us, 1.2 PFLOP/s (the plain linear
// 194), bound by the matrix cores and the decoding beside them.
#include "gemm_w4a4_epilogue.hpp"

namespace bsq {

hipError_t launch_gemm_w4a4_epilogue(const DecArgs& args, const Epilogue& ep, hipStream_t s) {
  DecArgs a = args;
  a.stream_y = stream_output((a.M + a.N) * (a.K / 2 + a.K / 16), a.M, a.N);
  const int64_t t64 = ((a.M + 63) / 64) * ((a.N + 63) / 64), t64x128 = ((a.M + 63) / 64) * ((a.N + 127) / 128);
  if (t64 <= 256) return run_w4a4_epilogue<64, 64, false>(a, ep, s);
  if (t64x128 <= 256) return run_w4a4_epilogue<64, 128, false>(a, ep, s);
  const int64_t c256 = rounds_cost(a.M, a.N, 256, 256, 76), c192 = rounds_cost(a.M, a.N, 256, 192, 60);
  const int64_t c128 = ((a.M + 127) / 128 * ((a.N + 127) / 128) + 511) / 512 * 49;
  if (c256 <= c192 && c256 <= c128) return run_w4a4_epilogue<256, 256, false>(a, ep, s);
  if (c192 <= c128) return run_w4a4_epilogue<256, 192, false>(a, ep, s);
  return run_w4a4_epilogue<128, 128, false>(a, ep, s);
}

}  // namespace bsq
