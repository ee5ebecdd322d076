// nvfp4 W4A4 GEMM with an epilogue for K % 256 != 0: the tiles of gemm_w4a4_tile.hpp with their block scales by way of
// registers, loaded with the stage's codes and written to LDS in front of the barrier that publishes it: 360 x 89 x 6048
// with everything 28 us and 4501 x 792 x 1184 23 us (the dword-DMA tile of gemm_dec.hip, one stage in flight: 179 and
// 40). Of gemm_w4a4.hip's tiles there are three here: 64 x 64 while its grid fits one round, then 128 x 128 or 256 x 192
// by whole rounds. What the partial stage and the missing 64 x 128 and 256 x 256 tiles cost together, cold:
// 777 x 1234 x 1056, 70 tiles of 128 x 128, 24.6 us where x 1024 takes 15.7 on 64 x 128; 4500 x 6100 x 1056 160 us, x 1024 136.
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
