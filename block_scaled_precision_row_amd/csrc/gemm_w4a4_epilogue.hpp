// The kernels of the nvfp4 W4A4 GEMM with an epilogue, for K % 256 == 0 (gemm_w4a4_epilogue.hip) and any other K
// (gemm_w4a4_any_epilogue.hip).
#pragma once

#include "epilogue.hpp"
#include "gemm_w4a4_tile.hpp"

namespace bsq {

namespace {

using namespace gemm;
using namespace w4a4;

template <int BM, int BN, int WPE, bool ANYK, int ACT>
__global__ __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(WPE, WPE)))
void gemm_w4a4_epilogue_kernel(DecArgs a, TileEpilogue<ACT> e) {
  w4a4_tile<BM, BN, false, TileEpilogue<ACT>, ANYK>(a, blockIdx.x, e);
}

template <int BM, int BN, bool ANYK>
hipError_t run_w4a4_epilogue(const DecArgs& a, const Epilogue& ep, hipStream_t s) {
  constexpr int WPE = BM == 128 && BN == 128 ? 2 : 1;
  const int tiles = (int)(((a.M + BM - 1) / BM) * ((a.N + BN - 1) / BN));
  return with_kind<TileEpilogue>(ep, [&](auto e) {
    hipLaunchKernelGGL((gemm_w4a4_epilogue_kernel<BM, BN, WPE, ANYK, decltype(e)::act>), dim3(tiles), dim3(kThreads), 0, s,
                       a, e);
    return hipGetLastError();
  });
}

}  // namespace
}  // namespace bsq
