// Internal launch interface of the token-serving operators (include/bsq_serve.h) between the C
// ABI (bsq_serve.cpp) and the kernels. Arguments are validated by the caller; each function
// enqueues its kernels on `s` and returns the launch status.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bsq_serve.h"
#include "kv_index.hpp"

namespace bsq {

// shared with bsq.h's entry points (bsq_api.cpp)
bsq_status current_device_status();
bsq_status hip_failure(hipError_t e);

// a [rows][heads][dim] tensor: strides in elements, dim contiguous
struct Strided {
  const void* p;
  int64_t st, sh;
};
struct Rotation {
  const float* inv_freq;  // [rot / 2], null when rot == 0
  int rot;
  bool interleaved;
  float factor;
};

hipError_t launch_rope(bsq_dtype dt, Strided x, const int64_t* positions, Rotation r, bool backward, Strided y,
                       int64_t T, int H, int D, hipStream_t s);

struct AppendArgs {
  kv::Cache c;
  const int32_t* cu;
  int64_t T;
  Strided k, v, q, qo;
  int q_heads;
  Rotation r;
};
hipError_t launch_kv_append(bsq_dtype dt, const AppendArgs& a, hipStream_t s);

struct AttnArgs {
  kv::Cache c;
  const int32_t* cu;
  int64_t T;
  int64_t max_q_len;
  Strided q, y;
  int q_heads;
  float scale;
  int64_t window;
  bool full;
  float* lse;
};
size_t attention_workspace(int64_t batch, int64_t T, int64_t max_q_len, int64_t q_heads, int64_t kv_heads,
                           int64_t head_dim);
hipError_t launch_attention(bsq_dtype dt, const AttnArgs& a, void* workspace, hipStream_t s);

struct Int4Args {
  const void* x;
  int64_t ldx;
  const uint8_t* w;
  const void* ws;
  const uint8_t* wz;
  int group;
  void* y;
  int64_t ldy;
  int64_t M, N;
  int K;
};
hipError_t launch_gemm_int4g(bsq_dtype dt, const Int4Args& a, hipStream_t s);

}  // namespace bsq
