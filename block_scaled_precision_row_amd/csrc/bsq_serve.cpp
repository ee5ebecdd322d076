// C ABI of the token-serving operators (declared in include/bsq_serve.h): argument checks on the
// host, then the launches.
#include "bsq_serve.h"

#include <cmath>

#include "serve_launch.hpp"

namespace {

constexpr int64_t kMaxStride = (int64_t)1 << 40;
constexpr int64_t kMaxRows = (int64_t)1 << 30;
constexpr int64_t kMaxBlocks = (int64_t)1 << 23;  // of 256 threads: below 2^31 threads a launch

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
bool is16(bsq_dtype dt) { return dt == BSQ_BF16 || dt == BSQ_FP16; }
bool stride_ok(int64_t st, int64_t sh) { return st >= 0 && sh >= 0 && st < kMaxStride && sh < kMaxStride; }

// rows of an output [T][H][D]: no two overlap
bool rows_apart(int64_t st, int64_t sh, int64_t T, int64_t H, int64_t D) {
  if (H > 1 && sh < D) return false;
  if (T > 1 && st < D) return false;
  if (H <= 1 || T <= 1) return true;
  return st >= (H - 1) * sh + D || sh >= (T - 1) * st + D;
}

bsq_status check_rotation(int64_t rot_dim, bsq_rope_layout layout, float factor) {
  if (layout != BSQ_ROPE_HALF && layout != BSQ_ROPE_INTERLEAVED) return BSQ_ERR_ARG;
  if (!std::isfinite(factor)) return BSQ_ERR_ARG;
  return rot_dim < 0 || rot_dim % 2 != 0 ? BSQ_ERR_SHAPE : BSQ_OK;
}

// shapes of a cache and a call's rows
bsq_status check_cache_shape(const bsq_kv8_cache* c, int64_t T) {
  if (!c) return BSQ_ERR_NULL;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return BSQ_ERR_SHAPE;
  const int64_t ps = c->page_size;
  if (ps != 16 && ps != 32 && ps != 64 && ps != 128 && ps != 256) return BSQ_ERR_SHAPE;
  if (c->kv_heads < 1 || c->kv_heads > 1024) return BSQ_ERR_SHAPE;
  if (c->num_pages < 1 || c->num_pages >= (int64_t)1 << 31) return BSQ_ERR_SHAPE;
  if (c->batch < 0 || c->batch > 65536) return BSQ_ERR_SHAPE;
  if (c->max_pages < 1 || c->max_pages > ((int64_t)1 << 31) || c->max_pages * ps >= ((int64_t)1 << 31) - 1024)
    return BSQ_ERR_SHAPE;
  if (c->table_stride < c->max_pages || c->table_stride >= kMaxStride) return BSQ_ERR_SHAPE;
  if (T < 0 || T > kMaxRows) return BSQ_ERR_SHAPE;
  return BSQ_OK;
}
bsq_status check_cache_pointers(const bsq_kv8_cache* c, const int32_t* cu) {
  if (!c->k || !c->v || !c->k_scale || !c->v_scale || !c->block_table || !c->seq_lens || !cu) return BSQ_ERR_NULL;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) ||
      !aligned(c->block_table, 4) || !aligned(c->seq_lens, 4) || !aligned(cu, 4))
    return BSQ_ERR_ALIGN;
  return BSQ_OK;
}
bsq::kv::Cache view_of(const bsq_kv8_cache* c) {
  bsq::kv::Cache v{};
  v.k = c->k; v.v = c->v; v.ks = c->k_scale; v.vs = c->v_scale;
  v.table = c->block_table; v.lens = c->seq_lens; v.table_stride = c->table_stride;
  v.num_pages = (int)c->num_pages; v.heads = (int)c->kv_heads;
  v.shift = __builtin_ctzll((unsigned long long)c->page_size);
  v.dim = (int)c->head_dim; v.batch = (int)c->batch; v.max_pages = (int)c->max_pages;
  return v;
}
// a 16-bit [T][H][D] operand read or written 16 bytes at a time
bsq_status check_wide(const void* p) {
  if (!p) return BSQ_ERR_NULL;
  return aligned(p, 16) ? BSQ_OK : BSQ_ERR_ALIGN;
}
bool wide_strides(int64_t st, int64_t sh) { return stride_ok(st, sh) && st % 8 == 0 && sh % 8 == 0; }

bsq_status finish(hipError_t e) { return e == hipSuccess ? BSQ_OK : bsq::hip_failure(e); }

}  // namespace

extern "C" {

bsq_status bsq_rope_inv_freq(int64_t rot_dim, double base, bsq_rope_scaling scaling, double factor,
                             int64_t trained_len, double beta_fast, double beta_slow, float* inv_freq,
                             float* attn_factor) {
  const int kind = (int)scaling;
  if (kind < BSQ_ROPE_PLAIN || kind > BSQ_ROPE_YARN) return BSQ_ERR_ARG;
  if (rot_dim < 2 || rot_dim > 1024 || rot_dim % 2 != 0 || (kind == BSQ_ROPE_NTK && rot_dim == 2))
    return BSQ_ERR_SHAPE;
  if (!std::isfinite(base) || base <= 1.0 || !std::isfinite(factor) || factor < 1.0) return BSQ_ERR_ARG;
  if (kind == BSQ_ROPE_PLAIN && factor != 1.0) return BSQ_ERR_ARG;
  if (kind == BSQ_ROPE_YARN && (trained_len < 1 || !(beta_slow >= 0.0) || !(beta_fast > beta_slow) ||
                                !std::isfinite(beta_fast)))
    return BSQ_ERR_ARG;
  if (!inv_freq || !attn_factor) return BSQ_ERR_NULL;
  const double r = (double)rot_dim;
  if (kind == BSQ_ROPE_NTK) base *= std::pow(factor, r / (r - 2.0));
  for (int64_t i = 0; i < rot_dim / 2; ++i) {
    double w = std::pow(base, -2.0 * (double)i / r);
    if (kind == BSQ_ROPE_LINEAR) w /= factor;
    if (kind == BSQ_ROPE_YARN) {
      const double turns = (double)trained_len * w / 6.283185307179586476925;
      double g = (turns - beta_slow) / (beta_fast - beta_slow);
      g = g < 0.0 ? 0.0 : (g > 1.0 ? 1.0 : g);
      w = w * g + w / factor * (1.0 - g);
    }
    inv_freq[i] = (float)w;
  }
  *attn_factor = kind == BSQ_ROPE_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.0f;
  return BSQ_OK;
}

bsq_status bsq_rope(bsq_dtype dtype, const void* x, int64_t x_stride_t, int64_t x_stride_h,
                    const int64_t* positions, const float* inv_freq, int64_t rot_dim, bsq_rope_layout layout,
                    float attn_factor, uint32_t flags, void* y, int64_t y_stride_t, int64_t y_stride_h, int64_t T,
                    int64_t H, int64_t D, hipStream_t stream) {
  if (!is16(dtype) && dtype != BSQ_FP32) return BSQ_ERR_ARG;
  if (flags & ~BSQ_ROPE_BACKWARD) return BSQ_ERR_ARG;
  bsq_status st = check_rotation(rot_dim, layout, attn_factor);
  if (st != BSQ_OK) return st;
  if (D < 1 || D > 1024 || rot_dim < 2 || rot_dim > D) return BSQ_ERR_SHAPE;
  if (T < 0 || T > kMaxRows || H < 0 || H > 65535) return BSQ_ERR_SHAPE;
  if (!stride_ok(x_stride_t, x_stride_h) || !stride_ok(y_stride_t, y_stride_h)) return BSQ_ERR_SHAPE;
  if (!rows_apart(y_stride_t, y_stride_h, T, H, D)) return BSQ_ERR_SHAPE;
  if (x == y && ((T > 1 && x_stride_t != y_stride_t) || (H > 1 && x_stride_h != y_stride_h))) return BSQ_ERR_SHAPE;
  if (T == 0 || H == 0) return BSQ_OK;
  if (!x || !y || !positions || !inv_freq) return BSQ_ERR_NULL;
  const uintptr_t size = dtype == BSQ_FP32 ? 4 : 2;
  if (!aligned(x, size) || !aligned(y, size) || !aligned(positions, 8) || !aligned(inv_freq, 4)) return BSQ_ERR_ALIGN;
  if ((st = bsq::current_device_status()) != BSQ_OK) return st;
  return finish(bsq::launch_rope(dtype, bsq::Strided{x, x_stride_t, x_stride_h}, positions,
                                 bsq::Rotation{inv_freq, (int)rot_dim, layout == BSQ_ROPE_INTERLEAVED, attn_factor},
                                 (flags & BSQ_ROPE_BACKWARD) != 0, bsq::Strided{y, y_stride_t, y_stride_h}, T, (int)H,
                                 (int)D, stream));
}

bsq_status bsq_kv_append(bsq_dtype dtype, const bsq_kv8_cache* cache, const int32_t* cu_seqlens, int64_t T,
                         const void* k, int64_t k_stride_t, int64_t k_stride_h, const void* v, int64_t v_stride_t,
                         int64_t v_stride_h, const float* inv_freq, int64_t rot_dim, bsq_rope_layout layout,
                         float attn_factor, const void* q, int64_t q_stride_t, int64_t q_stride_h, int64_t q_heads,
                         void* q_out, int64_t o_stride_t, int64_t o_stride_h, hipStream_t stream) {
  if (!is16(dtype)) return BSQ_ERR_ARG;
  bsq_status st = check_cache_shape(cache, T);
  if (st != BSQ_OK) return st;
  if ((st = check_rotation(rot_dim, layout, attn_factor)) != BSQ_OK) return st;
  if (rot_dim % 16 != 0 || rot_dim > cache->head_dim) return BSQ_ERR_SHAPE;
  if (!wide_strides(k_stride_t, k_stride_h) || !wide_strides(v_stride_t, v_stride_h)) return BSQ_ERR_SHAPE;
  const bool queries = q || q_out;
  if (queries) {
    if (q_heads < 1 || q_heads > 65535) return BSQ_ERR_SHAPE;
    if (!wide_strides(q_stride_t, q_stride_h) || !wide_strides(o_stride_t, o_stride_h)) return BSQ_ERR_SHAPE;
    if (!rows_apart(o_stride_t, o_stride_h, T, q_heads, cache->head_dim)) return BSQ_ERR_SHAPE;
    if (q == q_out && ((T > 1 && q_stride_t != o_stride_t) || (q_heads > 1 && q_stride_h != o_stride_h)))
      return BSQ_ERR_SHAPE;
  } else if (q_heads != 0) {
    return T > 0 && cache->batch > 0 ? BSQ_ERR_NULL : BSQ_ERR_SHAPE;
  }
  const int shift = __builtin_ctzll((unsigned long long)cache->page_size);
  const int64_t blocks = bsq::kv::append_slots(T, cache->batch, shift) * cache->kv_heads + (queries ? T : 0);
  if (blocks >= kMaxBlocks) return BSQ_ERR_SHAPE;
  if (T == 0 || cache->batch == 0) return BSQ_OK;
  if ((st = check_cache_pointers(cache, cu_seqlens)) != BSQ_OK) return st;
  if ((st = check_wide(k)) != BSQ_OK) return st;
  if ((st = check_wide(v)) != BSQ_OK) return st;
  if (rot_dim > 0 && !inv_freq) return BSQ_ERR_NULL;
  if (rot_dim > 0 && !aligned(inv_freq, 4)) return BSQ_ERR_ALIGN;
  if (queries) {
    if ((st = check_wide(q)) != BSQ_OK) return st;
    if ((st = check_wide(q_out)) != BSQ_OK) return st;
  }
  if ((st = bsq::current_device_status()) != BSQ_OK) return st;
  bsq::AppendArgs a{};
  a.c = view_of(cache);
  a.cu = cu_seqlens;
  a.T = T;
  a.k = bsq::Strided{k, k_stride_t, k_stride_h};
  a.v = bsq::Strided{v, v_stride_t, v_stride_h};
  a.q = bsq::Strided{q, q_stride_t, q_stride_h};
  a.qo = bsq::Strided{q_out, o_stride_t, o_stride_h};
  a.q_heads = (int)q_heads;
  a.r = bsq::Rotation{inv_freq, (int)rot_dim, layout == BSQ_ROPE_INTERLEAVED, attn_factor};
  return finish(bsq::launch_kv_append(dtype, a, stream));
}

namespace {
bool attention_shape(int64_t batch, int64_t T, int64_t max_q_len, int64_t q_heads, int64_t kv_heads,
                     int64_t head_dim) {
  if (batch < 0 || batch > 65536 || T < 0 || T > kMaxRows) return false;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return false;
  if (kv_heads < 1 || kv_heads > 1024 || q_heads < 1 || q_heads % kv_heads != 0 || q_heads > 65535) return false;
  if ((T * (q_heads / kv_heads) / 128 + batch) * kv_heads >= kMaxBlocks) return false;
  return max_q_len >= 0 && (max_q_len > 0 || T == 0);
}
}  // namespace

size_t bsq_attention_kv8_workspace_bytes(int64_t batch, int64_t T, int64_t max_q_len, int64_t q_heads,
                                         int64_t kv_heads, int64_t head_dim) {
  if (!attention_shape(batch, T, max_q_len, q_heads, kv_heads, head_dim) || batch == 0 || T == 0) return 0;
  return bsq::attention_workspace(batch, T, max_q_len, q_heads, kv_heads, head_dim);
}

bsq_status bsq_attention_kv8(bsq_dtype dtype, const bsq_kv8_cache* cache, const int32_t* cu_seqlens, int64_t T,
                             int64_t max_q_len, const void* q, int64_t q_stride_t, int64_t q_stride_h,
                             int64_t q_heads, float softmax_scale, int64_t window, uint32_t flags, void* y,
                             int64_t y_stride_t, int64_t y_stride_h, float* lse, void* workspace,
                             size_t workspace_bytes, hipStream_t stream) {
  if (!is16(dtype) || (flags & ~BSQ_ATTN_FULL)) return BSQ_ERR_ARG;
  bsq_status st = check_cache_shape(cache, T);
  if (st != BSQ_OK) return st;
  if (!std::isfinite(softmax_scale * 1.44269504088896340736f) || window < 0 || (window > 0 && (flags & BSQ_ATTN_FULL))) return BSQ_ERR_ARG;
  if (!attention_shape(cache->batch, T, max_q_len, q_heads, cache->kv_heads, cache->head_dim)) return BSQ_ERR_SHAPE;
  if (cache->batch * (cache->max_pages * cache->page_size / 64 + 1) >= (int64_t)1 << 31) return BSQ_ERR_SHAPE;
  if (!wide_strides(q_stride_t, q_stride_h) || !wide_strides(y_stride_t, y_stride_h)) return BSQ_ERR_SHAPE;
  if (!rows_apart(y_stride_t, y_stride_h, T, q_heads, cache->head_dim)) return BSQ_ERR_SHAPE;
  if (T == 0 || cache->batch == 0) return BSQ_OK;
  if ((st = check_cache_pointers(cache, cu_seqlens)) != BSQ_OK) return st;
  if ((st = check_wide(q)) != BSQ_OK) return st;
  if ((st = check_wide(y)) != BSQ_OK) return st;
  if (lse && !aligned(lse, 4)) return BSQ_ERR_ALIGN;
  const size_t need = bsq_attention_kv8_workspace_bytes(cache->batch, T, max_q_len, q_heads, cache->kv_heads,
                                                        cache->head_dim);
  if (need > 0 && (!workspace || workspace_bytes < need)) return BSQ_ERR_WORKSPACE;
  if (need > 0 && !aligned(workspace, 256)) return BSQ_ERR_ALIGN;
  if ((st = bsq::current_device_status()) != BSQ_OK) return st;
  bsq::AttnArgs a{};
  a.c = view_of(cache);
  a.cu = cu_seqlens;
  a.T = T;
  a.max_q_len = max_q_len;
  a.q = bsq::Strided{q, q_stride_t, q_stride_h};
  a.y = bsq::Strided{y, y_stride_t, y_stride_h};
  a.q_heads = (int)q_heads;
  a.scale = softmax_scale;
  // (positions are below 2^31: a window of 2^32 hides nothing, and a wider one must not take them past 64 bits)
  a.window = window < (int64_t)1 << 32 ? window : (int64_t)1 << 32;
  a.full = (flags & BSQ_ATTN_FULL) != 0;
  a.lse = lse;
  return finish(bsq::launch_attention(dtype, a, workspace, stream));
}

bsq_status bsq_gemm_int4g(bsq_dtype dtype, const void* x, int64_t ldx, const uint8_t* w, const void* w_scale,
                          const uint8_t* w_zero, int64_t group, void* y, int64_t ldy, int64_t M, int64_t N,
                          int64_t K, hipStream_t stream) {
  if (!is16(dtype)) return BSQ_ERR_ARG;
  if (group != 32 && group != 64 && group != 128) return BSQ_ERR_ARG;
  if (M < 0 || M > kMaxRows || N < 0 || N > kMaxRows) return BSQ_ERR_SHAPE;
  if (K <= 0 || K > (int64_t)1 << 20 || K % group != 0) return BSQ_ERR_SHAPE;
  if (ldx < K || ldx % 8 != 0 || ldx >= kMaxStride || ldy < N || ldy >= kMaxStride) return BSQ_ERR_SHAPE;
  if (M == 0 || N == 0) return BSQ_OK;
  if (!x || !w || !w_scale || !y) return BSQ_ERR_NULL;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(w_scale, 2) || !aligned(y, 16)) return BSQ_ERR_ALIGN;
  if ((M + 15) / 16 > 65535 || (N + 15) / 16 >= kMaxBlocks) return BSQ_ERR_SHAPE;
  bsq_status st = bsq::current_device_status();
  if (st != BSQ_OK) return st;
  bsq::Int4Args a{};
  a.x = x; a.ldx = ldx; a.w = w; a.ws = w_scale; a.wz = w_zero; a.group = (int)group;
  a.y = y; a.ldy = ldy; a.M = M; a.N = N; a.K = (int)K;
  return finish(bsq::launch_gemm_int4g(dtype, a, stream));
}

}  // extern "C"
