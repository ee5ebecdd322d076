/*
 * bsq_serve.h -- token-serving operators next to the quantized linears of
 * bsq.h: rotary positions, a paged key/value cache held in E4M3 with a scale
 * for each page and head (append and attention), and few-token linears with
 * 4-bit integer weights and group scales.
 *
 * The conventions of bsq.h hold: device pointers owned by the caller, work
 * enqueued on `stream`, nothing allocated, freed or synchronized, arguments
 * validated on the host before any HIP call, no exception across the ABI, the
 * same inputs give the same bits (no atomics). 16-bit tensors are passed as
 * `void*` with a bsq_dtype. What a call reads from device memory (lengths,
 * page tables) cannot be validated on the host; every entry point states what
 * it does with values out of range, and none of them reads or writes memory
 * outside the tensors it was given.
 */
#ifndef BSQ_SERVE_H
#define BSQ_SERVE_H

#include "bsq.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum { BSQ_BF16 = 1, BSQ_FP16 = 2, BSQ_FP32 = 3 } bsq_dtype;

/* Which elements of a head form the rotated pairs (r = rot_dim):
 * HALF: (i, i + r/2); INTERLEAVED: (2i, 2i + 1); 0 <= i < r/2. */
typedef enum { BSQ_ROPE_HALF = 1, BSQ_ROPE_INTERLEAVED = 2 } bsq_rope_layout;

/* Frequencies of a rotation over rot_dim elements (host function, plain host
 * memory): w_i = base^(-2i / rot_dim) for 0 <= i < rot_dim / 2, stretched for
 * contexts longer than the trained one:
 *   BSQ_ROPE_PLAIN   as they are (factor must be 1)
 *   BSQ_ROPE_LINEAR  w_i / factor
 *   BSQ_ROPE_NTK     base * factor^(r / (r - 2)) in the place of base (r > 2)
 *   BSQ_ROPE_YARN    w_i * g_i + w_i / factor * (1 - g_i), where
 *                    g_i = clamp((t_i - beta_slow) / (beta_fast - beta_slow), 0, 1)
 *                    and t_i = trained_len * w_i / (2 pi) is how often pair i
 *                    turns over the trained length: pairs of many turns keep
 *                    their frequency. *attn_factor = 0.1 ln(factor) + 1.
 *                    (A ramp along the pair's index i between the pairs of
 *                    beta_fast and beta_slow turns is another one: a checkpoint
 *                    that was trained with it needs its own frequencies, which
 *                    bsq_rope and bsq_kv_append take as they take these.)
 * Computed in 64 bits and rounded once to fp32. *attn_factor is 1 otherwise.
 * trained_len, beta_fast, beta_slow are read for YARN only.
 * BSQ_ERR_SHAPE: rot_dim odd, < 2 or > 1024 (for NTK also 2). BSQ_ERR_ARG: an
 * unknown scaling, base not finite or <= 1, factor not finite or < 1, or for
 * YARN trained_len < 1 or not 0 <= beta_slow < beta_fast (finite).
 *   inv_freq [rot_dim / 2] fp32 (host), attn_factor [1] fp32 (host)
 */
typedef enum { BSQ_ROPE_PLAIN = 0, BSQ_ROPE_LINEAR = 1, BSQ_ROPE_NTK = 2, BSQ_ROPE_YARN = 3 } bsq_rope_scaling;
bsq_status bsq_rope_inv_freq(int64_t rot_dim, double base, bsq_rope_scaling scaling, double factor,
                             int64_t trained_len, double beta_fast, double beta_slow, float* inv_freq,
                             float* attn_factor);

/*
 * Rotary positions. For token t at position p = positions[t] and every head,
 * with angle a_i = p * inv_freq[i] and f = attn_factor, pair i of the first
 * rot_dim elements becomes
 *   (x0, x1) -> f * (x0 cos a_i - x1 sin a_i, x1 cos a_i + x0 sin a_i);
 * the other elements are copied. With BSQ_ROPE_BACKWARD the angles are
 * negated: the gradient of x for a given gradient of y (the rotation's
 * transpose). Angles are reduced in 64 bits, so far positions lose nothing;
 * products and sums are fp32, rounded once to the tensor's type.
 *   x, y [T][H][D] of `dtype` (any of the three), D contiguous, strides in
 *     elements; x's strides may be 0 (a broadcast input). y may be x with the
 *     same strides (in place), otherwise they must not overlap.
 *   positions [T] int64 (any value of magnitude below 2^53), inv_freq
 *     [rot_dim / 2] fp32
 * 1 <= D <= 1024, rot_dim even, 2 <= rot_dim <= D; 0 <= T <= 2^30, 0 <= H <=
 * 65535 (0: nothing to do); strides >= 0 and < 2^40, y's rows must not overlap one another
 * (BSQ_ERR_SHAPE). Pointers aligned to their element size. BSQ_ERR_ARG for an
 * unknown dtype, layout or flag, or an attn_factor that is not finite.
 */
#define BSQ_ROPE_BACKWARD 0x1u
bsq_status bsq_rope(bsq_dtype dtype, const void* x, int64_t x_stride_t, int64_t x_stride_h,
                    const int64_t* positions, const float* inv_freq, int64_t rot_dim, bsq_rope_layout layout,
                    float attn_factor, uint32_t flags, void* y, int64_t y_stride_t, int64_t y_stride_h, int64_t T,
                    int64_t H, int64_t D, hipStream_t stream);

/*
 * A paged key/value cache in E4M3. A page holds page_size consecutive tokens
 * of one sequence, for every kv head:
 *   k [num_pages][kv_heads][page_size][head_dim] E4M3 codes
 *   v [num_pages][kv_heads][head_dim][page_size] E4M3 codes (each element's
 *     tokens contiguous, the order in which attention consumes them)
 *   k_scale, v_scale [num_pages][kv_heads] fp32, powers of two (or 0 for a
 *     page of zeros); a value is e4m3(code) * scale
 *   block_table [batch] rows of max_pages int32, table_stride apart: page j of
 *     sequence b holds its tokens j * page_size and on. An entry outside
 *     [0, num_pages) means that the page is absent.
 *   seq_lens [batch] int32: tokens of each sequence, those of the current
 *     call's queries / new tokens included
 * The struct is host memory, read during the call only. head_dim 64, 128 or
 * 256; page_size 16, 32, 64, 128 or 256; 1 <= kv_heads <= 1024, num_pages >= 1
 * (< 2^31), 0 <= batch <= 65536, max_pages >= 1, table_stride >= max_pages
 * (< 2^40), max_pages * page_size < 2^31 - 1024. k and v 16-byte aligned, the
 * others 4-byte. 0 <= T <= 2^30 and at most 65535 query heads; a call whose
 * work does not fit one launch is refused (BSQ_ERR_SHAPE): append from
 * (T / page_size + 2 batch) * kv_heads = 2^23 on (+ T with queries), attention from
 * (T * q_heads / kv_heads / 128 + batch) * kv_heads = 2^23 or
 * batch * (max_pages * page_size / 64 + 1) = 2^31 on.
 *
 * The tokens of a call are packed: sequence b's are rows cu_seqlens[b] to
 * cu_seqlens[b + 1] - 1 of a [T] tensor (int32 [batch + 1] device, starting at
 * 0 and not decreasing), and they are its last ones: row cu_seqlens[b] + i has
 * position seq_lens[b] - n_b + i, n_b = cu_seqlens[b + 1] - cu_seqlens[b]. Rows
 * from cu_seqlens[batch] on belong to no sequence: not written, and without effect.
 * Where cu_seqlens decreases or leaves [0, T], which rows and pages of the call's
 * tensors are read and written, and with what, is not defined.
 */
typedef struct {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  const int32_t* block_table;
  const int32_t* seq_lens;
  int64_t num_pages, kv_heads, page_size, head_dim;
  int64_t batch, max_pages, table_stride;
} bsq_kv8_cache;

/*
 * Append a call's new keys and values to the cache, the keys rotated on the
 * way (and, on request, the queries too, into q_out). For each page and kv
 * head that receives tokens, for K and V each:
 *   a = the largest finite magnitude among the new values of the page (keys
 *     after the rotation, which for keys is done in 64 bits), e = the least exponent with a <= 448 * 2^e
 *     (2^e >= 2^-126; a = 0 counts as scale 0),
 *   scale = max(2^e, the scale before if the page already holds tokens of the
 *     sequence), so that a first token starts its page anew,
 *   codes already there become E4M3(value * scale before / scale) (exact
 *     except where they fall below E4M3's normal range), the new ones
 *     E4M3(value / scale), rounded to nearest even, saturating at +-448.
 * NaN stays NaN and infinities saturate (at 0 where the page's scale is 0). Appending again with the same
 * arguments changes nothing. Codes behind the last token are left as they are.
 *   k, v [T][kv_heads][head_dim], q, q_out [T][q_heads][head_dim] of `dtype`
 *     (BSQ_BF16 or BSQ_FP16): 16-byte aligned, strides in elements, multiples
 *     of 8 (0 <= stride < 2^40). q may be NULL (q_out NULL, q_heads 0); q_out
 *     may be q with the same strides, and its rows must not overlap.
 *   inv_freq [rot_dim / 2], layout, attn_factor: as bsq_rope with the rows'
 *     positions; rot_dim a multiple of 16 up to head_dim, or 0 (inv_freq NULL):
 *     nothing is rotated and q_out is a copy.
 * A sequence with seq_lens[b] < n_b is skipped, and so are tokens whose page is
 * absent or lies past max_pages. A page that receives tokens must be in one
 * sequence's table only, and once (two writers of one page race: its codes and
 * scales are then either's).
 */
bsq_status bsq_kv_append(bsq_dtype dtype, const bsq_kv8_cache* cache, const int32_t* cu_seqlens, int64_t T,
                         const void* k, int64_t k_stride_t, int64_t k_stride_h, const void* v, int64_t v_stride_t,
                         int64_t v_stride_h, const float* inv_freq, int64_t rot_dim, bsq_rope_layout layout,
                         float attn_factor, const void* q, int64_t q_stride_t, int64_t q_stride_h, int64_t q_heads,
                         void* q_out, int64_t o_stride_t, int64_t o_stride_h, hipStream_t stream);

/*
 * Attention of a call's queries over the cache. Row (t, h) attends with kv
 * head h / (q_heads / kv_heads); its position is p (above), and it sees the
 * tokens j < seq_lens[b] with j <= p (unless BSQ_ATTN_FULL is set) and, with
 * window > 0, j > p - window, whose page is present:
 *   y[t][h] = sum_j softmax_j(softmax_scale * q . k_j) v_j,
 *   lse[t][h] = log sum_j exp(softmax_scale * q . k_j).
 * A row that sees nothing gets y = 0 and lse = -inf. What a row does not see
 * does not reach it, be it NaN or beyond the range of `dtype`. Scores, the
 * running maximum and sum and the output are held in fp32. V's codes enter the
 * second product as they are, and each token's weight, its probability times its
 * page's scale, as the sum of two fp16 numbers with an exponent of the row's own:
 * 21 bits, fewer where that would be below 2^-35 of the row's largest weight.
 * (The V scales of pages that one call sees may be up to 2^90 apart.)
 *   q, y [T][q_heads][head_dim] of `dtype` (BSQ_BF16 or BSQ_FP16): 16-byte
 *     aligned, strides multiples of 8 (0 <= stride < 2^40), y's rows must not
 *     overlap; lse [T][q_heads] fp32 or NULL
 *   max_q_len: at least the largest n_b (1 for a decode step; T always does);
 *     of a longer sequence only rows up to max_q_len are written
 *   window >= 0; BSQ_ERR_ARG for a window with BSQ_ATTN_FULL, an unknown flag
 *     or a softmax_scale that is not finite, also times log2(e) (in fp32)
 * A sequence with seq_lens[b] < n_b has negative positions: those rows see
 * nothing (with BSQ_ATTN_FULL they see all). Tokens past max_pages count as
 * absent. The scales of pages that a row sees have to be what bsq_kv_append
 * writes, powers of two or 0; those of other pages may be anything.
 * Workspace: bsq_attention_kv8_workspace_bytes(...) bytes, 256-byte aligned, not
 * shared by calls that may overlap: partial results of sequences that are
 * split over workgroups; nothing in it needs clearing or survives the call.
 */
#define BSQ_ATTN_FULL 0x1u
size_t bsq_attention_kv8_workspace_bytes(int64_t batch, int64_t T, int64_t max_q_len, int64_t q_heads,
                                         int64_t kv_heads, int64_t head_dim);
bsq_status bsq_attention_kv8(bsq_dtype dtype, const bsq_kv8_cache* cache, const int32_t* cu_seqlens, int64_t T,
                             int64_t max_q_len, const void* q, int64_t q_stride_t, int64_t q_stride_h,
                             int64_t q_heads, float softmax_scale, int64_t window, uint32_t flags, void* y,
                             int64_t y_stride_t, int64_t y_stride_h, float* lse, void* workspace,
                             size_t workspace_bytes, hipStream_t stream);

/*
 * Weight-only linear with 4-bit integer weights and group scales, for a few
 * tokens (a decode step; any M is correct, weights are read once per 64
 * tokens):
 *   y[m][n] = sum_k x[m][k] * w_scale[n][k / group] * (c[n][k] - z[n][k / group])
 * with codes c in 0..15 and zero points z (8 where w_zero is NULL). Products
 * and sums are fp32 (a group's integer products are exact), rounded once.
 *   x [M][ldx], y [M][ldy] of `dtype` (BSQ_BF16 or BSQ_FP16)
 *   w [N][K/2], element 2j in the low nibble of byte j
 *   w_scale [N][K/group] of `dtype`; w_zero [N][K/group] uint8 (0..255) or NULL
 * group 32, 64 or 128, K % group == 0; M <= 2^20 - 16, N <= 2^27 - 16, K <= 2^20; shape,
 * ld and alignment rules of bsq.h (w_scale 2-byte, w_zero 1-byte aligned). Sums
 * are of x c (BSQ_BF16: of x (c + 128), which x (z + 128) is taken from), so
 * they must not leave fp32's range: with |x| below 2^90 none does.
 */
bsq_status bsq_gemm_int4g(bsq_dtype dtype, const void* x, int64_t ldx, const uint8_t* w, const void* w_scale,
                          const uint8_t* w_zero, int64_t group, void* y, int64_t ldy, int64_t M, int64_t N,
                          int64_t K, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* BSQ_SERVE_H */
