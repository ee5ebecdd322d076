// What the attention kernels over the paged E4M3 cache share: arguments, the rows' masks, the tile of 64
// tokens in LDS and its loads, and the treatment of what a row must not see.
#pragma once

#include "bsq_launch.hpp"
#include "serve_device.hpp"

namespace bsq {
namespace attn {

using kv::Cache;

struct Args {
  Cache c;
  const int32_t* cu;
  int64_t T;
  const uint16_t* q;
  uint16_t* y;
  float* lse;
  int64_t qt, qh, yt, yh;
  int q_heads, group;
  uint32_t group_inverse;  // kv::inverse_of(group)
  float scale2;  // |softmax_scale| * log2(e)
  int64_t window;
  bool full;
  int sign;             // of softmax_scale, -1 or 1: q enters with it, scale2 is the magnitude
  int max_q_len;
  int small;            // most rows (tokens times group) of a sequence that the step kernel takes
  int target, least;    // step kernel: pieces of all sequences together; least tiles of a piece, or of a prompt block's part
  int splits;           // prompt kernel: parts that a block's tokens are cut into
  float* part_o;        // partial results: step [piece][kv head][16][D], prompt [block][kv head][split][128][D]
  float* part_ml;       // their maxima (of scores times log2 e) and sums [...][2]
};

constexpr float kLn2 = 0.693147180559945309f;
constexpr int kLag = 4, kLift = 11;  // of the weights of the second product (below)

__device__ __forceinline__ int room_of(const Cache& c) { return c.max_pages << c.shift; }

// row R (token R / group, query head R % group) of a sequence of n rows and what it sees
struct Row {
  int i;           // token of the sequence's n, -1 for none
  int head;        // query head
  int lo, hi;      // tokens seen
};
// (`few`: R below 16, divided by a multiplication)
__device__ __forceinline__ Row row_at(const Args& a, int R, int kvh, int n, int len, int room, bool few = false) {
  const kv::RowPlace at = kv::row_place(R, a.group, few ? a.group_inverse : 0u, kvh, n, a.max_q_len);
  Row r;
  r.i = at.i;
  r.head = at.head;
  if (r.i < 0) {
    r.lo = 0;
    r.hi = 0x7FFFFFFF;  // (computed, never stored: it must not ask for a mask)
    return r;
  }
  const int64_t pos = (int64_t)len - n + r.i;
  int64_t hi = a.full ? len : pos + 1;
  hi = hi > len ? len : hi;
  hi = hi > room ? room : hi;
  r.hi = hi < 0 ? 0 : (int)hi;
  const int64_t lo = a.window > 0 ? pos - a.window + 1 : 0;
  r.lo = lo < 0 ? 0 : (lo > 0x7FFFFFFF ? 0x7FFFFFFF : (int)lo);
  return r;
}
// bytes [lo, hi) of the 16 of a lane's granule stay, the others become 0
__device__ __forceinline__ uint32_t byte_mask(int lo, int hi) {
  lo = lo < 0 ? 0 : (lo > 4 ? 4 : lo);
  hi = hi < 0 ? 0 : (hi > 4 ? 4 : hi);
  const uint32_t up = hi == 4 ? 0xFFFFFFFFu : (1u << (8 * hi)) - 1u;
  const uint32_t below = lo == 4 ? 0xFFFFFFFFu : (1u << (8 * lo)) - 1u;
  return up & ~below;
}
// 0x80 in every byte of w that is a NaN code
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// the 64 tokens' bits of one element
__device__ __forceinline__ unsigned long long nan_map(const uint16_t* p) {
  return (unsigned long long)p[0] | (unsigned long long)p[1] << 16 | (unsigned long long)p[2] << 32 |
         (unsigned long long)p[3] << 48;
}

template <class E>
union Frag {  // an MFMA operand of eight 16-bit values
  typename E::vec8 v;
  typename E::vec2 p[4];
  uint32_t u[4];
  uint4 q;
};
// eight E4M3 codes times 2^exponent(scale)
template <class E>
__device__ __forceinline__ typename E::vec8 dec8(uint32_t lo, uint32_t hi, float scale) {
  Frag<E> f;
  f.p[0] = E::template dec<false>(lo, scale);
  f.p[1] = E::template dec<true>(lo, scale);
  f.p[2] = E::template dec<false>(hi, scale);
  f.p[3] = E::template dec<true>(hi, scale);
  return f.v;
}

// ---- a tile of 64 tokens in LDS (layout: kv_index.hpp) -------------------------------------
constexpr int tile_bytes(int D) { return 128 * D; }  // K, then V
constexpr int tile_loads(int D) { return D / 8; }    // of 1 KB

// 16 bytes a lane from `p` to LDS at `lds` + 16 lane. Inline assembly, so that the compiler does not
// make every LDS read wait for it; callers wait (wait_loads) before they read. (One wait state
// between the write of M0 and its use.) `once`: codes that nobody reads again, with the non-temporal hint (64
// sequences of 4000 to 8000 tokens, 773 MB: 158 us a call with it, 166 without).
template <bool once>
__device__ __forceinline__ void load_to_lds(const uint8_t* p, uint32_t lds) {
  if constexpr (once) asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off nt" ::"v"(p), "{m0}"(lds) : "memory");
  else asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(p), "{m0}"(lds) : "memory");
}
template <int n>
__device__ __forceinline__ void wait_loads() {  // until at most n vector-memory operations are outstanding
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(n) : "memory");
}

// until the wave's own LDS reads have returned (before loads that write where it has read)
__device__ __forceinline__ void wait_reads() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

// The granules of up to 16 tiles of a wave, lane l's granule l % 4 of tile l / 4: whether its page is present, where
// its codes begin and their scales. An absent page's place is taken by page 0's, whose codes are hidden.
//
// V's scale, a power of two, does not enter the conversion of its codes (448 * 2^8 is an infinity in fp16, and would
// reach rows that give it no weight), but the exponent of the probabilities, relative to a reference of the wave.
struct Pages {
  int absent;  // -1: the page is absent, 0
  uint32_t k_lo, k_hi, v_lo, v_hi;
  float ks;
  int vs;       // settled: the exponent of V's scale less the reference's
  int ref = 0;  // the reference, a biased exponent: the largest of the first pages that are not all zeros
  // tile i starts at token t0 + stride * i; granules that lie before `begin`, or from `end` on, are not looked up: no
  // row sees them, and what an unused page happens to hold as its scales must not become the reference
  template <int D>
  __device__ __forceinline__ void load(const Cache& c, int b, int head, int t0, int stride, int begin, int end) {
    const int lane = threadIdx.x & 63;
    const int64_t t = (int64_t)t0 + (int64_t)stride * (lane >> 2) + 16 * (lane & 3);
    const int id = t + 16 > begin && t < end ? kv::page_of(c, b, (int)t) : -1;
    absent = id >> 31;
    const int64_t at = (int64_t)(id < 0 ? 0 : id) * c.heads + head, codes = (at << c.shift) * D;
    const int in = (int)t & ((1 << c.shift) - 1);
    ks = c.ks[at];
    vs = __float_as_int(c.vs[at]);
    const int64_t k = codes + in * D, v = codes + in;
    k_lo = (uint32_t)k;
    k_hi = (uint32_t)(k >> 32);
    v_lo = (uint32_t)v;
    v_hi = (uint32_t)(v >> 32);
  }
  // Makes `vs` of the scale that load() brought (apart, so that the tile's loads need not wait for it). A page of zeros
  // may have any exponent: the reference's while there is none, and then a low one, so that it does not outweigh small values
  // in rows that do not see the page that set the reference, but not so low that its tokens leave the sum or that
  // sum, times 2^90, fp32.
  __device__ __forceinline__ void settle() {
    int e = vs >> 23 & 0xFF;
    e = absent || e == 0xFF ? 0 : e;
    if (ref == 0) ref = __builtin_amdgcn_readfirstlane((int)wave_max((float)e));
    vs = e == 0 ? (ref == 0 ? 0 : -90) : e - ref;
  }
  static __device__ __forceinline__ int place(int tile, int gran) { return (tile & 15) * 4 + gran; }
  __device__ __forceinline__ int gone(int tile, int gran) const { return __shfl(absent, place(tile, gran), 64); }
  __device__ __forceinline__ float kscale(int tile, int gran) const { return __shfl(ks, place(tile, gran), 64); }
  __device__ __forceinline__ int vshift(int tile, int gran) const { return __shfl(vs, place(tile, gran), 64); }
  __device__ __forceinline__ float unit() const {  // of the accumulators: the reference, less the weights' factor
    return __uint_as_float((uint32_t)ref << 23) * (1.0f / (1 << kLift));
  }
};

// Issues loads [first, last) of a tile (its number `tile` in `pages`) into LDS at `lds`.
template <int D, kv::Kind kind>
struct TileLoads {
  int k_lane[D / 64];  // granule 0's offsets; another granule exchanges pieces: an exclusive or
  int v_gran, v_col;
  __device__ __forceinline__ TileLoads(const Cache& c) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) k_lane[i] = kv::k_source<D, kind>(i, 0, lane);
    const kv::VSource v = kv::v_source(lane, kv::v_run(c.shift));
    v_gran = v.gran;
    v_col = v.col;
  }
  template <int first, int last>
  __device__ __forceinline__ void issue(const Cache& c, const Pages& pages, int tile, uint32_t lds) const {
    if constexpr (first < D / 16) {
#pragma unroll
      for (int gran = first / (D / 64); gran * (D / 64) < last && gran < 4; ++gran) {
        const int at = Pages::place(tile, gran);
        const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)pages.k_lo, at);
        const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)pages.k_hi, at);
        const uint8_t* kp = c.k + ((int64_t)hi << 32 | lo);
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
          const int n = gran * (D / 64) + i;
          if (n >= first && n < last)
            load_to_lds<kind == kv::kStep>(kp + (k_lane[i] ^ (16 * kv::k_flip<D, kind>(16 * gran))), lds + 1024 * n);
        }
      }
    }
    if constexpr (last > D / 16) {
      const int at = Pages::place(tile, v_gran);
      const uint32_t lo = (uint32_t)__shfl((int)pages.v_lo, at, 64), hi = (uint32_t)__shfl((int)pages.v_hi, at, 64);
      const uint8_t* vp = c.v + ((int64_t)hi << 32 | lo) + (v_col << c.shift);
#pragma unroll
      for (int n = first > D / 16 ? first : D / 16; n < last; ++n)
        load_to_lds<kind == kv::kStep>(vp + ((n - D / 16) << (4 + c.shift)), lds + 1024 * n);
    }
  }
};

// Hides tokens of a lane's 16 V codes: bytes outside [lo, hi) become 0. NaN codes among the others become 0
// too and are returned as bits (a row that does not see such a token must not meet it as 0 * NaN).
__device__ __forceinline__ uint32_t hide_codes(v4u& w, int lo, int hi) {
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] &= byte_mask(lo - 4 * i, hi - 4 * i);
    const uint32_t nb = nan_bytes(w[i]);
    bits |= ((nb >> 7 & 1u) | (nb >> 14 & 2u) | (nb >> 21 & 4u) | (nb >> 28 & 8u)) << (4 * i);
    w[i] &= ~((nb >> 7) * 0xFFu);
  }
  return bits;
}
// the tokens of a tile at t0 that a row sees, as bits
__device__ __forceinline__ unsigned long long seen_bits(const Row& row, int t0) {
  const int lo = row.lo - t0, hi = row.hi - t0;
  unsigned long long s = ~0ull;
  if (lo > 0) s = lo >= 64 ? 0ull : s << lo;
  if (hi < 64) s = hi <= 0 ? 0ull : s & ((1ull << hi) - 1ull);
  return s;
}

// Weights w_j = 2^(x_j + v_j - N) enter the second product: x_j a score times log2 e, v_j the exponent of its V scale less the
// reference. N is a whole number, so that v_j and it are taken off together without a rounding, and what is summed up is
// rescaled exactly. It may lag behind the largest x + v by 2^4, in which most tiles need no rescaling; weights are
// lifted by 2^11 and then at most 2^15, and the largest of a row is above 2^10. Each enters as the sum of two fp16
// numbers (21 bits; what is below 2^-35 of the row's largest weight is lost), so that y is as exact as with weights in
// fp32: with one of 11 bits its error against 64 bits grew from 0.00021 to 0.00031 for fp16 tensors over 130 000 tokens, and
// results in bf16 were rounded the other way here and there. The sum of the probabilities takes w_j 2^-v_j.
__device__ __forceinline__ bool outgrown(float top, float n) { return top > n + (float)kLag; }
// (a row that has seen nothing has -inf: its weights exp2(-inf - 0) are 0)
__device__ __forceinline__ float finite_base(float m) { return m == -INFINITY ? 0.0f : m; }
// from 2^22 on N and v_j are not taken off together: a step of fp32 might be more than v_j
__device__ __forceinline__ bool coarse(float n) { return fabsf(n) >= 4194304.0f && n != -INFINITY; }

// x - n, in that case, at most what keeps the weight within fp16 (NaN stays)
__device__ __forceinline__ float coarse_score(float d, int vs) { return d > (float)(kLag - vs) ? (float)(kLag - vs) : d; }

// two weights as the sum of two fp16 numbers each: the first rounded towards zero, what is left of it rounded to nearest
__device__ __forceinline__ void two_parts(float a, float b, uint32_t& first, uint32_t& rest) {
  union { decltype(__builtin_amdgcn_cvt_pkrtz(0.0f, 0.0f)) p; v2h h; uint32_t u; } f, r;
  float one = 1.0f;  // (from a register: with the constant the multiplication goes, and with it the one instruction that
  asm("" : "+s"(one));  // takes fp32 and fp16 operands to an fp16 result)
  f.p = __builtin_amdgcn_cvt_pkrtz(a, b);
  r.h = v2h{(_Float16)__builtin_fmaf(a, one, -(float)f.h[0]), (_Float16)__builtin_fmaf(b, one, -(float)f.h[1])};
  first = f.u;
  rest = r.u;
}

// eight query values with the softmax scale's sign
__device__ __forceinline__ uint4 signed_query(uint4 q, int sign) {
  const uint32_t flip = sign < 0 ? 0x80008000u : 0u;
  return make_uint4(q.x ^ flip, q.y ^ flip, q.z ^ flip, q.w ^ flip);
}

}  // namespace attn

// the prompt kernel (kv_prompt.hip): sequences of more than `a.small` rows; blocks of 128 rows
hipError_t launch_attn_prompt(bsq_dtype dt, const attn::Args& a, hipStream_t s);

}  // namespace bsq
