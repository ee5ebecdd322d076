// Appending keys (rotated) and values to the paged E4M3 cache, the queries rotated along.
//
// One workgroup takes one page and kv head that receives tokens: it is the only writer of that
// page's codes and scale, so the scale (a power of two over the largest magnitude) needs no atomics
// and the codes already there can be brought to a larger scale in place. Powers of two keep that
// exact except for codes that fall below E4M3's normal range, so a page filled token by token
// holds what it would hold if filled at once, up to those.
//
// Keys are rotated in 64 bits, so that next to a border between codes they fall on the right side.
//
// Bound by memory for prompts (2 bytes read and 1 written per element, the queries twice 2): 9000 tokens of 32 + 2 x 8
// heads of 128 in pages of 16, 214 MB, in 56 us, 3.8 TB/s (50 with angles and products in 32 bits, which
// put three times as many keys on the wrong side); and by the chain of dependent loads (row, length, page, scale,
// values) for a decode step: 96 tokens in 11 us (12.2 on average). What counted for the prompt: one wave to a token's queries with its
// loads on their way before the search for its sequence (-9 us), and the registers of a thread.
#include "serve_device.hpp"

namespace bsq {

namespace {

using kv::Cache;

struct Args {
  Cache c;
  const int32_t* cu;
  int64_t T;
  const uint16_t *k, *v, *q;
  int64_t kt, kh, vt, vh, qt, qh, ot, oh;
  uint16_t* qo;
  int q_heads;
  const float* inv_freq;
  int rot;
  float factor;
  uint64_t page_share;  // workgroups of pages in all, times 2^32, rounded up
};

// The last b in [0, batch) with at(b), -1 if none. 256 candidates a step, four independent loads to a lane: the
// search is part of a decode step's chain of dependent loads, and batches of up to 256 take one round trip.
template <class At>
__device__ __forceinline__ int last_sequence(int batch, At at) {
  const int lane = threadIdx.x & 63;
  return __builtin_amdgcn_readfirstlane(kv::last_of<256>(batch, [&](int lo, int step, int n) {
    int cnt = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = (lane + 64 * j) * step;
      cnt += __popcll(__ballot(i < n && at(lo + (i < n ? i : 0))));
    }
    return cnt;
  }));
}

// Elements of unit u (16 of a head's D): two pieces of eight, from e0 and e1 on, and whether they are rotated.
// In either layout the pieces of consecutive units follow each other, so that a wave's accesses fill lines: the
// first half of the rotated elements and the second, the first half of the rest and the second.
template <int D>
__device__ __forceinline__ bool unit_places(int u, int rot, int& e0, int& e1) {
  const bool turned = 16 * u < rot;
  e0 = turned ? 8 * u : (rot >> 1) + 8 * u;
  e1 = e0 + ((turned ? rot : D - rot) >> 1);
  return turned;
}
// rotates a unit by `rotate(pair, x0, x1)`: its pairs are one element of either piece (at pair e0 + j), or neighbours
// in a piece
template <bool INTER, class Rotate>
__device__ __forceinline__ void turn(float (&p)[8], float (&q)[8], int e0, int e1, Rotate rotate) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float& a = INTER ? (j < 4 ? p[(2 * j) & 7] : q[(2 * j) & 7]) : p[j];
    float& b = INTER ? (j < 4 ? p[(2 * j + 1) & 7] : q[(2 * j + 1) & 7]) : q[j];
    rotate(!INTER ? e0 + j : (j < 4 ? (e0 >> 1) + j : (e1 >> 1) + j - 4), a, b);
  }
}

__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a <= 3.40282347e38f ? a : 0.0f;  // NaN and infinities do not enter the scale
}
// the least power of two s >= 2^-126 with a <= 448 s; 0 for a = 0
__device__ __forceinline__ float scale_for(float a) {
  if (!(a > 0.0f)) return 0.0f;
  const uint32_t bits = __float_as_uint(a);
  // a = m 2^e, 1 <= m < 2; 448 = 1.75 2^8 (a subnormal a has e below -126, the floor catches it)
  int e = (int)(bits >> 23) - 127 - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = e < -126 ? -126 : e;
  return __uint_as_float((uint32_t)(e + 127) << 23);
}
// E4M3 code of x * r: NaN stays NaN, everything else saturates (r = 0 gives 0)
__device__ __forceinline__ float ready(float x, float r) {
  const float v = __builtin_amdgcn_fmed3f(x, -3.40282347e38f, 3.40282347e38f) * r;
  return x != x ? x : __builtin_amdgcn_fmed3f(v, -kE4M3Max, kE4M3Max);
}
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float r) {
  const uint32_t w = __builtin_amdgcn_cvt_pk_fp8_f32(ready(a, r), ready(b, r), 0u, false);
  return __builtin_amdgcn_cvt_pk_fp8_f32(ready(c, r), ready(d, r), w, true);
}
// the four codes of w at `ratio` (a power of two) times their values
__device__ __forceinline__ uint32_t recode4(uint32_t w, float ratio) {
  return encode4(dec_e4m3<0>(w), dec_e4m3<1>(w), dec_e4m3<2>(w), dec_e4m3<3>(w), ratio);
}

// largest magnitude over the workgroup, of K and of V
__device__ __forceinline__ void block_max2(float& x, float& y) {
  __shared__ float red[8];
  x = wave_max(x);
  y = wave_max(y);
  if ((threadIdx.x & 63) == 0) {
    red[threadIdx.x >> 6] = x;
    red[4 + (threadIdx.x >> 6)] = y;
  }
  __syncthreads();
  x = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  y = fmaxf(fmaxf(red[4], red[5]), fmaxf(red[6], red[7]));
}

// KEEP: units of K that a thread keeps between the two passes over them; larger pages are read and turned twice.
template <class E, int D, bool INTER, int KEEP>
__device__ __forceinline__ void append_page(const Args& a, int64_t slot, int head) {
  const int b = last_sequence(a.c.batch, [&](int i) { return kv::first_slot(a.cu, i, a.T, a.c.shift) <= slot; });
  if (b < 0) return;
  const kv::Touched tp = kv::touched_page(a.c, a.cu, b, slot - kv::first_slot(a.cu, b, a.T, a.c.shift), a.T);
  if (tp.n == 0) return;
  const int tid = threadIdx.x, ps = 1 << a.c.shift;
  const uint16_t* kr = a.k + (int64_t)tp.row * a.kt + (int64_t)head * a.kh;
  const uint16_t* vr = a.v + (int64_t)tp.row * a.vt + (int64_t)head * a.vh;
  // position of the first new token: tokens before it are the sequence's length less its rows
  const kv::Rows rows = kv::rows_of(a.cu, b, a.T);
  const int pos0 = a.c.lens[b] - rows.n + (tp.row - rows.first);

  constexpr int U = D / 16;
  const int kunits = tp.n * U;
  auto load_key = [&](int i, float(&p)[8], float(&q)[8]) {
    const int t = i / U, u = i % U;
    int e0, e1;
    const bool turned = unit_places<D>(u, a.rot, e0, e1);
    load8<E>(kr + (int64_t)t * a.kt + e0, p);
    load8<E>(kr + (int64_t)t * a.kt + e1, q);
    if (turned)
      turn<INTER>(p, q, e0, e1, [&](int i, float& x0, float& x1) {
        // in 64 bits: among millions of keys some lie next to a border between codes, and a value off by
        // 2^-22 falls on its wrong side three times as often as correctly rounded products do
        const Turn v = rope_turn((double)(pos0 + t), a.inv_freq[i], a.factor);
        const double u0 = (double)x0, u1 = (double)x1;
        x0 = to_odd(fma(u0, v.c, -(u1 * v.s)));
        x1 = to_odd(fma(u1, v.c, u0 * v.s));
      });
  };
  float kmax = 0.0f, vmax = 0.0f;
  float keep[KEEP][2][8];
  auto key_max = [&](float(&p)[8], float(&q)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) kmax = fmaxf(kmax, fmaxf(finite_abs(p[j]), finite_abs(q[j])));
  };
#pragma unroll
  for (int s = 0; s < KEEP; ++s) {
    const int i = tid + 256 * s;
    if (i < kunits) {
      load_key(i, keep[s][0], keep[s][1]);
      key_max(keep[s][0], keep[s][1]);
    }
  }
  for (int i = tid + 256 * KEEP; i < kunits; i += 256) {
    float p[8], q[8];
    load_key(i, p, q);
    key_max(p, q);
  }

  // V: two elements of 16 tokens a unit, so that a thread holds whole 16-byte pieces of the
  // cache's rows (tokens contiguous); the first unit is kept between the passes. Dealt from the last wave on:
  // a small page's keys are with the first ones.
  const int vtid = tid ^ 192;
  const int g0 = tp.at >> 4, g1 = (tp.at + tp.n + 15) >> 4;  // granules of 16 tokens that receive some
  const int vunits = (g1 - g0) * (D / 2);
  uint32_t vkeep[16];
  auto load_values = [&](int i, uint32_t(&w)[16]) {
    const int g = g0 + i / (D / 2), d = 2 * (i % (D / 2));
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int t = 16 * g + j - tp.at;
      w[j] = t >= 0 && t < tp.n ? *reinterpret_cast<const uint32_t*>(vr + (int64_t)t * a.vt + d) : 0u;
    }
  };
  auto value_max = [&](const uint32_t(&w)[16]) {
#pragma unroll
    for (int j = 0; j < 16; ++j) vmax = fmaxf(vmax, fmaxf(finite_abs(E::lo(w[j])), finite_abs(E::hi(w[j]))));
  };
  if (vtid < vunits) {
    load_values(vtid, vkeep);
    value_max(vkeep);
  }
  for (int i = vtid + 256; i < vunits; i += 256) {
    uint32_t w[16];
    load_values(i, w);
    value_max(w);
  }

  if (tp.page < 0) return;  // (asked only here: the values need not wait for the table)
  const int64_t codes = kv::codes_at(a.c, tp.page, head);
  uint8_t* kp = a.c.k + codes;
  uint8_t* vp = a.c.v + codes;
  const int64_t sc = (int64_t)tp.page * a.c.heads + head;
  const float ks0 = tp.at > 0 ? a.c.ks[sc] : 0.0f, vs0 = tp.at > 0 ? a.c.vs[sc] : 0.0f;
  block_max2(kmax, vmax);
  const float ks = fmaxf(scale_for(kmax), ks0), vs = fmaxf(scale_for(vmax), vs0);
  const float kinv = ks > 0.0f ? 1.0f / ks : 0.0f, vinv = vs > 0.0f ? 1.0f / vs : 0.0f;
  // codes already there, at the larger scale; dwords of V that also hold new tokens' places keep
  // those bytes, which are written after the barrier
  if (ks != ks0 && tp.at > 0) {
    uint32_t* w = reinterpret_cast<uint32_t*>(kp);
    for (int i = tid; i < tp.at * (D / 4); i += 256) w[i] = recode4(w[i], ks0 * kinv);
  }
  if (vs != vs0 && tp.at > 0) {
    const int words = (tp.at + 3) >> 2;
    for (int i = tid; i < words * D; i += 256) {
      const int d = i / words, wd = i - d * words;
      uint32_t* w = reinterpret_cast<uint32_t*>(vp + (int64_t)d * ps) + wd;
      const int left = tp.at - 4 * wd;  // old tokens of this dword
      const uint32_t mask = left >= 4 ? 0xFFFFFFFFu : (1u << (8 * left)) - 1u;
      const uint32_t old = *w;
      *w = (recode4(old, vs0 * vinv) & mask) | (old & ~mask);
    }
  }
  __syncthreads();
  if (tid == 0) {
    a.c.ks[sc] = ks;
    a.c.vs[sc] = vs;
  }

  auto store_key = [&](int i, float(&p)[8], float(&q)[8]) {
    const int t = i / U, u = i % U;
    int e0, e1;
    unit_places<D>(u, a.rot, e0, e1);
    uint8_t* row = kp + (int64_t)(tp.at + t) * D;
    *reinterpret_cast<uint2*>(row + e0) =
        make_uint2(encode4(p[0], p[1], p[2], p[3], kinv), encode4(p[4], p[5], p[6], p[7], kinv));
    *reinterpret_cast<uint2*>(row + e1) =
        make_uint2(encode4(q[0], q[1], q[2], q[3], kinv), encode4(q[4], q[5], q[6], q[7], kinv));
  };
#pragma unroll
  for (int s = 0; s < KEEP; ++s) {
    const int i = tid + 256 * s;
    if (i < kunits) store_key(i, keep[s][0], keep[s][1]);
  }
  for (int i = tid + 256 * KEEP; i < kunits; i += 256) {
    float p[8], q[8];
    load_key(i, p, q);
    store_key(i, p, q);
  }

  auto store_values = [&](int i, const uint32_t(&w)[16]) {
    const int g = g0 + i / (D / 2), d = 2 * (i % (D / 2));
    const int lo = tp.at - 16 * g, hi = tp.at + tp.n - 16 * g;  // this granule's new tokens
    uint32_t c0[4], c1[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      c0[j] = encode4(E::lo(w[4 * j]), E::lo(w[4 * j + 1]), E::lo(w[4 * j + 2]), E::lo(w[4 * j + 3]), vinv);
      c1[j] = encode4(E::hi(w[4 * j]), E::hi(w[4 * j + 1]), E::hi(w[4 * j + 2]), E::hi(w[4 * j + 3]), vinv);
    }
    uint8_t* row = vp + (int64_t)d * ps + 16 * g;
    if (lo <= 0 && hi >= 16) {
      *reinterpret_cast<uint4*>(row) = make_uint4(c0[0], c0[1], c0[2], c0[3]);
      *reinterpret_cast<uint4*>(row + ps) = make_uint4(c1[0], c1[1], c1[2], c1[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        if (j >= lo && j < hi) {
          row[j] = (uint8_t)(c0[j >> 2] >> (8 * (j & 3)));
          row[ps + j] = (uint8_t)(c1[j >> 2] >> (8 * (j & 3)));
        }
      }
    }
  };
  if (vtid < vunits) store_values(vtid, vkeep);
  for (int i = vtid + 256; i < vunits; i += 256) {
    uint32_t w[16];
    load_values(i, w);
    store_values(i, w);
  }
}

// One token's queries, by one wave: its angles once into LDS, then 16 elements a lane and step, the first steps'
// values on their way before the token's place is known.
constexpr int kAhead = 4;
template <class E, int D, bool INTER>
__device__ __forceinline__ void turn_queries(const Args& a, int64_t t) {
  __shared__ float2 angles[4][D / 2];
  float2* cs = angles[threadIdx.x >> 6];
  if (t >= a.T) return;
  const int lane = threadIdx.x & 63;
  const uint16_t* qr = a.q + t * a.qt;
  uint16_t* orow = a.qo + t * a.ot;
  constexpr int U = D / 16;
  const int units = a.q_heads * U;
  uint4 ahead[kAhead][2];
#pragma unroll
  for (int s = 0; s < kAhead; ++s) {
    const int x = lane + 64 * s;
    int e0, e1;
    unit_places<D>(x % U, a.rot, e0, e1);
    const uint16_t* src = qr + (int64_t)(x / U) * a.qh;
    if (x < units) {
      ahead[s][0] = *reinterpret_cast<const uint4*>(src + e0);
      ahead[s][1] = *reinterpret_cast<const uint4*>(src + e1);
    }
  }
  const int b = last_sequence(a.c.batch, [&](int i) { return a.cu[i] <= (int)t; });
  if (b < 0) return;
  const kv::Rows r = kv::rows_of(a.cu, b, a.T);
  const int i = (int)t - r.first;
  if (i < 0 || i >= r.n) return;  // a row of no sequence
  const int past = a.c.lens[b] - r.n;
  if (past < 0) return;
  for (int p = lane; p < (a.rot >> 1); p += 64) cs[p] = rope_angle((double)(past + i), a.inv_freq[p], a.factor);
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  auto finish = [&](int x, uint4 v0, uint4 v1) __attribute__((always_inline)) {
    const int h = x / U;
    int e0, e1;
    const bool turned = unit_places<D>(x % U, a.rot, e0, e1);
    float p[8], q[8];
    unpack8<E>(v0, p);
    unpack8<E>(v1, q);
    if (turned)
      turn<INTER>(p, q, e0, e1, [&](int i, float& x0, float& x1) {
        const float2 v = cs[i];
        const float u0 = x0, u1 = x1;
        x0 = u0 * v.x - u1 * v.y;
        x1 = u1 * v.x + u0 * v.y;
      });
    uint16_t* dst = orow + (int64_t)h * a.oh;
    store8<E>(dst + e0, p);
    store8<E>(dst + e1, q);
  };
#pragma unroll
  for (int s = 0; s < kAhead; ++s)
    if (lane + 64 * s < units) finish(lane + 64 * s, ahead[s][0], ahead[s][1]);
  for (int x = lane + 64 * kAhead; x < units; x += 64) {
    int e0, e1;
    unit_places<D>(x % U, a.rot, e0, e1);
    const uint16_t* src = qr + (int64_t)(x / U) * a.qh;
    finish(x, *reinterpret_cast<const uint4*>(src + e0), *reinterpret_cast<const uint4*>(src + e1));
  }
}

template <class E, int D, bool INTER, int KEEP>
__global__ __launch_bounds__(256) void kv_append_kernel(Args a) {
  // Workgroups that take a page's head lie evenly among those that take a token's queries: the ones wait for
  // memory, the others fill its bandwidth. `before`: how many of the first i take pages.
  const uint32_t id = blockIdx.x;
  const uint32_t before = (uint32_t)(id * a.page_share >> 32), then = (uint32_t)((id + 1) * a.page_share >> 32);
  if (then > before)
    append_page<E, D, INTER, KEEP>(a, before / (uint32_t)a.c.heads, (int)(before % (uint32_t)a.c.heads));
  else
    turn_queries<E, D, INTER>(a, 4 * (int64_t)(id - before) + (threadIdx.x >> 6));
}

template <class E, int D, bool INTER>
void launch_keep(const Args& a, unsigned blocks, hipStream_t s) {
  // a page of at most 256 units needs one kept; two are worth their registers above (64 tokens of 128 elements, 9000
  // tokens in all: 56 us with two, 62 with one; pages of 16, which never have a second: 56 with either)
  if (D / 16 << a.c.shift <= 256)
    hipLaunchKernelGGL((kv_append_kernel<E, D, INTER, 1>), dim3(blocks), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((kv_append_kernel<E, D, INTER, 2>), dim3(blocks), dim3(256), 0, s, a);
}
template <class E, int D>
hipError_t launch(const Args& a, bool inter, unsigned blocks, hipStream_t s) {
  if (inter) launch_keep<E, D, true>(a, blocks, s);
  else launch_keep<E, D, false>(a, blocks, s);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(bsq_dtype dt, const AppendArgs& p, hipStream_t s) {
  Args a{};
  a.c = p.c; a.cu = p.cu; a.T = p.T;
  a.k = static_cast<const uint16_t*>(p.k.p); a.kt = p.k.st; a.kh = p.k.sh;
  a.v = static_cast<const uint16_t*>(p.v.p); a.vt = p.v.st; a.vh = p.v.sh;
  a.q = static_cast<const uint16_t*>(p.q.p); a.qt = p.q.st; a.qh = p.q.sh;
  a.qo = static_cast<uint16_t*>(const_cast<void*>(p.qo.p)); a.ot = p.qo.st; a.oh = p.qo.sh;
  a.q_heads = p.q_heads;
  a.inv_freq = p.r.inv_freq; a.rot = p.r.rot; a.factor = p.r.factor;
  const int64_t pages = kv::append_slots(p.T, p.c.batch, p.c.shift) * p.c.heads;
  const int64_t blocks = pages + (p.q.p ? (p.T + 3) / 4 : 0);  // below 2^23
  a.page_share = (((uint64_t)pages << 32) + blocks - 1) / blocks;
  const bool inter = p.r.interleaved;
  const unsigned n = (unsigned)blocks;
  const bool half = dt == BSQ_FP16;
  switch (p.c.dim) {
    case 64: return half ? launch<Fp16, 64>(a, inter, n, s) : launch<Bf16, 64>(a, inter, n, s);
    case 128: return half ? launch<Fp16, 128>(a, inter, n, s) : launch<Bf16, 128>(a, inter, n, s);
    default: return half ? launch<Fp16, 256>(a, inter, n, s) : launch<Bf16, 256>(a, inter, n, s);
  }
}

}  // namespace bsq
