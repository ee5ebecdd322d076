// Attention over the paged E4M3 cache.
//
// step kernel: 16 rows (a token's queries of one kv head, or a few tokens') against a sequence's
// tokens, 64 a wave and step, one pass with the running maximum and sum of the softmax in fp32.
// S^T = K Q^T on 16x16x32 MFMA (rows: tokens, columns: query rows), then O^T += V^T P^T on the
// same. A lane of the first product's result holds column (query row) l % 16 and rows 4 (l / 16)
// + 0..3; row 4 g + r of K tile j is taken to be token 16 g + 4 j + r, so that over the four tiles
// a lane ends up with the 16 consecutive tokens of granule l / 16: one page, one scale of K and of V
// to a lane, and P in the order in which the second product wants its operand, without a shuffle
// or LDS. Codes go from memory to the operands in registers (V is stored tokens contiguous), 16
// bytes a lane and load; E4M3 becomes 16-bit exactly, two values an instruction.
//
// Bound by memory: 2 D bytes per token and kv head.
#include "bsq_launch.hpp"
#include "serve_device.hpp"

namespace bsq {

namespace {

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
  float scale2;  // softmax_scale * log2(e)
  int64_t window;
  bool full;
  int max_q_len, row_tiles;
  int target, least;  // pieces of all sequences together, least tiles of a piece
  float* part_o;      // [piece][kv head][row tile][16][D]
  float* part_ml;     // [piece][kv head][row tile][16][2]
};

constexpr float kLn2 = 0.693147180559945309f;

__device__ __forceinline__ int wave_sum(int v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}
__device__ __forceinline__ int wave_scan(int v) {  // inclusive
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(v, off, 64);
    if (lane >= off) v += o;
  }
  return v;
}

__device__ __forceinline__ int room_of(const Cache& c) { return c.max_pages << c.shift; }
// tiles of sequence b over all its rows; -1 for one without rows
__device__ __forceinline__ int sequence_tiles(const Args& a, int b) {
  const int n = kv::rows_of(a.cu, b, a.T).n;
  if (n == 0) return -1;
  const int len = a.c.lens[b];
  return kv::tiles_of(kv::seen_range(len < 0 ? 0 : len, room_of(a.c), n, 0, n, a.window, a.full));
}

// Which part of which sequence a workgroup takes. Every wave finds it by itself from the lengths:
// a sum over the sequences gives the piece size, a prefix sum of their pieces the sequence. So the
// host needs to know no length, and a batch of any raggedness is cut into equal pieces.
struct Piece {
  int b, index, count, first;  // first: number of the sequence's first piece
};
__device__ __forceinline__ int plan_chunk(const Args& a) {
  if (a.target <= 0) return 0x7FFFFFFF;
  const int lane = threadIdx.x & 63;
  int64_t total = 0;
  for (int b0 = 0; b0 < a.c.batch; b0 += 64) {
    const int t = b0 + lane < a.c.batch ? sequence_tiles(a, b0 + lane) : 0;
    total += wave_sum(t > 0 ? t : 0);
  }
  return kv::chunk_of(total, a.target, a.least);
}
__device__ __forceinline__ int piece_count(const Args& a, int b, int chunk) {
  const int t = sequence_tiles(a, b);
  return t < 0 ? 0 : kv::pieces_of(t, chunk);
}
__device__ __forceinline__ bool find_piece(const Args& a, int id, Piece& out) {
  const int lane = threadIdx.x & 63, chunk = plan_chunk(a);
  int before = 0;
  for (int b0 = 0; b0 < a.c.batch; b0 += 64) {
    const int n = b0 + lane < a.c.batch ? piece_count(a, b0 + lane, chunk) : 0;
    const int upto = before + wave_scan(n);
    const unsigned long long hit = __ballot(upto > id);
    if (hit) {
      const int at = __builtin_ctzll(hit);
      out.b = b0 + at;
      out.count = __shfl(n, at, 64);
      out.first = __shfl(upto - n, at, 64);
      out.index = id - out.first;
      return true;
    }
    before = __shfl(upto, 63, 64);
  }
  return false;
}

// rows [i0, ...) of a sequence as this wave's column l % 16 sees them
struct Row {
  int i;           // token of the sequence's n, -1 for none
  int head;        // query head
  int lo, hi;      // tokens seen
};
__device__ __forceinline__ Row row_at(const Args& a, int R, int kvh, int n, int len, int room) {
  Row r;
  r.i = R / a.group;
  r.head = kvh * a.group + (R - r.i * a.group);
  if (r.i >= n || r.i >= a.max_q_len) {
    r.i = -1;
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
__device__ __forceinline__ int wave_min16(int v) {  // over the 16 columns
#pragma unroll
  for (int off = 8; off >= 1; off >>= 1) {
    const int o = __shfl_xor(v, off, 64);
    v = o < v ? o : v;
  }
  return v;
}
__device__ __forceinline__ int wave_max16(int v) { return -wave_min16(-v); }

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
union Frag {
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

template <int D>
constexpr int step_lds() {  // four waves' results (rows padded), maxima and sums, NaN maps
  return 4 * 16 * (D + 4) * 4 + 4 * 16 * 2 * 4 + 4 * D * 8;
}

template <class E, int D>
__global__ __launch_bounds__(256, 2) void attn_step(Args a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  float* sh_o = reinterpret_cast<float*>(smem);                  // [4][16][D + 4]
  float* sh_ml = sh_o + 4 * 16 * (D + 4);                        // [4][16][2]
  uint16_t* sh_nan = reinterpret_cast<uint16_t*>(sh_ml + 4 * 16 * 2);  // [4][D][4 granules]
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, col = lane & 15, g = lane >> 4;
  const int kvh = blockIdx.y / a.row_tiles, rt = blockIdx.y % a.row_tiles;
  Piece pc;
  if (!find_piece(a, blockIdx.x, pc)) return;
  const int b = __builtin_amdgcn_readfirstlane(pc.b);
  const int pieces = __builtin_amdgcn_readfirstlane(pc.count);
  const kv::Rows rows = kv::rows_of(a.cu, b, a.T);
  if (rt * 16 >= rows.n * a.group) return;
  const int room = room_of(a.c);
  int len = a.c.lens[b];
  len = len < 0 ? 0 : len;
  const kv::Range all = kv::seen_range(len, room, rows.n, 0, rows.n, a.window, a.full);
  const int tiles = kv::tiles_of(all);
  const int index = __builtin_amdgcn_readfirstlane(pc.index);
  const int tile0 = kv::piece_begin(tiles, pieces, index), tile1 = kv::piece_begin(tiles, pieces, index + 1);

  const Row row = row_at(a, rt * 16 + col, kvh, rows.n, len, room);
  const int any_lo = wave_min16(row.i < 0 ? 0x7FFFFFFF : row.lo), any_hi = wave_max16(row.i < 0 ? 0 : row.hi);
  const int all_lo = wave_max16(row.i < 0 ? 0 : row.lo), all_hi = wave_min16(row.hi);

  Frag<E> q[D / 32];  // column col, elements 64 (s / 2) + 16 g + 8 (s % 2) + 0..7
  {
    const uint16_t* qr = a.q + (int64_t)(rows.first + (row.i < 0 ? 0 : row.i)) * a.qt + (int64_t)row.head * a.qh;
#pragma unroll
    for (int s = 0; s < D / 32; ++s)
      q[s].q = row.i < 0 ? make_uint4(0, 0, 0, 0)
                         : *reinterpret_cast<const uint4*>(qr + 64 * (s >> 1) + 16 * g + 8 * (s & 1));
  }

  v4f acc[D / 16];
#pragma unroll
  for (int i = 0; i < D / 16; ++i) acc[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  float m = -INFINITY, l = 0.0f;

  const int ps = 1 << a.c.shift;
  const int kg = col >> 2;  // granule of this lane's K rows
  for (int tile = tile0 + wave; tile < tile1; tile += 4) {
    const int t0 = all.lo + tile * kv::kTile;
    if (t0 >= any_hi || t0 + kv::kTile <= any_lo) continue;
    const int kt = t0 + 16 * kg, vt = t0 + 16 * g;
    const int kid = kt < any_hi ? kv::page_of(a.c, b, kt) : -1, vid = vt < any_hi ? kv::page_of(a.c, b, vt) : -1;
    // (an absent page's place is taken by page 0, whose codes are then hidden)
    const uint8_t* kp = a.c.k + kv::codes_at(a.c, kid < 0 ? 0 : kid, kvh) +
                        (int64_t)((kt & (ps - 1)) + (col & 3)) * D + 16 * g;
    const uint8_t* vp = a.c.v + kv::codes_at(a.c, vid < 0 ? 0 : vid, kvh) + (int64_t)col * ps + (vt & (ps - 1));
    uint4 kc[4][D / 64], vc[D / 16];
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < D / 64; ++i) kc[j][i] = *reinterpret_cast<const uint4*>(kp + 4 * j * D + 64 * i);
    const int64_t sc = (int64_t)(vid < 0 ? 0 : vid) * a.c.heads + kvh;
    const float ks = a.c.ks[sc] * a.scale2, vs = a.c.vs[sc];
#pragma unroll
    for (int i = 0; i < D / 16; ++i) vc[i] = *reinterpret_cast<const uint4*>(vp + (int64_t)16 * i * ps);

    float x[16];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v4f s = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        s = E::mfma(dec8<E>(kc[j][i].x, kc[j][i].y, 1.0f), q[2 * i].v, s);
        s = E::mfma(dec8<E>(kc[j][i].z, kc[j][i].w, 1.0f), q[2 * i + 1].v, s);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) x[4 * j + r] = s[r] * ks;
    }
    bool poisoned = false;  // a NaN code of V that some row sees and another does not
    const bool masked = t0 < all_lo || t0 + kv::kTile > all_hi || __ballot(vid < 0) != 0;
    if (masked) {
      const int lo = (vid < 0 ? 16 : row.lo - vt), hi = row.hi - vt;
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] = j >= lo && j < hi ? x[j] : -INFINITY;
      // V's codes that no row sees must not meet a probability of 0 as NaN
      const int vlo = vid < 0 ? 16 : any_lo - vt, vhi = any_hi - vt;
      const uint32_t k0 = byte_mask(vlo, vhi), k1 = byte_mask(vlo - 4, vhi - 4), k2 = byte_mask(vlo - 8, vhi - 8),
                     k3 = byte_mask(vlo - 12, vhi - 12);
      uint32_t bad = 0;
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        vc[i].x &= k0;
        vc[i].y &= k1;
        vc[i].z &= k2;
        vc[i].w &= k3;
        bad |= nan_bytes(vc[i].x) | nan_bytes(vc[i].y) | nan_bytes(vc[i].z) | nan_bytes(vc[i].w);
      }
      poisoned = __ballot(bad != 0) != 0 && (all_lo != any_lo || all_hi != any_hi);
      if (poisoned) {
        // which tokens of each element are NaN goes to LDS, the codes become 0; the rows that see
        // one get their NaN after the product
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          uint32_t bits = 0;
          uint32_t* w = reinterpret_cast<uint32_t*>(&vc[i]);
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            const uint32_t nb = nan_bytes(w[d]);
            bits |= (((nb >> 7) & 1u) | ((nb >> 14) & 2u) | ((nb >> 21) & 4u) | ((nb >> 28) & 8u)) << (4 * d);
            w[d] &= ~((nb >> 7) * 0xFFu);
          }
          sh_nan[(wave * D + 16 * i + col) * 4 + g] = (uint16_t)bits;
        }
      }
    }

    float top = x[0];
#pragma unroll
    for (int j = 1; j < 16; ++j) top = fmaxf(top, x[j]);
    top = fmaxf(top, __shfl_xor(top, 16, 64));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    const float mn = fmaxf(m, top);
    const float base = mn == -INFINITY ? 0.0f : mn;
    if (__ballot(mn != m)) {
      const float alpha = __builtin_amdgcn_exp2f(m - base);
      l *= alpha;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][r] *= alpha;
      m = mn;
    }
    Frag<E> p[2];
#pragma unroll
    for (int j = 0; j < 16; j += 2) {
      const float p0 = __builtin_amdgcn_exp2f(x[j] - base), p1 = __builtin_amdgcn_exp2f(x[j + 1] - base);
      l += p0 + p1;
      p[j >> 3].u[(j & 7) >> 1] = E::pack(p0, p1);
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      acc[i] = E::mfma(dec8<E>(vc[i].x, vc[i].y, vs), p[0].v, acc[i]);
      acc[i] = E::mfma(dec8<E>(vc[i].z, vc[i].w, vs), p[1].v, acc[i]);
    }
    if (poisoned) {
      __builtin_amdgcn_wave_barrier();
      __threadfence_block();
      unsigned long long seen = ~0ull;
      const int lo = row.lo - t0, hi = row.hi - t0;
      if (lo > 0) seen = lo >= 64 ? 0ull : seen << lo;
      if (hi < 64) seen = hi <= 0 ? 0ull : seen & ((1ull << hi) - 1ull);
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (nan_map(sh_nan + (wave * D + 16 * i + 4 * g + r) * 4) & seen) acc[i][r] = __builtin_nanf("");
      __builtin_amdgcn_wave_barrier();
    }
  }

  // the four waves' parts, joined in wave order
  l += __shfl_xor(l, 16, 64);
  l += __shfl_xor(l, 32, 64);
  float* mine = sh_o + (wave * 16 + col) * (D + 4);
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
    *reinterpret_cast<float4*>(mine + 16 * i + 4 * g) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
  if (g == 0) {
    sh_ml[(wave * 16 + col) * 2] = m;
    sh_ml[(wave * 16 + col) * 2 + 1] = l;
  }
  __syncthreads();
  const int jr = threadIdx.x >> 4, jd = threadIdx.x & 15;  // row, and elements 4 jd + 64 i
  const Row jrow = row_at(a, rt * 16 + jr, kvh, rows.n, len, room);
  if (jrow.i < 0) return;
  float M = -INFINITY, L = 0.0f, f[4];
#pragma unroll
  for (int w = 0; w < 4; ++w) M = fmaxf(M, sh_ml[(w * 16 + jr) * 2]);
  const float base = M == -INFINITY ? 0.0f : M;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    f[w] = __builtin_amdgcn_exp2f(sh_ml[(w * 16 + jr) * 2] - base);
    L += f[w] * sh_ml[(w * 16 + jr) * 2 + 1];
  }
  const int64_t slot = ((int64_t)blockIdx.x * gridDim.y + blockIdx.y) * 16 + jr;
#pragma unroll
  for (int i = 0; i < D / 64; ++i) {
    const int d = 4 * jd + 64 * i;
    float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float4 v = *reinterpret_cast<const float4*>(sh_o + (w * 16 + jr) * (D + 4) + d);
      o[0] += f[w] * v.x;
      o[1] += f[w] * v.y;
      o[2] += f[w] * v.z;
      o[3] += f[w] * v.w;
    }
    if (pieces == 1) {
      const float inv = L == 0.0f ? 0.0f : 1.0f / L;
      uint16_t* yr = a.y + (int64_t)(rows.first + jrow.i) * a.yt + (int64_t)jrow.head * a.yh;
      *reinterpret_cast<uint2*>(yr + d) = make_uint2(E::pack(o[0] * inv, o[1] * inv), E::pack(o[2] * inv, o[3] * inv));
    } else {
      *reinterpret_cast<float4*>(a.part_o + slot * D + d) = make_float4(o[0], o[1], o[2], o[3]);
    }
  }
  if (jd == 0) {
    if (pieces == 1) {
      if (a.lse) a.lse[(int64_t)(rows.first + jrow.i) * a.q_heads + jrow.head] = (M + __builtin_amdgcn_logf(L)) * kLn2;
    } else {
      a.part_ml[slot * 2] = M;
      a.part_ml[slot * 2 + 1] = L;
    }
  }
}

// joins the pieces of a sequence that was split: a workgroup per row (sequence, kv head, row of
// its 16), the pieces in a fixed order
template <class E, int D>
__global__ __launch_bounds__(256) void attn_join(Args a) {
  constexpr int LANES = D / 4, PER = 256 / LANES;  // threads over the elements, pieces at a time
  __shared__ float sh[PER][D + 4];
  __shared__ float sh_l[PER];
  const int b = blockIdx.x, kvh = blockIdx.y / 16, R = blockIdx.y % 16;
  const kv::Rows rows = kv::rows_of(a.cu, b, a.T);
  if (R >= rows.n * a.group) return;
  int len = a.c.lens[b];
  len = len < 0 ? 0 : len;
  const Row row = row_at(a, R, kvh, rows.n, len, room_of(a.c));
  if (row.i < 0) return;
  const int chunk = plan_chunk(a);
  const int pieces = piece_count(a, b, chunk);
  if (pieces <= 1) return;
  int before = 0;
  const int lane = threadIdx.x & 63;
  for (int b0 = 0; b0 < b; b0 += 64) before += wave_sum(b0 + lane < b ? piece_count(a, b0 + lane, chunk) : 0);
  const int64_t stride = (int64_t)a.c.heads * 16;  // rows of one piece
  const int64_t first = ((int64_t)before * a.c.heads + kvh) * 16 + R;
  float M = -INFINITY;
  for (int i = lane; i < pieces; i += 64) M = fmaxf(M, a.part_ml[(first + i * stride) * 2]);
  M = wave_max(M);
  const float base = M == -INFINITY ? 0.0f : M;
  const int who = threadIdx.x / LANES, d = 4 * (threadIdx.x % LANES);
  float o[4] = {0.0f, 0.0f, 0.0f, 0.0f}, L = 0.0f;
  for (int i = who; i < pieces; i += PER) {
    const int64_t at = first + i * stride;
    const float f = __builtin_amdgcn_exp2f(a.part_ml[at * 2] - base);
    const float4 v = *reinterpret_cast<const float4*>(a.part_o + at * D + d);
    L += f * a.part_ml[at * 2 + 1];
    o[0] += f * v.x;
    o[1] += f * v.y;
    o[2] += f * v.z;
    o[3] += f * v.w;
  }
  *reinterpret_cast<float4*>(&sh[who][d]) = make_float4(o[0], o[1], o[2], o[3]);
  if (d == 0) sh_l[who] = L;
  __syncthreads();
  if (who != 0) return;
#pragma unroll
  for (int w = 1; w < PER; ++w) {
    const float4 v = *reinterpret_cast<const float4*>(&sh[w][d]);
    o[0] += v.x;
    o[1] += v.y;
    o[2] += v.z;
    o[3] += v.w;
    L += sh_l[w];
  }
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
  uint16_t* yr = a.y + (int64_t)(rows.first + row.i) * a.yt + (int64_t)row.head * a.yh;
  *reinterpret_cast<uint2*>(yr + d) = make_uint2(E::pack(o[0] * inv, o[1] * inv), E::pack(o[2] * inv, o[3] * inv));
  if (d == 0 && a.lse)
    a.lse[(int64_t)(rows.first + row.i) * a.q_heads + row.head] = (M + __builtin_amdgcn_logf(L)) * kLn2;
}

// how a call is cut: row tiles of 16, and for a single one the pieces of all sequences together
struct Plan {
  int row_tiles, target;
  int64_t pieces;  // most pieces
};
Plan plan_of(int64_t batch, int64_t T, int64_t max_q_len, int64_t group, int64_t kv_heads) {
  Plan p;
  const int64_t most = max_q_len < T ? max_q_len : T;
  p.row_tiles = (int)((most * group + 15) / 16);
  int64_t target = p.row_tiles > 1 ? 0 : (512 + kv_heads - 1) / kv_heads;
  p.target = (int)target;
  p.pieces = target + batch;
  return p;
}
constexpr int kLeastTiles = 4;

template <class E, int D>
hipError_t launch(Args& a, const Plan& p, hipStream_t s) {
  static std::atomic<unsigned long long> raised{0};
  hipError_t e = ensure_lds_limit(reinterpret_cast<const void*>(attn_step<E, D>), step_lds<D>(), raised);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((attn_step<E, D>), dim3((unsigned)p.pieces, (unsigned)(a.c.heads * a.row_tiles)), dim3(256),
                     step_lds<D>(), s, a);
  e = hipGetLastError();
  if (e != hipSuccess || a.target == 0) return e;
  hipLaunchKernelGGL((attn_join<E, D>), dim3((unsigned)a.c.batch, (unsigned)a.c.heads * 16), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace

size_t attention_workspace(int64_t batch, int64_t T, int64_t max_q_len, int64_t q_heads, int64_t kv_heads,
                           int64_t head_dim) {
  const Plan p = plan_of(batch, T, max_q_len, q_heads / kv_heads, kv_heads);
  if (p.target == 0) return 0;
  return (size_t)(p.pieces * kv_heads * 16 * (head_dim + 2) * 4 + 255) & ~(size_t)255;
}

hipError_t launch_attention(bsq_dtype dt, const AttnArgs& p, void* workspace, hipStream_t s) {
  Args a{};
  a.c = p.c; a.cu = p.cu; a.T = p.T;
  a.q = static_cast<const uint16_t*>(p.q.p); a.qt = p.q.st; a.qh = p.q.sh;
  a.y = static_cast<uint16_t*>(const_cast<void*>(p.y.p)); a.yt = p.y.st; a.yh = p.y.sh;
  a.lse = p.lse;
  a.q_heads = p.q_heads;
  a.group = p.q_heads / p.c.heads;
  a.scale2 = p.scale * 1.44269504088896340736f;
  a.window = p.window;
  a.full = p.full;
  a.max_q_len = (int)(p.max_q_len < p.T ? p.max_q_len : p.T);
  const Plan plan = plan_of(p.c.batch, p.T, p.max_q_len, a.group, p.c.heads);
  a.row_tiles = plan.row_tiles;
  a.target = plan.target;
  a.least = kLeastTiles;
  a.part_o = static_cast<float*>(workspace);
  a.part_ml = a.part_o + plan.pieces * p.c.heads * 16 * p.c.dim;
  const bool half = dt == BSQ_FP16;
  switch (p.c.dim) {
    case 64: return half ? launch<Fp16, 64>(a, plan, s) : launch<Bf16, 64>(a, plan, s);
    case 128: return half ? launch<Fp16, 128>(a, plan, s) : launch<Bf16, 128>(a, plan, s);
    default: return half ? launch<Fp16, 256>(a, plan, s) : launch<Bf16, 256>(a, plan, s);
  }
}

}  // namespace bsq
