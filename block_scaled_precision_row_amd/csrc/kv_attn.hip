// Attention over the paged E4M3 cache: the step kernel (a decode step: up to 16 rows, a token's queries of
// one kv head or a few tokens', against all tokens of a sequence), the joining of its partial results,
// and the choice between it and the prompt kernel (kv_prompt.hip).
//
// One pass over the tokens with the running maximum and sum of the softmax in fp32. S^T = K Q^T on
// 16x16x32 MFMA (rows: tokens, columns: query rows), then O^T += V^T P^T on the same. A lane of the first
// product's result holds column (query row) l % 16 and rows 4 (l / 16) + 0..3; row 4 g + r of K tile j is
// taken to be token 16 g + 4 j + r, so that over the four tiles a lane ends up with the 16 consecutive
// tokens of granule l / 16: one page, one scale of K and of V to a lane, and P in the order in which the
// second product wants its operand, without a shuffle or LDS. E4M3 becomes 16-bit exactly, two values an
// instruction; V's scale is in the weights (kv_attn.hpp).
//
// Bound by memory: 2 D bytes per token and kv head. Every wave streams tiles of 64 tokens of its own
// through two LDS buffers (16 KB each for D 128), the next tile in flight while it works on one; two
// workgroups of 64 KB to a compute unit: 64 sequences of 4000 to 8000 tokens, 32 / 8 heads of 128, 773 MB, 158 us a call
// with the join (7.5), 5.1 TB/s. Loading the operands straight into registers, neighbouring lanes on
// neighbouring rows, left the address unit with 16-byte pieces (205 us).
#include "kv_attn.hpp"

namespace bsq {

namespace {

using namespace attn;

// v and what DPP control `ctrl` brings from other lanes of its row or of the rows before (0 where there is none)
template <int ctrl, int rows>
__device__ __forceinline__ int add_from(int v) {
  return v + __builtin_amdgcn_update_dpp(0, v, ctrl, rows, 0xF, false);
}
__device__ __forceinline__ int wave_scan(int v) {  // inclusive
  v = add_from<0x111, 0xF>(v);  // within 16 lanes: row_shr 1, 2, 4, 8
  v = add_from<0x112, 0xF>(v);
  v = add_from<0x114, 0xF>(v);
  v = add_from<0x118, 0xF>(v);
  v = add_from<0x142, 0xA>(v);  // row_bcast 15: rows 0 and 2 to 1 and 3
  return add_from<0x143, 0xC>(v);  // row_bcast 31: the first half to the second
}
__device__ __forceinline__ int wave_sum(int v) { return __builtin_amdgcn_readlane(wave_scan(v), 63); }

// tiles of sequence b over all its rows; -1 for one that the step kernel does not take
__device__ __forceinline__ int sequence_tiles(const Args& a, int b) {
  const int n = kv::rows_of(a.cu, b, a.T).n, len = a.c.lens[b];  // (loaded together)
  if (n == 0 || (int64_t)n * a.group > a.small) return -1;
  return kv::tiles_of(kv::seen_range(len < 0 ? 0 : len, room_of(a.c), n, 0, n, a.window, a.full));
}

// The tiles of all sequences together. Every wave finds sums and places by itself from the lengths, 64
// sequences at a time.
struct Tiles {
  int total, chunk;
  int mine, upto;  // this lane's sequence (batches of up to 64) and the sum up to it
};
__device__ __forceinline__ int lane_tiles(const Args& a, int b) {
  const int t = b < a.c.batch ? sequence_tiles(a, b) : 0;
  return t > 0 ? t : 0;
}
__device__ __forceinline__ Tiles count_tiles(const Args& a) {
  const int lane = threadIdx.x & 63;
  Tiles t;
  t.mine = lane_tiles(a, lane);
  t.upto = wave_scan(t.mine);
  t.total = __builtin_amdgcn_readlane(t.upto, 63);
  for (int b0 = 64; b0 < a.c.batch; b0 += 64) t.total += wave_sum(lane_tiles(a, b0 + lane));
  t.chunk = kv::chunk_of(t.total, a.target, a.least);
  return t;
}
// the sequence that holds tile x and the number of its tiles before x
__device__ __forceinline__ void find_tile(const Args& a, const Tiles& t, int x, int& b, int& before) {
  const int lane = threadIdx.x & 63;
  int sum = 0;
  int mine = t.mine, upto = t.upto;
  for (int b0 = 0;; b0 += 64) {
    if (b0 > 0) {
      mine = lane_tiles(a, b0 + lane);
      upto = wave_scan(mine);
    }
    const unsigned long long hit = __ballot(sum + upto > x);
    if (hit || b0 + 64 >= a.c.batch) {
      const int at = hit ? __builtin_ctzll(hit) : 63;
      b = __builtin_amdgcn_readfirstlane(b0 + at);
      before = x - sum - __builtin_amdgcn_readlane(upto - mine, at);
      return;
    }
    sum += __builtin_amdgcn_readlane(upto, 63);
  }
}
// tiles of the sequences before b
__device__ __forceinline__ int tiles_before(const Args& a, const Tiles& t, int b) {
  const int lane = threadIdx.x & 63;
  if (b < 64) return __builtin_amdgcn_readlane(t.upto - t.mine, b);
  int sum = 0;
  for (int b0 = 0; b0 < b; b0 += 64) sum += wave_sum(b0 + lane < b ? lane_tiles(a, b0 + lane) : 0);
  return sum;
}

__device__ __forceinline__ int min16(int v) {  // over the 16 columns
#pragma unroll
  for (int off = 8; off >= 1; off >>= 1) {
    const int o = __shfl_xor(v, off, 64);
    v = o < v ? o : v;
  }
  return v;
}
__device__ __forceinline__ int max16(int v) { return -min16(-v); }

constexpr int step_waves(int D) { return 256 / D; }
// two tile buffers a wave (taken over by the waves' results at the end), maxima and sums, NaN maps
constexpr int step_lds(int D) { return step_waves(D) * (2 * tile_bytes(D) + 16 * 2 * 4 + D * 8); }

template <class E, int D>
__global__ __launch_bounds__(64 * step_waves(D)) void attn_step(Args a) {
  constexpr int W = step_waves(D);
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  float* sh_o = reinterpret_cast<float*>(smem);  // [W][16][D + 4]
  static_assert(16 * (D + 4) * 4 <= 2 * tile_bytes(D), "results fit in the buffers");
  float* sh_ml = reinterpret_cast<float*>(smem + W * 2 * tile_bytes(D));  // [W][16][2]
  uint16_t* sh_nan = reinterpret_cast<uint16_t*>(sh_ml + W * 16 * 2);       // [W][D][4 granules]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, g = lane >> 4;
  const int kvh = blockIdx.y, room = room_of(a.c), range = blockIdx.x;
  const Tiles plan = count_tiles(a);
  const int64_t from = (int64_t)range * plan.chunk;
  if (from >= plan.total) return;
  const int begin = (int)from, end = plan.total - begin < plan.chunk ? plan.total : begin + plan.chunk;
  const TileLoads<D, kv::kStep> loads(a.c);
  const int v_off = kv::v_at(col, g, kv::v_run(a.c.shift));
  int k_off[4];  // K tile j: this lane's row
#pragma unroll
  for (int j = 0; j < 4; ++j) k_off[j] = 16 * (col >> 2) + 4 * j + (col & 3);

  for (int x0 = begin; x0 < end;) {  // the sequences of the range
  int b, tile0;
  find_tile(a, plan, x0, b, tile0);
  const kv::Rows rows = kv::rows_of(a.cu, b, a.T);
  int len = a.c.lens[b];
  len = len < 0 ? 0 : len;
  const kv::Range all = kv::seen_range(len, room, rows.n, 0, rows.n, a.window, a.full);
  const int tiles = kv::tiles_of(all);
  const int tile1 = end - x0 < tiles - tile0 ? tile0 + (end - x0) : tiles;
  const bool direct = tile0 == 0 && tile1 == tiles;
  const int64_t part = kv::partial_slot(range, x0 == begin);
  x0 += tile1 - tile0;
  const int count = tile1 - tile0 - wave > 0 ? (tile1 - tile0 - wave + W - 1) / W : 0;  // this wave's tiles
  const int first = all.lo + kv::kTile * (tile0 + wave), stride = kv::kTile * W;

  const uint8_t* buf = smem + wave * 2 * tile_bytes(D);
  const uint32_t buf_lds = lds_offset(buf);
  const int seen_lo = a.window > 0 ? row_at(a, 0, kvh, rows.n, len, room).lo : 0;  // the first token that any row sees
  Pages pages;
  if (count > 0) {
    pages.load<D>(a.c, b, kvh, first, stride, seen_lo, all.hi);
    loads.template issue<0, tile_loads(D)>(a.c, pages, 0, buf_lds);
  }

  const Row row = row_at(a, col, kvh, rows.n, len, room, true);
  const int any_lo = min16(row.i < 0 ? 0x7FFFFFFF : row.lo), any_hi = max16(row.i < 0 ? 0 : row.hi);
  const int all_lo = max16(row.i < 0 ? 0 : row.lo), all_hi = min16(row.hi);
  Frag<E> q[D / 32];  // column col, elements 64 (s / 2) + 16 g + 8 (s % 2) + 0..7
  {
    const uint16_t* qr = a.q + (int64_t)(rows.first + (row.i < 0 ? 0 : row.i)) * a.qt + (int64_t)row.head * a.qh;
#pragma unroll
    for (int s = 0; s < D / 32; ++s)
      q[s].q = row.i < 0 ? make_uint4(0, 0, 0, 0)
                         : signed_query(*reinterpret_cast<const uint4*>(qr + 64 * (s >> 1) + 16 * g + 8 * (s & 1)), a.sign);
  }

  v4f acc[D / 16];
#pragma unroll
  for (int i = 0; i < D / 16; ++i) acc[i] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
  float m = -INFINITY, l = 0.0f;
  bool large = false;

  for (int it = 0; it < count; ++it) {
    const int t0 = first + stride * it, vt = t0 + 16 * g;
    if ((it & 15) == 0) pages.settle();
    const int vid = pages.gone(it, g), vs = pages.vshift(it, g);
    const float ks = pages.kscale(it, g) * a.scale2;
    const uint8_t* kb = buf + (it & 1) * tile_bytes(D);
    const uint8_t* vb = kb + 64 * D;
    if (it + 1 < count) {
      if (((it + 1) & 15) == 0) pages.load<D>(a.c, b, kvh, t0 + stride, stride, seen_lo, all.hi);
      wait_reads();
      loads.template issue<0, tile_loads(D)>(a.c, pages, it + 1, buf_lds + ((it + 1) & 1) * tile_bytes(D));
      wait_loads<tile_loads(D)>();
    } else {
      wait_loads<0>();
    }

    float x[16];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v4f s = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        const uint4 k = *reinterpret_cast<const uint4*>(kb + kv::k_at<D, kv::kStep>(k_off[j], 4 * i + g));
        s = E::mfma(dec8<E>(k.x, k.y, 1.0f), q[2 * i].v, s);
        s = E::mfma(dec8<E>(k.z, k.w, 1.0f), q[2 * i + 1].v, s);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) x[4 * j + r] = s[r] * ks;
    }
    const bool masked = t0 < all_lo || t0 + kv::kTile > all_hi || __ballot(vid < 0) != 0;
    if (masked) {
      const int lo = vid < 0 ? 16 : row.lo - vt, hi = row.hi - vt;
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] = j >= lo && j < hi ? x[j] : -INFINITY;
    }
    float top = x[0];
#pragma unroll
    for (int j = 1; j < 16; ++j) top = fmaxf(top, x[j]);
    top += (float)vs;
    top = fmaxf(top, __shfl_xor(top, 16, 64));
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    if (__ballot(outgrown(top, m))) {
      const float mn = ceilf(fmaxf(m, top));
      const float alpha = __builtin_amdgcn_exp2f(m - finite_base(mn));
      l *= alpha;
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][r] *= alpha;
      m = mn;
      large = __ballot(coarse(m)) != 0;
    }
    float base = finite_base(m);
    if (large) {
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] = coarse_score(x[j] - base, vs);
      base = 0.0f;
    }
    base -= (float)(vs + kLift);
    float sum = 0.0f;
    Frag<Fp16> p[2], rest[2];
#pragma unroll
    for (int j = 0; j < 16; j += 2) {
      const float p0 = __builtin_amdgcn_exp2f(x[j] - base), p1 = __builtin_amdgcn_exp2f(x[j + 1] - base);
      sum += p0 + p1;
      two_parts(p0, p1, p[j >> 3].u[(j & 7) >> 1], rest[j >> 3].u[(j & 7) >> 1]);
    }
    l += ldexpf(sum, -vs);
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      v4u v = *reinterpret_cast<const v4u*>(vb + 1024 * i + v_off);
      bool poisoned = false;
      if (masked) {
        const uint32_t bits = hide_codes(v, vid < 0 ? 16 : any_lo - vt, any_hi - vt);
        poisoned = __ballot(bits != 0) != 0;
        if (poisoned) sh_nan[(wave * 16 + col) * 4 + g] = (uint16_t)bits;
      }
      const v8h v0 = dec8<Fp16>(v.x, v.y, 1.0f);
      acc[i] = Fp16::mfma(v0, rest[0].v, acc[i]);
      acc[i] = Fp16::mfma(v0, p[0].v, acc[i]);
      const v8h v1 = dec8<Fp16>(v.z, v.w, 1.0f);
      acc[i] = Fp16::mfma(v1, rest[1].v, acc[i]);
      acc[i] = Fp16::mfma(v1, p[1].v, acc[i]);
      if (poisoned) {  // the rows that see a NaN get it
        __threadfence_block();
        __builtin_amdgcn_wave_barrier();
        const unsigned long long seen = seen_bits(row, t0);
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (nan_map(sh_nan + (wave * 16 + 4 * g + r) * 4) & seen) acc[i][r] = __builtin_nanf("");
        __builtin_amdgcn_wave_barrier();
      }
    }
  }

  // the waves' parts, joined in wave order
  l += __shfl_xor(l, 16, 64);
  l += __shfl_xor(l, 32, 64);
  l *= 1.0f / (1 << kLift);
  const float unit = pages.unit();
  __syncthreads();
  float* mine = sh_o + (wave * 16 + col) * (D + 4);
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
    *reinterpret_cast<float4*>(mine + 16 * i + 4 * g) = make_float4(acc[i][0] * unit, acc[i][1] * unit, acc[i][2] * unit, acc[i][3] * unit);
  if (g == 0) {
    sh_ml[(wave * 16 + col) * 2] = m;
    sh_ml[(wave * 16 + col) * 2 + 1] = l;
  }
  __syncthreads();
  constexpr int kRowsAtOnce = 4 * W;  // 16 threads a row, 4 elements each at a time
#pragma unroll
  for (int jr = threadIdx.x >> 4; jr < 16; jr += kRowsAtOnce) {
    const int jd = threadIdx.x & 15;
    const Row jrow = row_at(a, jr, kvh, rows.n, len, room, true);
    if (jrow.i < 0) continue;
    float M = -INFINITY, L = 0.0f, f[W];
#pragma unroll
    for (int w = 0; w < W; ++w) M = fmaxf(M, sh_ml[(w * 16 + jr) * 2]);
    const float base = M == -INFINITY ? 0.0f : M;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      f[w] = __builtin_amdgcn_exp2f(sh_ml[(w * 16 + jr) * 2] - base);
      L += f[w] * sh_ml[(w * 16 + jr) * 2 + 1];
    }
    const int64_t slot = (part * a.c.heads + kvh) * 16 + jr;
    const int64_t out = (int64_t)(rows.first + jrow.i);
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
      const int d = 4 * jd + 64 * i;
      float o[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float4 v = *reinterpret_cast<const float4*>(sh_o + (w * 16 + jr) * (D + 4) + d);
        o[0] += f[w] * v.x;
        o[1] += f[w] * v.y;
        o[2] += f[w] * v.z;
        o[3] += f[w] * v.w;
      }
      if (direct) {
        const float inv = L == 0.0f ? 0.0f : 1.0f / L;
        uint16_t* yr = a.y + out * a.yt + (int64_t)jrow.head * a.yh;
        *reinterpret_cast<uint2*>(yr + d) = make_uint2(E::pack(o[0] * inv, o[1] * inv), E::pack(o[2] * inv, o[3] * inv));
      } else {
        *reinterpret_cast<float4*>(a.part_o + slot * D + d) = make_float4(o[0], o[1], o[2], o[3]);
      }
    }
    if (jd == 0) {
      if (direct) {
        if (a.lse) a.lse[out * a.q_heads + jrow.head] = (M + __builtin_amdgcn_logf(L)) * kLn2;
      } else {
        a.part_ml[slot * 2] = M;
        a.part_ml[slot * 2 + 1] = L;
      }
    }
  }
  __syncthreads();  // the results are read before the next sequence's tiles arrive in their place
  }
}

// Joins the partial results of a sequence that lies in several ranges, in their order, and writes the rows of
// one without tokens: a workgroup per row (sequence, kv head, row of its 16).
template <class E, int D>
__global__ __launch_bounds__(256) void attn_join(Args a, int rows_max) {
  constexpr int LANES = D / 4, PER = 256 / LANES;  // threads over the elements, partial results at a time
  __shared__ float sh[PER][D + 4];
  __shared__ float sh_l[PER];
  const int b = blockIdx.x, kvh = blockIdx.y / rows_max, R = blockIdx.y % rows_max;
  const kv::Rows rows = kv::rows_of(a.cu, b, a.T);
  const int tiles = sequence_tiles(a, b);
  if (tiles < 0) return;
  int len = a.c.lens[b];
  len = len < 0 ? 0 : len;
  const Row row = row_at(a, R, kvh, rows.n, len, room_of(a.c), true);
  if (row.i < 0) return;
  const int who = threadIdx.x / LANES, d = 4 * (threadIdx.x % LANES);
  uint16_t* yr = a.y + (int64_t)(rows.first + row.i) * a.yt + (int64_t)row.head * a.yh;
  float* lse = a.lse ? a.lse + (int64_t)(rows.first + row.i) * a.q_heads + row.head : nullptr;
  if (tiles == 0) {
    if (who == 0) *reinterpret_cast<uint2*>(yr + d) = make_uint2(0, 0);
    if (threadIdx.x == 0 && lse) *lse = -INFINITY;
    return;
  }
  const Tiles plan = count_tiles(a);
  const int x = tiles_before(a, plan, b);
  const int r0 = kv::range_of(plan.chunk, x), r1 = kv::range_of(plan.chunk, x + tiles - 1);
  if (r0 == r1) return;
  const int pieces = r1 - r0 + 1;
  const bool first_begins = x == r0 * plan.chunk;
  auto at = [&](int i) { return (kv::partial_slot(r0 + i, i > 0 || first_begins) * a.c.heads + kvh) * 16 + R; };
  // this thread's first pieces are on their way while the maximum is found
  constexpr int kAhead = 4;
  float4 v[kAhead];
  float2 ml[kAhead];
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    const int64_t p = at(who + PER * j < pieces ? who + PER * j : 0);
    v[j] = *reinterpret_cast<const float4*>(a.part_o + p * D + d);
    ml[j] = *reinterpret_cast<const float2*>(a.part_ml + p * 2);
  }
  float M = -INFINITY;
  for (int i = threadIdx.x & 63; i < pieces; i += 64) M = fmaxf(M, a.part_ml[at(i) * 2]);
  M = wave_max(M);
  const float base = finite_base(M);
  float o[4] = {0.0f, 0.0f, 0.0f, 0.0f}, L = 0.0f;
  auto add = [&](float4 x, float2 r) {
    const float f = __builtin_amdgcn_exp2f(r.x - base);
    L += f * r.y;
    o[0] += f * x.x;
    o[1] += f * x.y;
    o[2] += f * x.z;
    o[3] += f * x.w;
  };
#pragma unroll
  for (int j = 0; j < kAhead; ++j)
    if (who + PER * j < pieces) add(v[j], ml[j]);
#pragma unroll 4
  for (int i = who + PER * kAhead; i < pieces; i += PER) {
    const int64_t p = at(i);
    add(*reinterpret_cast<const float4*>(a.part_o + p * D + d), *reinterpret_cast<const float2*>(a.part_ml + p * 2));
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
  }
  L = sh_l[0];
#pragma unroll
  for (int w = 1; w < PER; ++w) L += sh_l[w];
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
  *reinterpret_cast<uint2*>(yr + d) = make_uint2(E::pack(o[0] * inv, o[1] * inv), E::pack(o[2] * inv, o[3] * inv));
  if (d == 0 && lse) *lse = (M + __builtin_amdgcn_logf(L)) * kLn2;
}

// How a call is cut. Sequences of at most 16 rows (tokens times group) go to the step kernel, longer ones
// to the prompt kernel. Where max_q_len, or a batch of one, rules one of them out it is not launched; nor the step
// kernel where short sequences cannot keep the prompt kernel waiting (launch_attention).
struct Cut {
  bool step, prompt;
  int target;        // step: most ranges
  int rows;          // step: most rows of a sequence and kv head
  int64_t blocks;    // prompt: most blocks of 128 rows
  int splits, least; // prompt: most parts of a block, least tiles of a part
  size_t step_bytes, prompt_bytes;
};
// (a tile takes a lone workgroup 1.7 us, most of it the wait for its loads: 20 rows over 900 tokens 36 us in parts of
// eight tiles at least, 22.6 of four, 20.3 of three, 21.2 of two; 64 over 3000 28.0 of three, 30.5 of two)
constexpr int kLeastPromptTiles = 3;
Cut cut_of(int64_t batch, int64_t T, int64_t max_q_len, int64_t group, int64_t kv_heads, int64_t D) {
  Cut p{};
  const int64_t most = (max_q_len < T ? max_q_len : T) * group;
  p.prompt = most > 16;
  p.step = most <= 16 || (group <= 16 && batch > 1);
  if (p.step) {
    p.target = (int)((512 + kv_heads - 1) / kv_heads);  // two workgroups to a compute unit
    p.rows = (int)(most < 16 ? most : 16);
    p.step_bytes = (size_t)(2 * p.target * kv_heads * 16 * (D + 2) * 4 + 255) & ~(size_t)255;
  }
  if (p.prompt) {
    p.blocks = kv::prompt_blocks(T, batch, group);
    const int64_t all = p.blocks * kv_heads;
    // One workgroup to a compute unit (two: 18 % faster to 25 % slower, for every part's results are written and read
    // again: 64 rows and 99 x 1 over 8000 tokens 95 us against 117, 100 rows over 8000, two heads of 64, 46 against 37). Blocks
    // for more than half of them are cut in two where they are long, if two workgroups fit a unit (900 rows over
    // 6000 tokens, 32 / 8 heads of 64: 119 us whole, 101 cut, of 128: 160 and 154; over 2000 of 64 46 and 51, of 128 62 and 69;
    // 600 over 2000, heads of 256, of which one fits: 123 and 131).
    if (all <= 128) {
      p.splits = (int)(256 / all > 64 ? 64 : 256 / all);
      p.least = kLeastPromptTiles;
    } else {
      p.splits = all < 256 && D < 256 ? 2 : 1;
      p.least = 32;
    }
    if (p.splits > 1) p.prompt_bytes = (size_t)(all * p.splits * 128 * (D + 2) * 4 + 255) & ~(size_t)255;
  }
  return p;
}
constexpr int kLeastTiles = 2;

template <class E, int D>
hipError_t launch_step(const Args& a, const Cut& p, hipStream_t s) {
  static std::atomic<unsigned long long> raised{0};
  hipError_t e = ensure_lds_limit(reinterpret_cast<const void*>(attn_step<E, D>), step_lds(D), raised);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((attn_step<E, D>), dim3((unsigned)p.target, (unsigned)a.c.heads), dim3(64 * step_waves(D)),
                     step_lds(D), s, a);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((attn_join<E, D>), dim3((unsigned)a.c.batch, (unsigned)(a.c.heads * p.rows)), dim3(256), 0, s, a,
                     p.rows);
  return hipGetLastError();
}

}  // namespace

size_t attention_workspace(int64_t batch, int64_t T, int64_t max_q_len, int64_t q_heads, int64_t kv_heads,
                           int64_t head_dim) {
  const Cut p = cut_of(batch, T, max_q_len, q_heads / kv_heads, kv_heads, head_dim);
  return p.step_bytes + p.prompt_bytes;
}

hipError_t launch_attention(bsq_dtype dt, const AttnArgs& p, void* workspace, hipStream_t s) {
  Args a{};
  a.c = p.c; a.cu = p.cu; a.T = p.T;
  a.q = static_cast<const uint16_t*>(p.q.p); a.qt = p.q.st; a.qh = p.q.sh;
  a.y = static_cast<uint16_t*>(const_cast<void*>(p.y.p)); a.yt = p.y.st; a.yh = p.y.sh;
  a.lse = p.lse;
  a.q_heads = p.q_heads;
  a.group = p.q_heads / p.c.heads;
  a.group_inverse = kv::inverse_of(a.group);
  a.sign = p.scale < 0.0f ? -1 : 1;
  a.scale2 = fabsf(p.scale) * 1.44269504088896340736f;
  a.window = p.window;
  a.full = p.full;
  a.max_q_len = (int)(p.max_q_len < p.T ? p.max_q_len : p.T);
  Cut plan = cut_of(p.c.batch, p.T, p.max_q_len, a.group, p.c.heads, p.c.dim);
  // Short sequences go along with the prompt kernel where none of its workgroups can have more than 64 tiles for
  // that (one token's block costs it about what it costs the step kernel, and an idle step kernel and its join 3 to 4 us,
  // 9 on the card: 64 rows and 27 x 1 over 700 tokens 43 us with the step kernel, 23 without; 64 and 99 x 1 over 8000,
  // one kv head, 165 and 117; 200 and 63 x 1 over 3000 91 and 77). A longer one would keep its workgroup for itself: 2048 rows
  // and 7 x 1 over 8000 tokens 112 us with the step kernel, 216 without; 2048 rows and three of 40000 to 60000 tokens 146 and
  // 1479. That goes by the table's width, for the lengths are on the device: with a wide table the step kernel and its
  // join are launched beside any prompt of several sequences.
  const int64_t most_tiles = ((int64_t)p.c.max_pages << p.c.shift) / kv::kTile + 1;
  if (plan.prompt && most_tiles <= 64 * (int64_t)plan.splits) plan.step = false;
  // no parts, no join, where the table has no room for a block of several (a join costs 5 us)
  if (plan.prompt && most_tiles / plan.least < plan.splits)
    plan.splits = most_tiles < 2 * plan.least ? 1 : (int)(most_tiles / plan.least);
  a.least = kLeastTiles;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  hipError_t e = hipSuccess;
  if (plan.prompt) {
    Args b = a;
    b.small = plan.step ? 16 : 0;
    b.splits = plan.splits;
    b.least = plan.least;
    b.part_o = reinterpret_cast<float*>(ws + plan.step_bytes);
    b.part_ml = b.part_o + plan.blocks * p.c.heads * plan.splits * 128 * p.c.dim;
    e = launch_attn_prompt(dt, b, s);
  }
  if (e != hipSuccess || !plan.step) return e;
  a.small = plan.prompt ? 16 : 0x7FFFFFFF;  // (a sequence longer than max_q_len promised is cut, not left out)
  a.target = plan.target;
  a.part_o = reinterpret_cast<float*>(ws);
  a.part_ml = a.part_o + (int64_t)2 * plan.target * p.c.heads * 16 * p.c.dim;
  const bool half = dt == BSQ_FP16;
  switch (p.c.dim) {
    case 64: return half ? launch_step<Fp16, 64>(a, plan, s) : launch_step<Bf16, 64>(a, plan, s);
    case 128: return half ? launch_step<Fp16, 128>(a, plan, s) : launch_step<Bf16, 128>(a, plan, s);
    default: return half ? launch_step<Fp16, 256>(a, plan, s) : launch_step<Bf16, 256>(a, plan, s);
  }
}

}  // namespace bsq
