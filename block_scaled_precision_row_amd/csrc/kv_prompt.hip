// Attention of many rows over the paged E4M3 cache (prompts and their chunks, wide groups): blocks of 128 rows
// (token, query head of the group) of one sequence and kv head, 32 to a wave, against tiles of 64
// tokens that the four waves share in LDS.
//
// S^T = K Q^T on 32x32x16 MFMA, then O^T += V^T P^T on the same. A lane of the first product's result holds
// column (query row) l % 32 and rows 8 a + 4 (l / 32) + b (a, b < 4); row 8 a + 4 h + b of K tile j is taken to
// be token 32 h + 16 j + 4 a + b, so that a lane holds the 16 consecutive tokens of granule 2 (l / 32) + j in
// tile j: one scale of K and of V each, and P in the order in which the second product wants its operand.
//
// Bound by the vector instructions of the softmax and the decoding of E4M3 (two values an instruction), some 170 to
// every 24 products of 32 rows and tokens, and by the matrix cores, a third of whose work is the weights' second part
// (kv_attn.hpp). Tiles come into two LDS buffers, one in flight while the other is worked on, with one barrier a tile.
// 3 sequences of 750 to 1500 rows over up to 6000 tokens, 32 / 8 heads of 128: 333 us, 613 TFLOP/s (281 with weights of 11
// bits). Two waves a SIMD for heads of 128 (three: 63 registers spilled, 354 us), three for 64 (205 us for the same
// sequences; two: 223). K and V are read again by every block of rows, from the L2 cache for the most part.
#include <type_traits>

#include "kv_attn.hpp"

namespace bsq {

namespace {

using namespace attn;

using kv::kBlock;

// the last b whose first block is at most `id`, -1 if none: 64 candidates a step
__device__ __forceinline__ int block_sequence(const Args& a, int64_t id) {
  const int lane = threadIdx.x & 63;
  return __builtin_amdgcn_readfirstlane(kv::last_of<64>(a.c.batch, [&](int lo, int step, int n) {
    const bool in = lane * step < n && kv::first_block(a.cu, lo + lane * step, a.T, a.group) <= id;
    return (int)__popcll(__ballot(in));
  }));
}

// a block's rows and the tokens they see
struct Block {
  int b, r0;  // sequence, first row of its n * group
  kv::Rows rows;
  int len;
  kv::Range range;
};
__device__ __forceinline__ bool find_block(const Args& a, int64_t id, Block& o) {
  o.b = block_sequence(a, id);
  if (o.b < 0) return false;
  o.rows = kv::rows_of(a.cu, o.b, a.T);
  o.r0 = kv::block_row(a.cu, o.b, o.rows, a.T, a.group, id, a.small, a.max_q_len);
  if (o.r0 < 0) return false;
  const int len = a.c.lens[o.b];
  o.len = len < 0 ? 0 : len;
  const int i0 = o.r0 / a.group;
  const int64_t i1 = ((int64_t)o.r0 + kBlock - 1) / a.group;
  const int last = i1 < o.rows.n - 1 ? (int)i1 : o.rows.n - 1;
  o.range = kv::seen_range(o.len, room_of(a.c), o.rows.n, i0, last - i0 + 1, a.window, a.full);
  return true;
}
// parts that a block's tiles are cut into
__device__ __forceinline__ int parts_of(const Args& a, int tiles) {
  const int most = tiles / a.least < 1 ? 1 : tiles / a.least;
  return a.splits < most ? a.splits : most;
}

constexpr int prompt_lds(int D) { return 2 * tile_bytes(D) + D * 8; }  // buffers; the NaN map

template <class E, int D>
__global__ __launch_bounds__(256, D == 256 ? 1 : (D == 128 ? 2 : 3)) void attn_prompt(Args a) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  uint16_t* sh_nan = reinterpret_cast<uint16_t*>(smem + 2 * tile_bytes(D));  // [D][4 granules]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 31, h = lane >> 5;
  // later blocks see more tokens: they go first; neighbouring workgroups, which go to different XCDs, take
  // different heads, so that an XCD's L2 holds few of them
  const int kvh = blockIdx.x % a.c.heads;
  const int64_t id = (gridDim.x - 1 - blockIdx.x) / a.c.heads;
  Block blk;
  if (!find_block(a, id, blk)) return;
  const int tiles = kv::tiles_of(blk.range), parts = parts_of(a, tiles);
  if ((int)blockIdx.y >= parts) return;
  const int tile0 = kv::piece_begin(tiles, parts, blockIdx.y), tile1 = kv::piece_begin(tiles, parts, blockIdx.y + 1);
  const int count = tile1 - tile0, first = blk.range.lo + kv::kTile * tile0;
  const int room = room_of(a.c);

  const uint32_t lds = lds_offset(smem);
  const TileLoads<D, kv::kPrompt> loads(a.c);
  constexpr int kMine = tile_loads(D) / 4;  // a wave's share of a tile's loads
  const int seen_lo = row_at(a, blk.r0, kvh, blk.rows.n, blk.len, room).lo;  // the first token that any row sees
  Pages pages;
  auto issue = [&](int tile, uint32_t at) __attribute__((always_inline)) {
    if (wave == 0) loads.template issue<0, kMine>(a.c, pages, tile, at);
    else if (wave == 1) loads.template issue<kMine, 2 * kMine>(a.c, pages, tile, at);
    else if (wave == 2) loads.template issue<2 * kMine, 3 * kMine>(a.c, pages, tile, at);
    else loads.template issue<3 * kMine, 4 * kMine>(a.c, pages, tile, at);
  };
  if (count > 0) {
    pages.load<D>(a.c, blk.b, kvh, first, kv::kTile, seen_lo, blk.range.hi);
    issue(0, lds);
  }

  const int R = blk.r0 + 32 * wave + col;
  const Row row = row_at(a, R, kvh, blk.rows.n, blk.len, room);
  Frag<E> q[D / 16];  // elements 32 (s / 2) + 16 h + 8 (s % 2) + 0..7
  {
    const uint16_t* qr = a.q + (int64_t)(blk.rows.first + (row.i < 0 ? 0 : row.i)) * a.qt + (int64_t)row.head * a.qh;
#pragma unroll
    for (int s = 0; s < D / 16; ++s)
      q[s].q = row.i < 0 ? make_uint4(0, 0, 0, 0)
                         : signed_query(*reinterpret_cast<const uint4*>(qr + 32 * (s >> 1) + 16 * h + 8 * (s & 1)), a.sign);
  }
  const int k_token = 32 * (col >> 2 & 1) + 4 * (col >> 3) + (col & 3);  // K tile 0's row; tile 1's is 16 on
  const int run = kv::v_run(a.c.shift);
  int v_off[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) v_off[j] = kv::v_at(col, 2 * h + j, run);

  v16f acc[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[i][r] = 0.0f;
  float m = -INFINITY, l = 0.0f;
  bool large = false;

  // Granules j and 2 + j of a tile; `masked`: some row of the block does not see some of the tile.
  auto half_tile = [&](auto masked, int j, int t0, const uint8_t* kb, int vid, float ks, int vs)
                       __attribute__((always_inline)) {
    const uint8_t* vb = kb + 64 * D;
    v16f s;
#pragma unroll
    for (int r = 0; r < 16; ++r) s[r] = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint4 k = *reinterpret_cast<const uint4*>(kb + kv::k_at<D, kv::kPrompt>(k_token + 16 * j, 2 * i + h));
      s = E::mfma32(dec8<E>(k.x, k.y, 1.0f), q[2 * i].v, s);
      s = E::mfma32(dec8<E>(k.z, k.w, 1.0f), q[2 * i + 1].v, s);
    }
    if constexpr (masked) {
      const int vt = t0 + 32 * h + 16 * j, lo = vid < 0 ? 16 : row.lo - vt, hi = row.hi - vt;
#pragma unroll
      for (int r = 0; r < 16; ++r) s[r] = r >= lo && r < hi ? s[r] * ks : -INFINITY;
      ks = 1.0f;
    }
    float top = s[0];
#pragma unroll
    for (int r = 1; r < 16; ++r) top = fmaxf(top, s[r]);
    top = fmaf(top, ks, (float)vs);
    top = fmaxf(top, __shfl_xor(top, 32, 64));
    if (__ballot(outgrown(top, m))) {
      const float mn = ceilf(fmaxf(m, top));
      const float alpha = __builtin_amdgcn_exp2f(m - finite_base(mn));
      l *= alpha;
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][r] *= alpha;
      m = mn;
      large = __ballot(coarse(m)) != 0;
    }
    float base = finite_base(m);
    if (large) {
#pragma unroll
      for (int r = 0; r < 16; ++r) s[r] = coarse_score(fmaf(s[r], ks, -base), vs);
      ks = 1.0f;
      base = 0.0f;
    }
    base -= (float)(vs + kLift);
    float sum = 0.0f;
    Frag<Fp16> p[2], rest[2];  // tokens 8 i + 0..7 of the granule
#pragma unroll
    for (int r = 0; r < 16; r += 2) {
      const float p0 = __builtin_amdgcn_exp2f(fmaf(s[r], ks, -base));
      const float p1 = __builtin_amdgcn_exp2f(fmaf(s[r + 1], ks, -base));
      sum += p0 + p1;
      two_parts(p0, p1, p[r >> 3].u[(r & 7) >> 1], rest[r >> 3].u[(r & 7) >> 1]);
    }
    l += ldexpf(sum, -vs);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const uint4 v = *reinterpret_cast<const uint4*>(vb + 2048 * i + v_off[j]);
      const v8h v0 = dec8<Fp16>(v.x, v.y, 1.0f);
      acc[i] = Fp16::mfma32(v0, rest[0].v, acc[i]);
      acc[i] = Fp16::mfma32(v0, p[0].v, acc[i]);
      const v8h v1 = dec8<Fp16>(v.z, v.w, 1.0f);
      acc[i] = Fp16::mfma32(v1, rest[1].v, acc[i]);
      acc[i] = Fp16::mfma32(v1, p[1].v, acc[i]);
    }
  };
  // waits for tile `it`, lets the next one start and gives the tile's pages and scales
  auto advance = [&](int it, int t0, int(&vid)[2], float(&ks)[2], int(&vs)[2]) __attribute__((always_inline)) {
    if ((it & 15) == 0) pages.settle();
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      vid[j] = pages.gone(it, 2 * h + j);
      ks[j] = pages.kscale(it, 2 * h + j) * a.scale2;
      vs[j] = pages.vshift(it, 2 * h + j);
    }
    wait_loads<0>();
    __syncthreads();
    if (it + 1 < count) {
      if (((it + 1) & 15) == 0) pages.load<D>(a.c, blk.b, kvh, t0 + kv::kTile, kv::kTile, seen_lo, blk.range.hi);
      issue(it + 1, lds + ((it + 1) & 1) * tile_bytes(D));
    }
  };
  // Tiles [whole_begin, whole_end), which all rows of the block see whole, run in a loop of their own, the others
  // with the masks (one loop with a branch kept two copies of the accumulators: 250 registers spilled).
  // With an absent page anywhere there are none.
  int64_t last = (int64_t)blk.r0 + kBlock - 1;
  const int64_t all = (int64_t)(blk.rows.n < a.max_q_len ? blk.rows.n : a.max_q_len) * a.group;
  last = last < all ? last : all - 1;
  const Row row0 = row_at(a, blk.r0, kvh, blk.rows.n, blk.len, room);
  const Row row1 = row_at(a, (int)last, kvh, blk.rows.n, blk.len, room);
  const int any_lo = row0.lo, any_hi = row1.hi;
  int whole_begin = 0, whole_end = count;
  {
    bool absent = false;
    const int end = first + kv::kTile * count < blk.range.hi ? first + kv::kTile * count : blk.range.hi;
    for (int64_t t = (int64_t)first + 16 * lane; t < end; t += 1024) absent = absent || kv::page_of(a.c, blk.b, (int)t) < 0;
    const int upto = row0.hi > first ? (row0.hi - first) / kv::kTile : 0;
    if (row1.lo > first) whole_begin = (row1.lo - first + kv::kTile - 1) / kv::kTile;
    whole_begin = whole_begin < count ? whole_begin : count;
    whole_end = __ballot(absent) ? 0 : (upto < count ? upto : count);
    whole_end = whole_end < whole_begin ? whole_begin : whole_end;
    whole_begin = __builtin_amdgcn_readfirstlane(whole_begin);
    whole_end = __builtin_amdgcn_readfirstlane(whole_end);
  }
  uint32_t bad[(D + 63) / 64] = {};  // accumulators (by number) whose row has seen a NaN of V
  auto masked_tiles = [&](int from, int to) __attribute__((always_inline)) {
    for (int it = from; it < to; ++it) {
      const int t0 = first + kv::kTile * it;
      const uint8_t* kb = smem + (it & 1) * tile_bytes(D);
      const int vgran = pages.gone(it, loads.v_gran);
      int vid[2], vs[2];
      float ks[2];
      advance(it, t0, vid, ks, vs);
      // V's codes that no row sees, and NaN codes, become 0 in LDS (a probability of 0 must not meet them); which
      // were NaN is kept for the rows that see them
      uint32_t found = 0;
      for (int n = wave; n < D / 16; n += 4) {
        v4u* at = reinterpret_cast<v4u*>(smem + (it & 1) * tile_bytes(D) + 64 * D + 1024 * n + 16 * lane);
        v4u v = *at;
        const int t = t0 + 16 * loads.v_gran;
        const uint32_t bits = hide_codes(v, vgran < 0 ? 16 : any_lo - t, any_hi - t);
        *at = v;
        sh_nan[(16 * n + loads.v_col) * 4 + loads.v_gran] = (uint16_t)bits;
        found |= bits;
      }
      const bool poisoned = __syncthreads_or(found != 0);
#pragma unroll
      for (int j = 0; j < 2; ++j) half_tile(std::true_type(), j, t0, kb, vid[j], ks[j], vs[j]);
      if (poisoned) {
        const unsigned long long seen = seen_bits(row, t0);
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            if (nan_map(sh_nan + (32 * i + 8 * (r >> 2) + 4 * h + (r & 3)) * 4) & seen)
              bad[i >> 1] |= 1u << (16 * (i & 1) + r);
      }
    }
  };
  masked_tiles(0, whole_begin);
  for (int it = whole_begin; it < whole_end; ++it) {
    const int t0 = first + kv::kTile * it;
    const uint8_t* kb = smem + (it & 1) * tile_bytes(D);
    int vid[2], vs[2];
    float ks[2];
    advance(it, t0, vid, ks, vs);
#pragma unroll
    for (int j = 0; j < 2; ++j) half_tile(std::false_type(), j, t0, kb, vid[j], ks[j], vs[j]);
  }
  masked_tiles(whole_end, count);
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r)
      if (bad[i >> 1] >> (16 * (i & 1) + r) & 1) acc[i][r] = __builtin_nanf("");

  l += __shfl_xor(l, 32, 64);
  l *= 1.0f / (1 << kLift);
  const float unit = pages.unit();
  if (row.i < 0) return;
  if (parts == 1) {
    const float inv = l == 0.0f ? 0.0f : unit / l;
    const int64_t out = (int64_t)(blk.rows.first + row.i);
    uint16_t* yr = a.y + out * a.yt + (int64_t)row.head * a.yh;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int r = 0; r < 16; r += 4)
        *reinterpret_cast<uint2*>(yr + 32 * i + 2 * r + 4 * h) = make_uint2(
            E::pack(acc[i][r] * inv, acc[i][r + 1] * inv), E::pack(acc[i][r + 2] * inv, acc[i][r + 3] * inv));
    if (h == 0 && a.lse) a.lse[out * a.q_heads + row.head] = (m + __builtin_amdgcn_logf(l)) * kLn2;
  } else {
    const int64_t slot = (((id * a.c.heads + kvh) * a.splits + blockIdx.y) * kBlock) + 32 * wave + col;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
#pragma unroll
      for (int r = 0; r < 16; r += 4)
        *reinterpret_cast<float4*>(a.part_o + slot * D + 32 * i + 2 * r + 4 * h) =
            make_float4(acc[i][r] * unit, acc[i][r + 1] * unit, acc[i][r + 2] * unit, acc[i][r + 3] * unit);
    if (h == 0) {
      a.part_ml[slot * 2] = m;
      a.part_ml[slot * 2 + 1] = l;
    }
  }
}

// joins the parts of a block: a thread takes four elements of a row, the parts in order
template <class E, int D>
__global__ __launch_bounds__(256) void attn_prompt_join(Args a) {
  constexpr int LANES = D / 4;
  const int kvh = blockIdx.x % a.c.heads;
  const int64_t id = blockIdx.x / a.c.heads;
  Block blk;
  if (!find_block(a, id, blk)) return;
  const int parts = parts_of(a, kv::tiles_of(blk.range));
  if (parts == 1) return;
  const int i = blockIdx.y * 256 + threadIdx.x, r = i / LANES, d = 4 * (i % LANES);
  const Row row = row_at(a, blk.r0 + r, kvh, blk.rows.n, blk.len, room_of(a.c));
  if (row.i < 0) return;
  const int64_t first = ((id * a.c.heads + kvh) * a.splits) * kBlock + r;
  float M = -INFINITY;
  for (int p = 0; p < parts; ++p) M = fmaxf(M, a.part_ml[(first + (int64_t)p * kBlock) * 2]);
  const float base = M == -INFINITY ? 0.0f : M;
  float o[4] = {0.0f, 0.0f, 0.0f, 0.0f}, L = 0.0f;
  for (int p = 0; p < parts; ++p) {
    const int64_t at = first + (int64_t)p * kBlock;
    const float f = __builtin_amdgcn_exp2f(a.part_ml[at * 2] - base);
    const float4 v = *reinterpret_cast<const float4*>(a.part_o + at * D + d);
    L += f * a.part_ml[at * 2 + 1];
    o[0] += f * v.x;
    o[1] += f * v.y;
    o[2] += f * v.z;
    o[3] += f * v.w;
  }
  const float inv = L == 0.0f ? 0.0f : 1.0f / L;
  const int64_t out = (int64_t)(blk.rows.first + row.i);
  uint16_t* yr = a.y + out * a.yt + (int64_t)row.head * a.yh;
  *reinterpret_cast<uint2*>(yr + d) = make_uint2(E::pack(o[0] * inv, o[1] * inv), E::pack(o[2] * inv, o[3] * inv));
  if (d == 0 && a.lse) a.lse[out * a.q_heads + row.head] = (M + __builtin_amdgcn_logf(L)) * kLn2;
}

template <class E, int D>
hipError_t launch(const Args& a, hipStream_t s) {
  static std::atomic<unsigned long long> raised{0};
  hipError_t e = ensure_lds_limit(reinterpret_cast<const void*>(attn_prompt<E, D>), prompt_lds(D), raised);
  if (e != hipSuccess) return e;
  const unsigned blocks = (unsigned)(kv::prompt_blocks(a.T, a.c.batch, a.group) * a.c.heads);
  hipLaunchKernelGGL((attn_prompt<E, D>), dim3(blocks, (unsigned)a.splits), dim3(256),
                     prompt_lds(D), s, a);
  e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  hipLaunchKernelGGL((attn_prompt_join<E, D>), dim3(blocks, kBlock * D / 4 / 256), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_prompt(bsq_dtype dt, const attn::Args& a, hipStream_t s) {
  const bool half = dt == BSQ_FP16;
  switch (a.c.dim) {
    case 64: return half ? launch<Fp16, 64>(a, s) : launch<Bf16, 64>(a, s);
    case 128: return half ? launch<Fp16, 128>(a, s) : launch<Bf16, 128>(a, s);
    default: return half ? launch<Fp16, 256>(a, s) : launch<Bf16, 256>(a, s);
  }
}

}  // namespace bsq
