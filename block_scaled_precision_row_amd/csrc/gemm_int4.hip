// Few-token linears with 4-bit integer weights and group scales:
//   y[m][n] = sum_g s[n][g] * sum_{k in g} x[m][k] (c[n][k] - z[n][g]).
//
// Codes become 16-bit numbers by or-ing them into the mantissa of a power of two:
//   fp16: 1024 + c, from which a packed subtraction of 1024 + z leaves c - z exactly;
//   bf16 (no packed arithmetic): 128 + c stays, and (128 + z) times the sum of x over the group is taken away in
//   fp32.
// The order of nibbles in a dword gives pairs (k, k + 4); x is put in the same order. A group's sum is complete in
// fp32 before its scale is applied.
//
// The floor is memory: K / 2 bytes a row and its scales (cold: 1 x 16384 x 8192 18.9 us, 3.9 TB/s; 1 x 4096 x 4096
// 5.2 us, of which a launch is 3). With more tokens the compute units are half empty: what a workgroup stages takes 90 KB
// of LDS (two tiles of 32 rows and tokens to each of eight waves), so that one fits a unit, two waves a SIMD, which keep
// the vector units 40 % busy, and the last round of workgroups fills what it fills (24 x 12288 x 4096 in groups of 32: 24 us,
// 384 workgroups of 32 rows on 256 units).
//
// From 33 tokens on, two tiles of 16 rows and four of 16 tokens need more than a wave's 256 registers: 6 to 9 are
// spilled, in groups of 32 19 (fp16) and 83 (bf16); with one tile of rows none, or 3 (48 x 8192 x 8192: 39.4 us with
// two and 48.9 with one).
#include <type_traits>

#include "bsq_launch.hpp"
#include "serve_device.hpp"

namespace bsq {

namespace {

struct Args {
  const uint16_t* x;
  int64_t ldx;
  const uint8_t* w;
  const uint16_t* ws;
  const uint8_t* wz;
  uint16_t* y;
  int64_t ldy;
  int64_t M, N;
  int K;
};

template <class E>
union Frag {
  typename E::vec8 v;
  typename E::vec2 p[4];
  uint32_t u[4];
  uint4 q;
};

// the eight values of a dword as pairs (k, k + 4)
template <class E>
__device__ __forceinline__ typename E::vec8 codes8(uint32_t w, uint32_t minus) {
  // (the constants from registers, so that mask and magic number are one instruction: a three-operand one takes no
  // literal)
  uint32_t mask = 0x000F000Fu, magic = E::is_half ? 0x64006400u : 0x43004300u;
  asm("" : "+s"(mask));
  asm("" : "+v"(magic));
  Frag<E> f;
#pragma unroll
  for (int i = 0; i < 4; ++i) f.u[i] = ((w >> (4 * i)) & mask) | magic;
  if constexpr (E::is_half) {
    union { uint32_t u; v2h h; } c;
    c.u = minus;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      union { uint32_t u; v2h h; } t;
      t.u = f.u[i];
      t.h = t.h - c.h;
      f.u[i] = t.u;
    }
  }
  return f.v;
}
template <class E>
__device__ __forceinline__ typename E::vec8 paired(uint4 x) {
  Frag<E> f;
  f.u[0] = __builtin_amdgcn_perm(x.z, x.x, 0x05040100u);
  f.u[1] = __builtin_amdgcn_perm(x.z, x.x, 0x07060302u);
  f.u[2] = __builtin_amdgcn_perm(x.w, x.y, 0x05040100u);
  f.u[3] = __builtin_amdgcn_perm(x.w, x.y, 0x07060302u);
  return f.v;
}

// ---- three tokens and more: 16-row tiles on the matrix units ------------------------------
// A workgroup takes RT tiles of 16 rows, each of its eight waves every eighth stage of 128 K values on 16x16x32 MFMA
// (A: x, B: W), joined through LDS in order at the end. (A stage of x shared by two or four waves, with the codes
// four stages ahead: 5 x 16384 x 8192 40 us against 28, for x is then reordered per row tile.)
//
// What a wave reads of one stage, as it loads it: whole segments of rows by neighbouring lanes (the four lanes
// 4 i .. 4 i + 3 read row i's 64 bytes of codes, 16 lanes a token's 256 bytes of x). With the operands' own order
// (neighbouring lanes on neighbouring rows) the address unit took 49 cycles an instruction and bounded
// the kernel (24 x 12288 x 4096: 28 us). Past K a lane reads what lies before it (those blocks are
// skipped); rows past M or N read the last one (their results are not stored).
template <int TM, int RT, int GROUP>
struct Stage {
  static constexpr int G = 128 / GROUP;
  v4u w[RT];  // (a built-in vector: copies of the class type go through scratch memory)
  v4u x[4 * TM];
  uint32_t s[(G + 1) / 2], z;  // lanes 16 r .. 16 r + 15: row tile r's scales and zero points
};
// LDS of a wave: rows padded so that the operand reads are free of bank conflicts
constexpr int kWPitch = 80, kXPitch = 272;
template <int TM, int RT>
constexpr int wave_lds() {
  return 16 * RT * kWPitch + 16 * TM * kXPitch;
}
template <int TM, int RT, int WAVES>
constexpr int mfma_lds() {
  const int stage = WAVES * wave_lds<TM, RT>(), join = WAVES * RT * TM * 1024;
  return stage > join ? stage : join;
}
__device__ __forceinline__ void wave_lds_fence() {  // LDS written by other lanes of the wave is there
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <class E, int TM, int RT, int GROUP, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void int4_mfma(Args a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  constexpr int G = 128 / GROUP;
  typedef Stage<TM, RT, GROUP> S;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 15, kq = lane >> 4;
  uint8_t* sw = smem + wave * wave_lds<TM, RT>();
  uint8_t* sx = sw + 16 * RT * kWPitch;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * RT), m0 = (int64_t)blockIdx.y * (16 * TM);
  const int groups = a.K / GROUP;
  // each row's scales of a stage in one load
  const bool wide = groups % G == 0 && (reinterpret_cast<uintptr_t>(a.ws) & (2 * G - 1)) == 0 &&
                    (reinterpret_cast<uintptr_t>(a.wz) & (G - 1)) == 0;
  const uint8_t* wr[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int64_t n = n0 + 16 * r + (lane >> 2);
    wr[r] = a.w + (n < a.N ? n : a.N - 1) * (a.K / 2);
  }
  const int64_t ns = n0 + lane < a.N ? n0 + lane : a.N - 1;  // row whose scales this lane loads
  const uint16_t* sr = a.ws + ns * groups;
  const uint8_t* zr = a.wz + ns * groups;
  const uint16_t* xr[4 * TM];
#pragma unroll
  for (int t = 0; t < 4 * TM; ++t) {
    const int64_t m = m0 + 4 * t + kq;
    xr[t] = a.x + (m < a.M ? m : a.M - 1) * a.ldx;
  }
  Frag<E> ones;
  ones.q = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
  v4f acc[RT][TM];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < TM; ++t) acc[r][t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  auto fetch = [&](int k0, S& o) __attribute__((always_inline)) {
    const int kw = k0 + 32 * (lane & 3) < a.K - 32 ? k0 + 32 * (lane & 3) : a.K - 32;
    const int kx = k0 + 8 * col < a.K - 8 ? k0 + 8 * col : a.K - 8;
#pragma unroll
    for (int r = 0; r < RT; ++r) o.w[r] = *reinterpret_cast<const v4u*>(wr[r] + (kw >> 1));
#pragma unroll
    for (int t = 0; t < 4 * TM; ++t) o.x[t] = *reinterpret_cast<const v4u*>(xr[t] + kx);
    const int gi = k0 / GROUP;
    if (lane < 16 * RT) {
      if (wide) {
        if constexpr (G == 4) {
          const uint2 v = *reinterpret_cast<const uint2*>(sr + gi);
          o.s[0] = v.x;
          o.s[1] = v.y;
          o.z = a.wz ? *reinterpret_cast<const uint32_t*>(zr + gi) : 0u;
        } else if constexpr (G == 2) {
          o.s[0] = *reinterpret_cast<const uint32_t*>(sr + gi);
          o.z = a.wz ? *reinterpret_cast<const uint16_t*>(zr + gi) : 0u;
        } else {
          o.s[0] = sr[gi];
          o.z = a.wz ? zr[gi] : 0u;
        }
      } else {
        o.z = 0;
#pragma unroll
        for (int i = 0; i < G; ++i) {
          const int at = gi + i < groups ? gi + i : groups - 1;
          const uint32_t v = sr[at];
          o.s[i >> 1] = i & 1 ? o.s[i >> 1] | v << 16 : v;
          if (a.wz) o.z |= (uint32_t)zr[at] << (8 * i);
        }
      }
    }
  };
  auto compute = [&](auto partial, int k0, const S& cur) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < RT; ++r)
      *reinterpret_cast<v4u*>(sw + (16 * r + (lane >> 2)) * kWPitch + 16 * (lane & 3)) = cur.w[r];
#pragma unroll
    for (int t = 0; t < 4 * TM; ++t) *reinterpret_cast<v4u*>(sx + (4 * t + kq) * kXPitch + 16 * col) = cur.x[t];
    wave_lds_fence();
#pragma unroll
    for (int e0 = 0; e0 < 4; e0 += GROUP / 32) {
      if (partial && k0 + 32 * e0 >= a.K) continue;
      v4f c[RT][TM], cx[TM];
#pragma unroll
      for (int t = 0; t < TM; ++t) {
        cx[t] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int r = 0; r < RT; ++r) c[r][t] = cx[t];
      }
      constexpr int kPer = GROUP / 32;
      const int gi = e0 / kPer;
      float s[RT], z[RT];
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        s[r] = E::up((uint32_t)__shfl((int)cur.s[gi >> 1], 16 * r + col, 64) >> (16 * (gi & 1)) & 0xFFFFu);
        z[r] = a.wz ? (float)((uint32_t)__shfl((int)cur.z, 16 * r + col, 64) >> (8 * gi) & 0xFFu) : 8.0f;
      }
#pragma unroll
      for (int e = e0; e < e0 + kPer; ++e) {
        typename E::vec8 wf[RT];
#pragma unroll
        for (int r = 0; r < RT; ++r)
          wf[r] = codes8<E>(*reinterpret_cast<const uint32_t*>(sw + (16 * r + col) * kWPitch + 16 * e + 4 * kq),
                            E::is_half ? E::pack(1024.0f + z[r], 1024.0f + z[r]) : 0u);
#pragma unroll
        for (int t = 0; t < TM; ++t) {
          const typename E::vec8 xf =
              paired<E>(*reinterpret_cast<const uint4*>(sx + (16 * t + col) * kXPitch + 64 * e + 16 * kq));
          if constexpr (!E::is_half) cx[t] = E::mfma(xf, ones.v, cx[t]);
#pragma unroll
          for (int r = 0; r < RT; ++r) c[r][t] = E::mfma(xf, wf[r], c[r][t]);
        }
      }
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int t = 0; t < TM; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[r][t][i] = fmaf(s[r], E::is_half ? c[r][t][i] : fmaf(-(128.0f + z[r]), cx[t][i], c[r][t][i]), acc[r][t][i]);
    }
    wave_lds_fence();  // read before the next stage is written
  };
  // the walk over K starts at a place of the workgroup's own: rows lie a power of two apart more often
  // than not, and workgroups in step would all read from the same few memory channels
  constexpr int kStep = 128 * WAVES;
  const int span = (a.K + 127) / 128 * 128, turn = (int)(blockIdx.x * 7u % (unsigned)(span / 128)) * 128;
  auto place = [&](int k) { return k + turn < span ? k + turn : k + turn - span; };
  S next;
  if (128 * wave < span) fetch(place(128 * wave), next);
  for (int k = 128 * wave; k < span; k += kStep) {
    S cur;
    cur = next;
    if (k + kStep < span) fetch(place(k + kStep), next);
    const int at = place(k);
    if (at + 128 <= a.K) compute(std::false_type(), at, cur);
    else compute(std::true_type(), at, cur);
  }
  __syncthreads();
  float* sh = reinterpret_cast<float*>(smem);  // [wave][tile][lane][4]
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < TM; ++t)
      *reinterpret_cast<float4*>(sh + ((wave * RT * TM + r * TM + t) * 64 + lane) * 4) =
          make_float4(acc[r][t][0], acc[r][t][1], acc[r][t][2], acc[r][t][3]);
  __syncthreads();
  for (int i = wave; i < RT * TM; i += WAVES) {
    float4 v = *reinterpret_cast<const float4*>(sh + (i * 64 + lane) * 4);
#pragma unroll
    for (int w = 1; w < WAVES; ++w) {
      const float4 o = *reinterpret_cast<const float4*>(sh + ((w * RT * TM + i) * 64 + lane) * 4);
      v.x += o.x;
      v.y += o.y;
      v.z += o.z;
      v.w += o.w;
    }
    const int64_t n = n0 + 16 * (i / TM) + col, m = m0 + 16 * (i % TM) + 4 * kq;
    const float out[4] = {v.x, v.y, v.z, v.w};
    if (n < a.N)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (m + j < a.M) a.y[(m + j) * a.ldy + n] = (uint16_t)E::pack(out[j], 0.0f);
  }
}

// ---- one token or two: dot products, lanes along K ------------------------------------
// A lane keeps the 32 x values of its place in a slab of 2048 (16 registers a token) and meets them with
// its 16 bytes of each row: a wave's load of a row is 1 KB without a gap, a lane's values lie in one
// group, so its sum is scaled in its own registers. A wave walks blocks of kRows rows, the next
// block's loads in flight while it works on the present one. The slabs of a row are the waves of one
// workgroup (at most eight, which then take several each), joined through LDS in order at the end.
constexpr int kRows = 4;
constexpr int kMaxBlocks = 16;  // blocks of rows that a wave walks

__device__ __forceinline__ float dot2(v2bf a, v2bf b, float c) { return __builtin_amdgcn_fdot2_f32_bf16(a, b, c, false); }
__device__ __forceinline__ float dot2(v2h a, v2h b, float c) { return __builtin_amdgcn_fdot2(a, b, c, false); }

template <int ctrl>
__device__ __forceinline__ float add_rotated(float v) {
  return v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), ctrl, 0xF, 0xF, false));
}
// four values' sums over the wave: lane l ends up with that of value l / 16
__device__ __forceinline__ float sum4(float (&v)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[i]), __float_as_uint(v[i + 2]), false, false);
    v[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  }
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v[0]), __float_as_uint(v[1]), false, false);
  float o = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  o = add_rotated<0x128>(o);  // row_ror within 16 lanes: 8, 4, 2, 1
  o = add_rotated<0x124>(o);
  o = add_rotated<0x122>(o);
  return add_rotated<0x121>(o);
}

template <class E, int TM>
__global__ __launch_bounds__(512) void int4_dot(Args a, int shift, int per_row, int row_sets, int blocks) {
  extern __shared__ float shd[];  // [wave][block][TM][kRows]
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int part = wave % per_row, set = wave / per_row;
  const int64_t n0 = ((int64_t)blockIdx.x * row_sets + set) * blocks * kRows;
  const int groups = a.K >> shift;
  const int span = 2048 * per_row, chunks = (a.K + span - 1) / span;  // of K, per block
  const int steps = blocks * chunks;

  struct Block {
    uint4 w[kRows];
    uint16_t s[kRows];
    uint8_t z[kRows];
  };
  auto fetch = [&](int block, int chunk, Block& o) {
    const int k = chunk * span + 2048 * part + 32 * lane;
    const bool in = k < a.K;
    const int gi = in ? k >> shift : 0;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const int64_t row = n0 + block * kRows + r;
      const int64_t n = row < a.N ? row : a.N - 1;
      o.w[r] = make_uint4(0, 0, 0, 0);
      if (in) o.w[r] = *reinterpret_cast<const uint4*>(a.w + n * (a.K / 2) + (k >> 1));
      o.s[r] = a.ws[n * groups + gi];
      o.z[r] = a.wz ? a.wz[n * groups + gi] : 8;
    }
  };
  Frag<E> x[TM][4];
  float sum[TM];
  auto fetch_x = [&](int chunk) {
    const int k = chunk * span + 2048 * part + 32 * lane;
#pragma unroll
    for (int t = 0; t < TM; ++t) {
      sum[t] = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (k < a.K && t < a.M) u = *reinterpret_cast<const uint4*>(a.x + t * a.ldx + k + 8 * i);
        x[t][i].v = paired<E>(u);
        if constexpr (!E::is_half)
#pragma unroll
          for (int j = 0; j < 4; ++j) sum[t] += E::lo(x[t][i].u[j]) + E::hi(x[t][i].u[j]);
      }
    }
  };
  float v[TM][kRows];
#pragma unroll
  for (int t = 0; t < TM; ++t)
#pragma unroll
    for (int r = 0; r < kRows; ++r) v[t][r] = 0.0f;
  Block next;
  fetch(0, 0, next);
  fetch_x(0);
  int block = 0, chunk = 0;
  for (int i = 0; i < steps; ++i) {
    Block b = next;
    const int nc = chunk + 1 < chunks ? chunk + 1 : 0, nb = nc ? block : block + 1;
    if (i + 1 < steps) fetch(nb, nc, next);
    const bool in = chunk * span + 2048 * part + 32 * lane < a.K;
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const uint32_t d[4] = {b.w[r].x, b.w[r].y, b.w[r].z, b.w[r].w};
      const float zf = (float)b.z[r];
      const uint32_t minus = E::is_half ? E::pack(1024.0f + zf, 1024.0f + zf) : 0u;
      float c[TM];
#pragma unroll
      for (int t = 0; t < TM; ++t) c[t] = 0.0f;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        Frag<E> f;
        f.v = codes8<E>(d[q], minus);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int t = 0; t < TM; ++t) c[t] = dot2(f.p[j], x[t][q].p[j], c[t]);
      }
      const float sf = E::up(b.s[r]);
#pragma unroll
      for (int t = 0; t < TM; ++t) v[t][r] += in ? sf * (E::is_half ? c[t] : c[t] - (128.0f + zf) * sum[t]) : 0.0f;
    }
    if (nc == 0) {
#pragma unroll
      for (int t = 0; t < TM; ++t) {
        const float o = sum4(v[t]);
        if ((lane & 15) == 0) shd[((wave * blocks + block) * TM + t) * kRows + (lane >> 4)] = o;
#pragma unroll
        for (int r = 0; r < kRows; ++r) v[t][r] = 0.0f;
      }
    }
    if (chunks > 1 && i + 1 < steps) fetch_x(nc);
    block = nb;
    chunk = nc;
  }
  __syncthreads();
  const int rows = blocks * kRows;  // of a row set
  for (int i = threadIdx.x; i < row_sets * TM * rows; i += blockDim.x) {
    const int r = i % rows, t = i / rows % TM, q = i / (rows * TM);
    float o = 0.0f;
    for (int p = 0; p < per_row; ++p)
      o += shd[(((q * per_row + p) * blocks + r / kRows) * TM + t) * kRows + r % kRows];
    const int64_t n = ((int64_t)blockIdx.x * row_sets + q) * rows + r;
    if (n < a.N && t < a.M) a.y[t * a.ldy + n] = (uint16_t)E::pack(o, 0.0f);
  }
}

template <class E, int TM, int RT, int GROUP, int WAVES>
hipError_t launch_mfma(const Args& a, hipStream_t s) {
  static std::atomic<unsigned long long> raised{0};
  constexpr int lds = mfma_lds<TM, RT, WAVES>();
  hipError_t e = ensure_lds_limit(reinterpret_cast<const void*>(int4_mfma<E, TM, RT, GROUP, WAVES>), lds, raised);
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)((a.N + 16 * RT - 1) / (16 * RT)), (unsigned)((a.M + 16 * TM - 1) / (16 * TM)));
  hipLaunchKernelGGL((int4_mfma<E, TM, RT, GROUP, WAVES>), grid, dim3(64 * WAVES), lds, s, a);
  return hipGetLastError();
}
template <class E, int TM, int RT, int WAVES>
hipError_t launch(const Args& a, int group, hipStream_t s) {
  if (group == 32) return launch_mfma<E, TM, RT, 32, WAVES>(a, s);
  return group == 64 ? launch_mfma<E, TM, RT, 64, WAVES>(a, s) : launch_mfma<E, TM, RT, 128, WAVES>(a, s);
}
template <class E, int TM>
hipError_t launch_dot(const Args& a, int group, hipStream_t s) {
  const int slabs = (a.K + 2047) / 2048, per_row = slabs < 8 ? slabs : 8, sets = per_row >= 4 ? 1 : 4 / per_row;
  // about four waves a SIMD, each walking its blocks
  const int64_t all = (a.N + (int64_t)sets * kRows - 1) / (sets * kRows);
  const int64_t room = 4096 / (per_row * sets);
  int64_t blocks = (all + room - 1) / room;
  blocks = blocks < 1 ? 1 : (blocks > kMaxBlocks ? kMaxBlocks : blocks);
  hipLaunchKernelGGL((int4_dot<E, TM>), dim3((unsigned)((all + blocks - 1) / blocks)), dim3(64 * per_row * sets),
                     sizeof(float) * per_row * sets * blocks * TM * kRows, s, a, __builtin_ctz(group), per_row, sets,
                     (int)blocks);
  return hipGetLastError();
}
// Two row tiles to a wave share its x; with few rows one, so that more units work (8 x 4096 x 4096: 7.3 us
// with one, 8.2 with two; 5 x 16384 x 8192: 33.6 and 29.2, 48 x 8192 x 8192: 48.9 and 39.4).
template <class E, int TM>
hipError_t launch_rows(const Args& a, int group, hipStream_t s) {
  return a.N <= 6144 ? launch<E, TM, 1, 8>(a, group, s) : launch<E, TM, 2, 8>(a, group, s);
}
template <class E>
hipError_t launch_tokens(const Args& a, int group, hipStream_t s) {
  // Dot products up to two tokens, the matrix units above (bf16, dot against matrix units: 16384 x 8192 groups of 64,
  // 1 token 18.9 and 27.2 us, 2: 23.7 and 27.4, 3: 30.2 and 26.8; 12288 x 4096 groups of 32, 2: 11.3 and 18.3, 3:
  // 15.9 and 18.5; 4096 x 4096 groups of 128, 2: 6.5 and 7.0, 3: 8.0 and 7.0).
  if (a.M == 1) return launch_dot<E, 1>(a, group, s);
  if (a.M == 2) return launch_dot<E, 2>(a, group, s);
  if (a.M <= 16) return launch_rows<E, 1>(a, group, s);
  if (a.M <= 32) return launch_rows<E, 2>(a, group, s);
  return launch_rows<E, 4>(a, group, s);
}

}  // namespace

hipError_t launch_gemm_int4g(bsq_dtype dt, const Int4Args& p, hipStream_t s) {
  const Args a{static_cast<const uint16_t*>(p.x), p.ldx, p.w, static_cast<const uint16_t*>(p.ws), p.wz,
               static_cast<uint16_t*>(p.y), p.ldy, p.M, p.N, p.K};
  return dt == BSQ_FP16 ? launch_tokens<Fp16>(a, p.group, s) : launch_tokens<Bf16>(a, p.group, s);
}

}  // namespace bsq
