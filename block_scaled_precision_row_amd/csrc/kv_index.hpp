// Index arithmetic of the paged E4M3 key/value cache (include/bsq_serve.h), shared by the
// kernels and, compiled for the host, by the audit that enumerates it on the CPU: everything that
// turns device-side lengths and page tables into addresses is here, and clamps what it reads, so
// that no table or length leads outside the tensors of a call.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bsq {
namespace kv {

#define BSQ_HD __host__ __device__ __forceinline__

struct Cache {
  uint8_t* k;            // [pages][heads][page][dim]
  uint8_t* v;            // [pages][heads][dim][page]
  float* ks;             // [pages][heads]
  float* vs;
  const int32_t* table;  // [batch][table_stride]
  const int32_t* lens;   // [batch]
  int64_t table_stride;
  int num_pages, heads, shift;  // page size 1 << shift
  int dim, batch, max_pages;
};

constexpr int kTile = 64;  // tokens that a wave of the attention kernels takes at once

// rows of sequence b in the packed tensors
struct Rows {
  int first, n;
};
BSQ_HD Rows rows_of(const int32_t* cu, int b, int64_t T) {
  const int t = (int)T;
  int lo = cu[b], hi = cu[b + 1];
  lo = lo < 0 ? 0 : (lo > t ? t : lo);
  hi = hi < lo ? lo : (hi > t ? t : hi);
  return Rows{lo, hi - lo};
}

// The last b in [0, n) for which a condition holds that holds for a prefix, -1 if for none: `count(lo, step, n)` says
// for how many of lo, lo + step, ... (below lo + n, at most WIDTH of them) it does. Where it holds for no prefix
// (starts that decrease) the result is some b in range, and what is made of it has to be checked.
template <int WIDTH, class Count>
BSQ_HD int last_of(int n, Count count) {
  int lo = 0;
  while (true) {
    const int step = (n + WIDTH - 1) / WIDTH, cnt = count(lo, step, n);
    if (cnt == 0) return -1;
    const int skip = (cnt - 1) * step;
    lo += skip;
    n = step < n - skip ? step : n - skip;
    if (step == 1) return lo;
  }
}

// the page of sequence b's token t, -1 where it is absent
BSQ_HD int page_of(const Cache& c, int b, int t) {
  const int j = t >> c.shift;
  if (t < 0 || j >= c.max_pages) return -1;
  const int id = c.table[(int64_t)b * c.table_stride + j];
  return id < 0 || id >= c.num_pages ? -1 : id;
}

// offset of a page's codes of one head, in K and in V alike
BSQ_HD int64_t codes_at(const Cache& c, int page, int head) {
  return (((int64_t)page * c.heads + head) << c.shift) * c.dim;
}

// ---- append: one workgroup per touched page --------------------------------------------
// Sequence b's n new tokens touch at most n / page + 2 pages, so giving it the slots from
// first_slot(b) = cu[b] / page + 2 b on leaves room for them: first_slot(b + 1) - first_slot(b)
// >= n / page + 2. A slot's sequence is the last b whose first slot is not behind it.
BSQ_HD int64_t first_slot(const int32_t* cu, int b, int64_t T, int shift) {
  const int t = cu[b];
  return (int64_t)((t < 0 ? 0 : (t > (int)T ? (int)T : t)) >> shift) + 2 * (int64_t)b;
}
BSQ_HD int64_t append_slots(int64_t T, int64_t batch, int shift) { return (T >> shift) + 2 * batch; }

// what slot `first_slot(b) + j` appends: tokens [at, at + n) of page `page` (-1: absent), from row `row` on
struct Touched {
  int page, at, n, row;
};
BSQ_HD Touched touched_page(const Cache& c, const int32_t* cu, int b, int64_t j, int64_t T) {
  const Touched none{-1, 0, 0, 0};
  const Rows r = rows_of(cu, b, T);
  const int64_t len = c.lens[b], past = len - r.n;
  if (r.n == 0 || past < 0) return none;
  if (j < 0) return none;  // (starts that decrease)
  const int64_t start = ((past >> c.shift) + j) << c.shift;
  if (start >= len || (start >> c.shift) >= c.max_pages) return none;
  const int64_t lo = past > start ? past : start;
  const int64_t end = start + ((int64_t)1 << c.shift), hi = len < end ? len : end;
  return Touched{page_of(c, b, (int)start), (int)(lo - start), (int)(hi - lo), (int)(r.first + (lo - past))};
}

// ---- attention: the tokens of a sequence split over workgroups -----------------------------
// Tokens that some row of rows [i0, i0 + rows) of a sequence's n sees: [lo, hi), lo a multiple
// of kTile. `full`: no causal mask.
struct Range {
  int lo, hi;
};
BSQ_HD Range seen_range(int len, int room, int n, int i0, int rows, int64_t window, bool full) {
  int64_t hi = full ? len : (int64_t)len - n + i0 + rows;
  if (hi > len) hi = len;
  if (hi > room) hi = room;
  int64_t lo = 0;
  if (window > 0) lo = (int64_t)len - n + i0 - window + 1;
  if (lo < 0) lo = 0;
  lo = lo / kTile * kTile;
  return hi <= lo ? Range{0, 0} : Range{(int)lo, (int)hi};
}
BSQ_HD int tiles_of(Range r) { return (r.hi - r.lo + kTile - 1) / kTile; }

// The tiles of all sequences, one after the other, are cut into equal runs of `chunk` tiles, one to a
// workgroup, which may end one sequence and begin another. So a batch of any raggedness keeps all workgroups
// equally long, and the host needs to know no length. (The caller keeps the total below 2^31.)
BSQ_HD int chunk_of(int total, int target, int least) {
  const int c = (int)(((unsigned)total + (unsigned)target - 1) / (unsigned)target);
  return c < least ? least : c;
}
BSQ_HD int range_of(int chunk, int x) { return (int)((unsigned)x / (unsigned)chunk); }
// A sequence that lies in several ranges leaves a partial result in each: at most one range begins inside
// it or with it (slot 2 r) for every one but the first, which may hold others before it (slot 2 r + 1).
BSQ_HD int64_t partial_slot(int r, bool at_begin) { return 2 * (int64_t)r + (at_begin ? 0 : 1); }

// ---- prompts: blocks of 128 rows (token, query head of the group) of a sequence and kv head -------
// Blocks of sequence b start at first_block(b) = cu[b] * group / 128 + b; n tokens need at most
// n * group / 128 + 1 of them.
constexpr int kBlock = 128;
BSQ_HD int64_t first_block(const int32_t* cu, int b, int64_t T, int group) {
  const int t = cu[b];
  return (int64_t)(t < 0 ? 0 : (t > (int)T ? (int)T : t)) * group / kBlock + b;
}
BSQ_HD int64_t prompt_blocks(int64_t T, int64_t batch, int64_t group) { return T * group / kBlock + batch; }
// first row of block `id` among the n * group of sequence b; -1 where the block has none (of max_q_len tokens), or the
// sequence has at most `small` rows
BSQ_HD int block_row(const int32_t* cu, int b, const Rows& rows, int64_t T, int group, int64_t id, int small, int max_q_len) {
  const int64_t all = (int64_t)rows.n * group, r0 = (id - first_block(cu, b, T, group)) * kBlock;
  if (r0 < 0) return -1;  // (starts that decrease)
  return all <= small || r0 >= all || r0 / group >= max_q_len ? -1 : (int)r0;
}
// token (of the sequence's n, -1 for none) and query head of row R >= 0. `inverse`: ceil(2^32 / group), with which
// rows below 16 are divided by a group of at most 16; 0: any row and group
struct RowPlace {
  int i, head;
};
BSQ_HD uint32_t inverse_of(int group) { return group == 1 ? 1u : (uint32_t)((((uint64_t)1 << 32) + group - 1) / group); }
BSQ_HD RowPlace row_place(int R, int group, uint32_t inverse, int kvh, int n, int max_q_len) {
  const int i = inverse == 0 ? R / group : (group == 1 ? R : (int)((uint64_t)(uint32_t)R * inverse >> 32));
  return RowPlace{i >= n || i >= max_q_len ? -1 : i, kvh * group + (R - i * group)};
}

// A prompt block's tiles are cut into equal parts.
BSQ_HD int piece_begin(int tiles, int pieces, int i) { return (int)((int64_t)tiles * i / pieces); }

// ---- a tile of 64 tokens of one head in LDS ---------------------------------------------
// K [token][D], then V [D / 16][slot][16 tokens], loaded 1 KB an instruction, lane l's 16 bytes at 16 l.
// What a lane fetches is permuted within a granule (16 tokens) so that neighbouring lanes read
// neighbouring 16-byte pieces of memory, and the operand reads meet no bank conflict: the 16 lanes that a
// 16-byte LDS read serves at once have to fall into different sixteenths of 256 bytes. Those lanes
// are, for the step kernel, tokens 16 g + r (r < 4, g < 4) and, for the prompt kernel, tokens
// 32 h + 4 a + b (h, a < 2, b < 4), at one piece; for V 16 elements at one granule.
enum Kind : int { kStep = 0, kPrompt = 1 };
template <int D, Kind kind>
BSQ_HD int k_flip(int token) {  // pieces of a K row are exchanged by this
  const int gran = token >> 4 & 3;
  if (kind == kStep) {
    if (D == 64) return gran;
    return D == 128 ? (token >> 1 & 1) | gran << 1 : (token & 3) | gran << 2;
  }
  const int half = gran >> 1;
  if (D == 64) return (token >> 2 & 1) | half << 1;
  return D == 128 ? (token >> 1 & 3) | half << 2 : (token & 7) | half << 3;
}
// byte of a granule's K codes that lane `lane` fetches in its load `i` of D / 64, granule `gran`
template <int D, Kind kind>
BSQ_HD int k_source(int i, int gran, int lane) {
  const int at = 1024 * i + 16 * lane, token = at / D, piece = at % D / 16;
  return token * D + 16 * (piece ^ k_flip<D, kind>(16 * gran + token));
}
// where piece `piece` (16 elements) of a token lies in the tile
template <int D, Kind kind>
BSQ_HD int k_at(int token, int piece) {
  return token * D + 16 * (piece ^ k_flip<D, kind>(token));
}
// V: a page holds 1 << run granules of an element side by side (at most a tile's four)
BSQ_HD int v_run(int page_shift) { return page_shift >= 6 ? 2 : page_shift - 4; }
// where the 16 tokens of granule g of element `d` lie in the tile's V
BSQ_HD int v_at(int d, int g, int run) {
  const int c = d & 15, in = (1 << run) - 1;
  return (d >> 4) * 1024 + 16 * (((g >> run) << (4 + run)) + (c << run) + ((g & in) ^ (c << run >> 4)));
}
// granule and element (of 16) that lane `lane` fetches in each of its V loads
struct VSource {
  int gran, col;
};
BSQ_HD VSource v_source(int lane, int run) {
  const int in = (1 << run) - 1, col = lane >> run & 15;
  return VSource{((lane >> (4 + run)) << run) + ((lane & in) ^ (col << run >> 4)), col};
}

}  // namespace kv
}  // namespace bsq
