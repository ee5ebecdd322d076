// Host-side audit of the paged cache's index arithmetic (built and run by tests/test_kv_audit.py;
// no GPU involved): the functions of kv_index.hpp that the append and attention kernels take their
// addresses from, over regular batches and over lengths and tables out of every range.
//  * append: the slots give every touched page of every sequence exactly once, each new token is
//    in exactly one, and rows, page ids and places lie inside their tensors whatever is read;
//  * attention: the tokens that rows see are covered by the ranges exactly once, partial results have slots of
//    their own and are found again, and every page looked up is a page of the pool or absent.
// Prints one line and exits with 1 on the first violation.
#include <cstdio>
#include <cstdlib>
#include <cstdint>
#include <random>
#include <set>
#include <vector>

#include "kv_index.hpp"

using namespace bsq::kv;

namespace {

[[noreturn]] void fail(const char* what, long a, long b, long c, long d) {
  std::printf("VIOLATION %s (%ld %ld %ld %ld)\n", what, a, b, c, d);
  std::exit(1);
}

long g_checked = 0;

int slot_sequence(const Cache& c, const int32_t* cu, int64_t T, int64_t slot) {
  int b = -1;
  for (int i = 0; i < c.batch; ++i)
    if (first_slot(cu, i, T, c.shift) <= slot) b = i;
  return b;
}

void check_append(const Cache& c, const std::vector<int32_t>& cu, int64_t T, bool regular) {
  const int ps = 1 << c.shift;
  const int64_t slots = append_slots(T, c.batch, c.shift);
  std::vector<int> taken((size_t)T, 0);
  std::set<std::pair<int, int64_t>> seen;
  for (int64_t s = 0; s < slots; ++s) {
    const int b = slot_sequence(c, cu.data(), T, s);
    if (b < 0) continue;
    const int64_t j = s - first_slot(cu.data(), b, T, c.shift);
    const Touched t = touched_page(c, cu.data(), b, j, T);
    if (t.page < 0) continue;
    ++g_checked;
    if (t.page >= c.num_pages) fail("page outside the pool", t.page, c.num_pages, b, s);
    if (t.n < 1 || t.at < 0 || t.at + t.n > ps) fail("tokens outside the page", t.at, t.n, b, s);
    if (t.row < 0 || t.row + t.n > T) fail("rows outside the tensor", t.row, t.n, b, s);
    if (!seen.insert({b, j}).second) fail("a page twice", b, j, s, 0);
    for (int i = 0; i < t.n; ++i) taken[(size_t)(t.row + i)]++;
  }
  if (!regular) return;
  for (int b = 0; b < c.batch; ++b) {
    const int n = cu[b + 1] - cu[b];
    for (int i = 0; i < n; ++i) {
      const int64_t pos = (int64_t)c.lens[b] - n + i;
      const bool want = (int64_t)c.lens[b] >= n && page_of(c, b, (int)pos) >= 0;
      if (taken[(size_t)(cu[b] + i)] != (want ? 1 : 0)) fail("a token not appended once", b, i, taken[(size_t)(cu[b] + i)], want);
    }
  }
  for (int64_t t = cu[c.batch]; t < T; ++t)
    if (taken[(size_t)t]) fail("a row of no sequence appended", t, 0, 0, 0);
}

void check_attention(const Cache& c, const std::vector<int32_t>& cu, int64_t T, int64_t window, bool full, int target,
                     int least) {
  const int room = c.max_pages << c.shift;
  int64_t total = 0;
  std::vector<int> tiles((size_t)c.batch, -1);
  std::vector<Range> range((size_t)c.batch);
  for (int b = 0; b < c.batch; ++b) {
    const int n = rows_of(cu.data(), b, T).n;
    if (n == 0) continue;
    const int len = c.lens[b] < 0 ? 0 : c.lens[b];
    range[b] = seen_range(len, room, n, 0, n, window, full);
    tiles[b] = tiles_of(range[b]);
    if (range[b].lo % kTile || range[b].lo < 0 || range[b].hi > room || tiles[b] < 0) fail("range", b, range[b].lo, range[b].hi, room);
    for (int i = 0; i < n; ++i) {  // what a row sees lies inside
      const int64_t pos = (int64_t)len - n + i;
      int64_t hi = full ? len : pos + 1, lo = window > 0 ? pos - window + 1 : 0;
      hi = hi > room ? room : hi;
      lo = lo < 0 ? 0 : lo;
      if (hi > lo && (lo < range[b].lo || hi > range[b].hi)) fail("a row sees past the range", b, i, lo, hi);
    }
    total += tiles[b];
  }
  for (int b = 0; b < c.batch; ++b)
    for (int t = range[b].lo; tiles[b] > 0 && t < range[b].hi && t < range[b].lo + 4096; t += 16) {
      const int id = page_of(c, b, t);
      if (id < -1 || id >= c.num_pages) fail("page outside the pool", b, t, id, 0);
    }
  if (total == 0) return;
  // the ranges as the workgroups walk them: every tile of every sequence once, partial results in slots of
  // their own, and the joining looks for exactly those
  const int chunk = chunk_of((int)total, target, least);
  const int ranges = range_of(chunk, (int)total - 1) + 1;
  if (ranges < 1 || ranges > target) fail("ranges", ranges, target, total, chunk);
  std::vector<int64_t> before((size_t)c.batch + 1, 0);
  for (int b = 0; b < c.batch; ++b) before[b + 1] = before[b] + (tiles[b] > 0 ? tiles[b] : 0);
  std::set<int64_t> slots;
  std::vector<std::set<int64_t>> left((size_t)c.batch);
  std::vector<int64_t> done((size_t)c.batch, 0);
  for (int r = 0; r < ranges; ++r) {
    const int64_t begin = (int64_t)r * chunk, end = begin + chunk < total ? begin + chunk : total;
    for (int64_t x = begin; x < end;) {
      int b = 0;
      while (before[b + 1] <= x) ++b;
      const int64_t t0 = x - before[b], t1 = end - x < tiles[b] - t0 ? t0 + (end - x) : tiles[b];
      if (t0 != done[b] || t1 <= t0) fail("tiles not in turn", b, t0, t1, done[b]);
      done[b] = t1;
      if (!(t0 == 0 && t1 == tiles[b])) {
        const int64_t s = partial_slot(r, x == begin);
        if (s < 0 || s >= 2 * (int64_t)target || !slots.insert(s).second) fail("slot", b, r, s, 0);
        left[b].insert(s);
      }
      if (range_of(chunk, (int)x) != r || range_of(chunk, (int)(x + (t1 - t0) - 1)) != r) fail("range of a tile", b, r, x, 0);
      x += t1 - t0;
      ++g_checked;
    }
  }
  for (int b = 0; b < c.batch; ++b) {
    if (tiles[b] <= 0) continue;
    if (done[b] != tiles[b]) fail("tiles left out", b, done[b], tiles[b], 0);
    const int r0 = range_of(chunk, (int)before[b]), r1 = range_of(chunk, (int)before[b + 1] - 1);
    std::set<int64_t> want;
    if (r0 != r1)
      for (int r = r0; r <= r1; ++r) want.insert(partial_slot(r, r > r0 || before[b] == (int64_t)r0 * chunk));
    if (want != left[b]) fail("the join looks elsewhere", b, r0, r1, (long)left[b].size());
  }
}

// One tile in LDS: every byte of the 64 tokens comes exactly once, the operand reads find what they name, and
// the 16 lanes that a 16-byte read serves at once fall into different sixteenths of 256 bytes.
void apart(const char* what, const std::vector<int>& at) {
  std::set<int> slots;
  for (int o : at) {
    if (o % 16) fail(what, o, 0, 0, 0);
    slots.insert(o / 16 % 16);
  }
  if (slots.size() != 16 || at.size() != 16) fail(what, (long)slots.size(), at[0], at[1], 0);
}
template <int D, Kind kind>
void check_k_tile() {
  std::vector<int> holds((size_t)(64 * D / 16), -1);  // piece of the tile (token * D / 16 + piece) at each 16 bytes
  for (int n = 0; n < D / 16; ++n)
    for (int lane = 0; lane < 64; ++lane) {
      const int gran = n / (D / 64), i = n % (D / 64);
      // as the loads form it: granule 0's offset with the granule's exchange on top
      const int src = k_source<D, kind>(i, 0, lane) ^ (16 * k_flip<D, kind>(16 * gran));
      if (src != k_source<D, kind>(i, gran, lane)) fail("granule exchange", D, kind, n, lane);
      if (src < 0 || src + 16 > 16 * D) fail("source outside the granule", D, kind, n, lane);
      holds[(size_t)(64 * n + lane)] = gran * D + src / 16;
      ++g_checked;
    }
  for (int token = 0; token < 64; ++token)
    for (int piece = 0; piece < D / 16; ++piece) {
      const int at = k_at<D, kind>(token, piece);
      if (holds[(size_t)(at / 16)] != token * (D / 16) + piece) fail("K read finds another piece", D, kind, token, piece);
    }
  for (int piece = 0; piece < D / 16; ++piece)
    for (int j = 0; j < 4; ++j) {
      std::vector<int> at;
      for (int l = 0; l < 16; ++l) {
        if (kind == kStep) at.push_back(k_at<D, kind>(16 * (l >> 2) + 4 * j + (l & 3), piece));
        else {  // lanes 16 (j % 2) .. + 15 of tile j / 2
          const int c = l + 16 * (j & 1);
          at.push_back(k_at<D, kind>(32 * (c >> 2 & 1) + 16 * (j >> 1) + 4 * (c >> 3) + (c & 3), piece));
        }
      }
      apart("K bank conflict", at);
    }
}
void check_v_tile() {
  for (int page : {16, 32, 64, 128, 256}) {
    const int run = v_run(__builtin_ctz(page)), gp = 1 << run;
    std::vector<int> seen(64, 0);
    for (int lane = 0; lane < 64; ++lane) {
      const VSource v = v_source(lane, run);
      if (v.gran < 0 || v.gran > 3 || v.col < 0 || v.col > 15) fail("V source", page, lane, v.gran, v.col);
      seen[(size_t)(16 * v.gran + v.col)]++;
      for (int blk = 0; blk < 16; ++blk)
        if (v_at(16 * blk + v.col, v.gran, run) != 1024 * blk + 16 * lane) fail("V read finds another piece", page, lane, blk, 0);
    }
    for (int s : seen)
      if (s != 1) fail("V piece not fetched once", page, s, 0, 0);
    for (int g = 0; g < 4; ++g) {
      std::vector<int> at;
      for (int c = 0; c < 16; ++c) at.push_back(v_at(c, g, run));
      apart("V bank conflict", at);
    }
    // a tile's granules lie in pages as v_run says
    for (int g = 0; g < 4; ++g)
      if (page >= 64 ? (16 * g & (page - 1)) != 16 * g : (16 * g & (page - 1)) != 16 * (g % gp)) fail("V run", page, g, gp, 0);
  }
}

}  // namespace

int main() {
  check_k_tile<64, kStep>();
  check_k_tile<128, kStep>();
  check_k_tile<256, kStep>();
  check_k_tile<64, kPrompt>();
  check_k_tile<128, kPrompt>();
  check_k_tile<256, kPrompt>();
  check_v_tile();
  std::mt19937 rng(1);
  auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
  for (int round = 0; round < 1500; ++round) {
    Cache c{};
    c.shift = pick(4, 8);
    const int ps = 1 << c.shift;
    c.heads = pick(1, 4);
    c.dim = 64;
    c.batch = pick(1, round % 10 == 0 ? 300 : 9);
    c.max_pages = pick(1, 12);
    c.table_stride = c.max_pages + pick(0, 3);
    c.num_pages = pick(1, 40);
    std::vector<int32_t> cu((size_t)c.batch + 1, 0), lens((size_t)c.batch), table((size_t)(c.batch * c.table_stride));
    const bool regular = round % 4 != 3;
    for (int b = 0; b < c.batch; ++b) {
      const int n = pick(0, 3) == 0 ? 0 : (pick(0, 2) ? pick(1, 3) : pick(1, 3 * ps));
      cu[b + 1] = cu[b] + n;
      lens[b] = n + (pick(0, 2) ? pick(0, 6 * ps) : 0);
      if (pick(0, 15) == 0) lens[b] = pick(0, n);          // fewer tokens than rows
    }
    for (auto& t : table) t = pick(0, 12) == 0 ? pick(-3, 60) : pick(0, c.num_pages - 1);
    int64_t T = cu[c.batch] + (pick(0, 3) ? 0 : pick(0, 50));  // rows of no sequence behind
    if (!regular) {
      const int32_t wild[] = {-2147483647 - 1, -1, 0, 1, 1000, 2147483647};
      for (auto& v : cu) if (pick(0, 2) == 0) v = wild[pick(0, 5)];
      for (auto& v : lens) if (pick(0, 2) == 0) v = wild[pick(0, 5)];
      for (auto& v : table) if (pick(0, 2) == 0) v = wild[pick(0, 5)];
    }
    c.table = table.data();
    c.lens = lens.data();
    if (T > 0) check_append(c, cu, T, regular);
    for (int w = 0; w < 3; ++w)
      check_attention(c, cu, T, w == 1 ? pick(1, 300) : 0, w == 2, pick(1, 600), pick(1, 8));
  }
  std::printf("ok: %ld pages and pieces checked\n", g_checked);
  return 0;
}
