// Host-side audit of how the kernels over the paged cache find the rows of a workgroup (built and run by
// tests/test_kv_order_audit.py; no GPU involved): the searches over cu_seqlens, the pages that an append's slot takes, the
// rows and query heads of a prompt's block and of a step, over starts that rise and over starts that do not.
//  * whatever cu_seqlens, lengths and tables hold, and whichever sequence a search ends at, a slot's tokens lie inside
//    one page of the pool and inside the rows, and every row of a block is a token and a query head of the tensors or none;
//  * where the starts rise, the searches find the last sequence that they ask for, every row of a sequence of more
//    than `small` rows is in one block once, and the multiplication divides like a division.
// Prints one line and exits with 1 on the first violation.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>

#include "kv_index.hpp"

using namespace bsq::kv;

namespace {

[[noreturn]] void fail(const char* what, long a, long b, long c, long d) {
  std::printf("VIOLATION %s (%ld %ld %ld %ld)\n", what, a, b, c, d);
  std::exit(1);
}

long g_checked = 0;

template <int WIDTH, class Holds>
int search(int n, Holds holds) {  // as a wave does it: how many of the candidates, not which
  return last_of<WIDTH>(n, [&](int lo, int step, int left) {
    int cnt = 0;
    for (int i = 0; i < WIDTH; ++i)
      if (i * (long)step < left) {
        if (lo + i * step >= n) fail("a candidate past the batch", lo, i, step, n);
        cnt += holds(lo + i * step) ? 1 : 0;
      }
    return cnt;
  });
}

void check_slot(const Cache& c, const std::vector<int32_t>& cu, int64_t T, int64_t slot, int b) {
  const int ps = 1 << c.shift;
  const Touched t = touched_page(c, cu.data(), b, slot - first_slot(cu.data(), b, T, c.shift), T);
  ++g_checked;
  if (t.n == 0) return;  // (what the kernel returns on)
  if (t.n < 0 || t.at < 0 || t.at + t.n > ps) fail("tokens outside the page", t.at, t.n, b, slot);
  if (t.row < 0 || t.row + t.n > T) fail("rows outside the tensor", t.row, t.n, b, slot);
  if (t.page < -1 || t.page >= c.num_pages) fail("page outside the pool", t.page, c.num_pages, b, slot);
}

void check_row(int R, int group, uint32_t inverse, int kvh, const Rows& rows, int64_t T, int q_heads, int most) {
  const RowPlace p = row_place(R, group, inverse, kvh, rows.n, most);
  ++g_checked;
  if (p.i == -1) return;
  if (p.i < 0 || p.i >= rows.n || p.i >= most || rows.first + p.i >= T) fail("a token outside", R, p.i, rows.first, rows.n);
  if (p.head < kvh * group || p.head >= (kvh + 1) * group || p.head >= q_heads) fail("a head outside", R, p.head, kvh, group);
}

void check(const Cache& c, const std::vector<int32_t>& cu, int64_t T, int group, int small, int most, bool rising) {
  const int q_heads = c.heads * group;
  const int64_t slots = append_slots(T, c.batch, c.shift), blocks = prompt_blocks(T, c.batch, group);
  for (int64_t s = 0; s < slots; ++s) {
    const auto holds = [&](int b) { return first_slot(cu.data(), b, T, c.shift) <= s; };
    const int found = search<256>(c.batch, holds);
    if (found < -1 || found >= c.batch) fail("a sequence outside", found, c.batch, s, 0);
    if (rising) {
      int last = -1;
      for (int b = 0; b < c.batch; ++b)
        if (holds(b)) last = b;
      if (last != found) fail("another sequence of a slot", found, last, s, 0);
    }
    if (found >= 0) check_slot(c, cu, T, s, found);
    if (!rising)
      for (int b = 0; b < c.batch; ++b) check_slot(c, cu, T, s, b);
  }
  std::vector<int> taken((size_t)(T * group), 0);
  for (int64_t id = 0; id < blocks; ++id) {
    const auto holds = [&](int b) { return first_block(cu.data(), b, T, group) <= id; };
    const int found = search<64>(c.batch, holds);
    if (found < -1 || found >= c.batch) fail("a sequence outside", found, c.batch, id, 1);
    if (rising) {
      int last = -1;
      for (int b = 0; b < c.batch; ++b)
        if (holds(b)) last = b;
      if (last != found) fail("another sequence of a block", found, last, id, 1);
    }
    for (int b = rising ? found : 0; b >= 0 && b < (rising ? found + 1 : c.batch); ++b) {
      const Rows rows = rows_of(cu.data(), b, T);
      const int r0 = block_row(cu.data(), b, rows, T, group, id, small, most);
      if (r0 == -1) continue;
      if (r0 < 0 || r0 % kBlock || r0 >= (int64_t)rows.n * group) fail("a block outside its sequence", r0, rows.n, b, id);
      for (int R = r0; R < r0 + kBlock; ++R) {
        check_row(R, group, 0, id % c.heads, rows, T, q_heads, most);
        const RowPlace p = row_place(R, group, 0, 0, rows.n, most);
        if (rising && p.i >= 0) taken[(size_t)((rows.first + p.i) * group + p.head)]++;
      }
    }
  }
  for (int b = 0; b < c.batch; ++b) {
    const Rows rows = rows_of(cu.data(), b, T);
    for (int i = 0; i < rows.n && rising; ++i)
      for (int h = 0; h < group; ++h) {
        const int want = (int64_t)rows.n * group > small && i < most ? 1 : 0;
        const int got = taken[(size_t)((rows.first + i) * group + h)];
        if (got != want) fail("a row not in one block", b, i, h, got);
      }
    if (group <= 16)
      for (int R = 0; R < 16; ++R) {  // a step's rows
        const RowPlace p = row_place(R, group, inverse_of(group), 1, rows.n, most), q = row_place(R, group, 0, 1, rows.n, most);
        if (p.i != q.i || (p.i >= 0 && p.head != q.head)) fail("the multiplication divides otherwise", R, group, p.i, q.i);
        check_row(R, group, inverse_of(group), c.heads - 1, rows, T, q_heads, most);
      }
  }
}

}  // namespace

int main() {
  std::mt19937 rng(7);
  auto pick = [&](int lo, int hi) { return lo + (int)(rng() % (unsigned)(hi - lo + 1)); };
  for (int round = 0; round < 900; ++round) {
    Cache c{};
    c.shift = pick(4, 8);
    c.heads = pick(1, 4);
    c.dim = 64;
    c.batch = pick(1, round % 30 == 0 ? 700 : 9);
    c.max_pages = pick(1, 60);
    c.table_stride = c.max_pages;
    c.num_pages = pick(1, 40);
    std::vector<int32_t> cu((size_t)c.batch + 1, 0), lens((size_t)c.batch), table((size_t)(c.batch * c.table_stride));
    for (int b = 0; b < c.batch; ++b) {
      const int n = pick(0, 3) == 0 ? 0 : (pick(0, 2) ? pick(1, 3) : pick(1, c.batch > 9 ? 9 : 400));
      cu[b + 1] = cu[b] + n;
      lens[b] = n + pick(0, 500);
    }
    for (auto& t : table) t = pick(0, c.num_pages - 1);
    const int64_t T = cu[c.batch] + pick(0, 20);
    const bool rising = round % 2 == 0;
    if (!rising) {  // starts that fall, within the rows and far outside
      const int32_t wild[] = {-2147483647 - 1, -1, 0, 2147483647};
      for (auto& v : cu)
        if (pick(0, 2) == 0) v = pick(0, 5) ? pick(0, (int)T) : wild[pick(0, 3)];
    }
    c.table = table.data();
    c.lens = lens.data();
    if (T == 0) continue;
    const int groups[] = {1, 2, 3, 4, 7, 8, 16, 20, 33, 128, 300};
    check(c, cu, T, groups[pick(0, c.batch > 9 ? 4 : 10)], pick(0, 1) ? 16 : 0, pick(0, 2) ? 0x7FFFFFFF : pick(1, 200), rising);
  }
  // block 31 of group 4 lies before the first of the sequence that the search ends at
  {
    Cache c{};
    std::vector<int32_t> cu = {0, 1000, 1200, 100, 150}, lens = {2000, 1500, 300, 400}, table(4 * 40, 0);
    c.shift = 6; c.heads = 2; c.dim = 64; c.batch = 4; c.max_pages = 40; c.table_stride = 40; c.num_pages = 1;
    c.table = table.data();
    c.lens = lens.data();
    check(c, cu, 1200, 4, 0, 1000, false);
  }
  std::printf("ok: %ld slots and rows checked\n", g_checked);
  return 0;
}
