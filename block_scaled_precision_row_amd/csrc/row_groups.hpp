// Rows that fall into groups with vectors of their own (include/bsq_block.h): which group a row has.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace bsq {

struct RowGroups {
  const int32_t* starts;  // [groups + 1], or null: `per` rows each
  int groups;
  int per;
  int rows;  // of the call
  int end;   // starts[end] ends the last group (a call without vectors of groups counts all its rows as one's)
};

// rows of groups: from here on a row is not written
__device__ __forceinline__ int group_limit(const RowGroups& r) {
  if (!r.starts) return r.rows;
  const int n = r.starts[r.end];
  return n < 0 ? 0 : (n < r.rows ? n : r.rows);
}

// The group of a row that is the same for the whole wave: how many of starts[1 .. groups - 1] are at most the row, by
// 64 of them at a time (one load up to 64 groups). Always in [0, groups), whatever the starts hold.
__device__ __forceinline__ int group_of_wave(const RowGroups& r, int row, int lane) {
  if (r.groups <= 1) return 0;
  if (!r.starts) return row / r.per;
  int lo = 0, n = r.groups;
  while (n > 1) {
    const int step = (n + 63) >> 6, at = (lane + 1) * step;
    const bool past = at < n && r.starts[lo + at] <= row;
    const int k = __popcll(__ballot(past));  // (at most (n - 1) / step lanes have at < n)
    lo += k * step;
    n = n - k * step < step ? n - k * step : step;
  }
  return __builtin_amdgcn_readfirstlane(lo);
}

// the first row behind group g
__device__ __forceinline__ int group_end(const RowGroups& r, int g) {
  if (!r.starts) return (g + 1) * r.per;
  return r.starts[g + 1];
}

// the group of each lane's own row, which lies between those of two rows whose groups are first and last
__device__ __forceinline__ int group_of_lane(const RowGroups& r, int row, int first, int last) {
  if (!r.starts) return r.groups <= 1 ? 0 : row / r.per;
  int lo = first, hi = last;  // the largest g with starts[g] <= row
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (r.starts[mid] <= row) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

}  // namespace bsq
