// Row ranges of groups and the tiles they are cut into: the integer arithmetic on
// which the product kernel's shared memory is laid out and its tables are built.
// Plain C++, for the host and the device.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define QSW_HD __host__ __device__ __forceinline__
#else
#define QSW_HD inline
#endif

namespace qsw {

constexpr int kMaxRecs = 256;     // tiles per CTA; more tiles launch more CTAs

QSW_HD int ceil_div(int a, int b) { return (a + b - 1) / b; }
QSW_HD int64_t ceil_div64(int64_t a, int64_t b) { return (a + b - 1) / b; }

// An entry of a caller's offset table as it is used: within the rows, and no less
// than `top`, the largest such entry before it.  A group's rows run from its own
// entry to the next one's, so that no two groups have a row in common whatever the
// table holds, and the groups' sizes add up to at most `rows`.
QSW_HD int raised_offset(int entry, int top, int rows) {
  const int v = entry < 0 ? 0 : entry > rows ? rows : entry;
  return v < top ? top : v;
}

// Token tiles of a group of m rows, at most bt tokens each.
QSW_HD int token_tiles(int m, int bt) { return ceil_div(m, bt); }

// No more tiles than this for groups whose sizes add up to at most `rows`: a group of
// m rows has at most m / bt whole tiles and another one.
QSW_HD int64_t most_tiles(int rows, int groups, int bt, int n_tiles) {
  return (static_cast<int64_t>(rows) / bt + (groups < rows ? groups : rows)) * n_tiles;
}

// Sharing out at most `most` tiles, each the work of `unit` CTAs: `slots` such units,
// one per `unit` SMs but no more than tiles, and more where a unit would get
// more tiles than there are records; `recs` tiles per unit at most.
struct TilePlan {
  int64_t slots, recs;
};
QSW_HD TilePlan plan_tiles(int64_t most, int num_sms, int unit) {
  TilePlan t;
  t.slots = num_sms / unit;
  if (most < t.slots) t.slots = most;
  if (ceil_div64(most, t.slots) > kMaxRecs) t.slots = ceil_div64(most, kMaxRecs);
  t.recs = ceil_div64(most, t.slots);
  return t;
}

// Tiles of the unit of index `slot` out of `total`: every slots-th from its own on.
QSW_HD int tiles_of(int total, int slot, int slots) { return total > slot ? ceil_div(total - slot, slots) : 0; }

}  // namespace qsw
