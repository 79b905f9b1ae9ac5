// gvr_shares.h -- how attend_shared's work is cut into shares: the work of all units lies on one line, which CTAs take
// equal ranges of.  Plain C++ as well, so that those who walk over a share and those who join its pieces are tested
// against each other on the host.
#pragma once

#include "../csrc_cache/gvr_cache_index.h"

namespace gvrc {

// What a unit costs beside its steps (queries, first pages, its piece), in tile steps.  With 2, 3, 4 and 6 the benchmark's
// small groups took 40.9, 41.2, 42.3 and 44.9 us, its document 65, 62.1, 61.8 and 61.9; too little lets those who have
// several units end last, too much those who have none.
constexpr int UNIT_WORK = 3;

// The work of a unit of `steps` steps, each taken by one tile or by both.
GVRC_FN int unit_work(int steps, int both) { return UNIT_WORK + (steps << both); }

// Of a set's units, whose steps are as many, the first `full` are taken by both tiles.  Where a unit begins in the set's work,
// and the unit that lies at a place of it.
GVRC_FN int unit_start(int unit, int full, int steps) {
  const int wide = unit < full ? unit : full;
  return wide * unit_work(steps, 1) + (unit - wide) * unit_work(steps, 0);
}
GVRC_FN int unit_at(int at, int full, int steps) {
  const int wide = full * unit_work(steps, 1);
  return at < wide ? at / unit_work(steps, 1) : full + (at - wide) / unit_work(steps, 0);
}

// Where share c begins, of `total` work cut into `ctas` shares.
GVRC_FN int share_start(int c, int ctas, int total) { return int(int64_t(c) * total / ctas); }

// The share that `at` lies in: the last one that begins at or before it.
GVRC_FN int share_of(int at, int ctas, int total) { return int((int64_t(at + 1) * ctas - 1) / total); }

// The steps before `at` of a unit whose work begins at `start`: a step of work 2 belongs to where its first half lies.
GVRC_FN int step_of(int at, int start, int both, int steps) {
  const int x = at - start - UNIT_WORK;
  if (x <= 0) return 0;
  const int step = both ? (x + 1) >> 1 : x;
  return step < steps ? step : steps;
}

}  // namespace gvrc
