// Which units a launch of the dual-path linear has and in which order (host and
// device; no CUDA needed).
//
// A launch's units are its T tiles, then its main tiles, then, in place of the last of
// them, their pieces along K. CTA c of G takes units c, c + G, ... in order. A unit may
// wait for others: a main tile for its T tiles, a split tile's finisher (piece 0) for
// the other pieces.
//
// Order. A unit waits only for units before it. Blocks are started in the order of
// their indices, so in a launch of one round (as many CTAs as units) whatever a
// running CTA waits for has been started before it and itself waits, at most, for
// units earlier still: the launch completes with any number of its CTAs on the GPU,
// however many SMs other launches hold. Hence the finisher is the last of a tile's units.
#pragma once

#include <algorithm>

#ifdef __CUDACC__
#define DUAL_HD __host__ __device__
#else
#define DUAL_HD
#endif

namespace dual_units {

constexpr int kMaxSplit = 4;  // pieces of a tile, at most

// Unit j of the split tiles.
struct SplitUnit {
  int tile;   // among the split ones
  int piece;  // 0: the one that adds the others' sums
};
DUAL_HD inline SplitUnit split_unit(int j, int k) {
  const int tile = j / k;
  return {tile, k - 1 - (j - tile * k)};
}

// The last, partial round of main tiles, split along K over the CTAs (or pairs) that it
// would leave idle: 3 or 4 pieces, each of at least 2 K-blocks. (Two do not pay for the
// hand-off of the partial sums: measured on 256 x 256 tiles, the round got slower.)
// few_too: also a launch whose units all together would leave two thirds of the GPU
// idle, in one round still.
struct Split {
  int tiles;  // split ones (the last main tiles)
  int k;      // pieces of each; 1: none is split
};
inline Split split_plan(long long t_units, long long main_tiles, long long resident,
                        int kb_total, bool few_too) {
  const long long units = t_units + main_tiles;
  long long rem, room;
  if (units > resident) {
    rem = units % resident;
    room = resident;
  } else if (few_too && 3 * units <= resident) {
    rem = main_tiles;
    room = resident - t_units;
  } else {
    return {0, 1};
  }
  if (rem == 0 || rem > main_tiles) return {0, 1};
  int k = static_cast<int>(std::min<long long>(kMaxSplit, room / rem));
  while (k > 1 && kb_total < 2 * k) --k;
  if (k < 3) return {0, 1};
  return {static_cast<int>(rem), k};
}

}  // namespace dual_units
