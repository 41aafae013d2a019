// The waits of bf16_wide.hip's pipeline: how many of a wave's own copies and
// stores may still be on their way at the end of each step.  Plain C++, so
// that the host can check them against the order in which the kernel issues.
#pragma once

#include "bf16_plan.h"

namespace moe {
namespace bf16 {
namespace waits {

// Stores of the first and second phase of a half's epilogue, at least (kGlu:
// without the kept outputs).  A panel's four are issued when the next one
// begins, the last one's at the end: 4 panels, kWgrad 8, kGlu 2; kDgradGlu four
// every other slot.
constexpr int stores(int mode, int part) {
  if (mode == kGlu) return part ? 8 : 0;
  if (mode == kDgradGlu) return 16;
  if (mode == kWgrad) return part ? 20 : 12;
  return part ? 12 : 4;
}

constexpr int most(int n) { return n < 63 ? n : 63; }  // what the counter holds

// End of a phase (0..3) of a tile's first, last or other K block.  The copies
// that the next phase reads have landed, after which six phases of four copies
// were issued, and where an epilogue runs in them its stores: those of the
// tile before in a first block's phases 0 and 1, of this tile in a last block's
// phases 2 and 3.  Anything else issued among them makes the wait stricter.
constexpr int phase(int mode, bool first, bool last, int p) {
  const int s0 = stores(mode, 0), s1 = stores(mode, 1);
  if (first) return most(24 + (p == 0 ? 2 * s0 + s1 : 2 * s0 + 2 * s1));
  if (last && p >= 2) return most(24 + (p == 2 ? s0 : s0 + s1));
  return 24;
}

}  // namespace waits
}  // namespace bf16
}  // namespace moe
