// The waits of int8_wide.hip's pipeline: how many of a wave's own copies and
// stores may still be on their way at the end of each step.  Plain C++, so
// that the host can check them against the order in which the kernel issues.
#pragma once

namespace moe {
namespace int8 {
namespace waits {

// Stores of the first and second phase of a half's epilogue (two a block of
// 32 x 32 results; 8 blocks a half, 4 with SwiGLU).
constexpr int stores(bool swiglu, int part) { return part ? (swiglu ? 6 : 10) : (swiglu ? 2 : 6); }

// Prologue, after the copies of two K blocks (32, in the order they are read:
// A0, B0, B1, A1): before A0 and B0 of the first are read; before A0's region
// is filled again (the third block's, 4 copies); before the first phase: the
// first tile's phases wait as every tile's do, for stores that no tile before
// it issued, so both blocks have landed by then.
constexpr int prologue(int step) { return step < 2 ? 24 : 4; }

// End of a phase (0..3) of a tile's first, last or other K block.  The copies
// that the next phase reads have landed, after which six phases of four copies
// were issued, and where an epilogue runs in them its stores: those of the
// tile before in a first block's phases 0 and 1, of this tile in a last
// block's phases 2 and 3.
constexpr int phase(bool swiglu, bool first, bool last, int p) {
  const int s0 = stores(swiglu, 0), s1 = stores(swiglu, 1);
  if (first) return 24 + (p == 0 ? 2 * s0 + s1 : 2 * s0 + 2 * s1);
  if (last && p >= 2) return 24 + (p == 2 ? s0 : s0 + s1);
  return 24;
}

}  // namespace waits
}  // namespace int8
}  // namespace moe
