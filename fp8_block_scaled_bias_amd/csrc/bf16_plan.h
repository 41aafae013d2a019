// Which kernel takes a grouped bf16 product.  Plain C++, so that the host's
// tests can ask for the choice that the launch makes.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace moe {
namespace bf16 {

enum Mode { kPlain = 0, kGlu = 1, kDgrad = 2, kDgradGlu = 3, kWgrad = 4 };

enum Plan {
  kWide = 0,  // 256 x 256 tiles (bf16_wide.hip)
  kMid = 1,   // 128 x 128 tiles (bf16_mid.hip)
};

struct Shape {
  Mode mode;
  bool gather;
  int64_t A_rows, G, M_total;
  int64_t N, K;  // of the weights; kGlu: N = I, half of their rows; kDgradGlu: K = I
};

inline int64_t parts(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline Plan plan(const Shape& s, int64_t cus) {
  const int64_t avg = s.M_total / s.G;
  const int64_t rows = s.mode == kWgrad ? s.N : avg;
  const int64_t cols = s.mode == kPlain ? s.N : s.mode == kGlu ? 2 * s.N : s.K;
  const int64_t wide_tiles = s.G * parts(rows, 256) * parts(cols, 256);
  const bool fits = !s.gather || s.A_rows * s.K < 0x7FF80000ll;  // 32-bit offsets into a gathered A
  return fits && wide_tiles >= cus && (s.mode == kWgrad || avg > 16) ? kWide : kMid;
}

}  // namespace bf16
}  // namespace moe
