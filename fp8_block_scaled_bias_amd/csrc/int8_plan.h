// Which kernel takes a grouped int8 product.  Plain C++, so that the host's
// tests can ask for the choice that the launch makes.
#pragma once

#include <stdint.h>

#include <algorithm>

namespace moe {
namespace int8 {

enum Plan {
  kWide = 0,        // 256 x 256 tiles (int8_wide.hip)
  kMid = 1,         // 128 x 128 tiles (int8_mid.hip)
  kFlow = 2,        // weights into registers (int8_stream.hip): 16 rows, a wave a tile
  kSplit16x64 = 3,  // a workgroup a tile, of so many rows and columns (SwiGLU: half of 64)
  kSplit16x16 = 4,
  kSplit64x64 = 5,
  kSplit64x32 = 6,  // (never with SwiGLU)
  kSplit64x16 = 7,
};

struct Shape {
  bool swiglu, gather;
  int64_t A_rows, G, M_total;
  int64_t N;  // columns of the output
  int64_t K;
};

inline int64_t parts(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Row tiles and column tiles of the register kernels (the host does not know
// the groups' own sizes: at most so many, or what groups of average size have)
inline int64_t m16(const Shape& s) { return std::min(s.M_total, s.G + s.M_total / 16); }
inline int64_t m64(const Shape& s) { return s.G * parts(s.M_total / s.G, 64); }
inline int64_t n64(const Shape& s) { return parts(s.N, s.swiglu ? 32 : 64); }
inline int64_t n32(const Shape& s) { return parts(s.N, 32); }
inline int64_t n16(const Shape& s) { return parts(s.N, 16); }

// The kernel by the rows of a group of average size and by how many tiles
// there are for the CUs.  Times on 64 groups, N = 4096, K = 7168 (wide / mid /
// registers): 8 rows 351 / 360 / 317 us, 16: 352 / 360 / 327, 32: 360 / 362 /
// 374, 128: 420 / 441 / 828; on one group: 16 rows 63 / 38 / 9 us, 64: 63 / 39
// / 19, 256: 63 / 41 / 30 (256 tiles of 64 x 64), 1024: 65 / 45 / 105.  Those are
// groups of equal size: one that holds most of the rows of a small average is
// done in tiles of 16 rows, each reading its weights again.
//
// Of the register kernels, wider column tiles read a token's row for more
// weights, narrower ones are more: the widest that still gives every CU one (16
// to 64 rows; one group of 30, N = 16384, K = 4096: 14.5 us with 64 columns,
// 24.5 with 16; of 64, N = 4096, K = 7168: 22.4 us with 32, 19.4 with 16) or
// two.
inline Plan plan(const Shape& s, int64_t cus) {
  const int64_t avg = s.M_total / s.G, cols = s.swiglu ? 2 * s.N : s.N;
  const int64_t wide_tiles = s.G * parts(avg, 256) * parts(cols, 256);
  const int64_t small_tiles = s.G * parts(avg, 64) * parts(cols, 64);
  const bool fits = !s.gather || s.A_rows * s.K < 0xFFF00000ll;  // 32-bit offsets into a gathered A
  if (fits && avg > 16 && small_tiles > cus) return s.K > 128 && wide_tiles >= cus ? kWide : kMid;
  if (avg <= 16) {
    const int64_t tiles = m16(s) * n64(s);
    return tiles >= 8 * cus ? kFlow : tiles >= 2 * cus ? kSplit16x64 : kSplit16x16;
  }
  if (m64(s) * n64(s) >= cus) return kSplit64x64;
  return !s.swiglu && m64(s) * n32(s) >= cus ? kSplit64x32 : kSplit64x16;
}

}  // namespace int8
}  // namespace moe
