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
  // weights into registers (bf16_stream.hip; kPlain and kGlu only): a workgroup
  // a tile of so many rows and weight rows
  kSplit16x64 = 2,
  kSplit16x16 = 3,
  kSplit64x64 = 4,
  kSplit64x32 = 5,  // (never with kGlu)
  kSplit64x16 = 6,
};

struct Shape {
  Mode mode;
  bool gather;
  int64_t A_rows, G, M_total;
  int64_t N, K;  // of the weights; kGlu: N = I, half of their rows; kDgradGlu: K = I
};

inline int64_t parts(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Row tiles and column tiles of the register kernels (the host does not know
// the groups' own sizes: at most so many, or what groups of average size have)
inline int64_t m16(const Shape& s) { return std::min(s.M_total, s.G + s.M_total / 16); }
inline int64_t m64(const Shape& s) { return s.G * parts(s.M_total / s.G, 64); }
inline int64_t n64(const Shape& s) { return parts(s.N, s.mode == kGlu ? 32 : 64); }
inline int64_t n32(const Shape& s) { return parts(s.N, 32); }
inline int64_t n16(const Shape& s) { return parts(s.N, s.mode == kGlu ? 8 : 16); }

// A 256 x 256 tile takes as long as two of 128 x 128, one a CU, so the wide
// tiles are taken where they save more than half of the rounds of the CUs.
// Times in us, 256 x 256 / 128 x 128 tiles, N x K of the weights:
//                          4096 x 7168      7168 x 2048
//   64 groups,  17 rows    690 / 656        354 / 346
//               64         725 / 714        387 / 396
//              128         770 / 799        409 / 437
//              192         840 / 1446       453 / 691
//              256         893 / 1283       483 / 705
//   one group, 1024 rows   119 / 74          42 / 43
//             1536         117 / 121         46 / 63
//             2048         129 / 138         53 / 85
//             4096         171 / 281        100 / 163
//   input gradient of one group
//             1024          83 / 84         135 / 72
//             2048         101 / 164        138 / 84
//             4096         203 / 317        152 / 153
// The rule takes the faster one but where they are within 8 %.
//
// The register kernels where there are too few tiles for the CUs: of few rows
// (16 rows of one group 15 us, 56 with 128 x 128 tiles, 4096 x 7168; 9.3 and 20,
// 7168 x 2048) and of up to a 64 x 64 tile a CU (256 rows of one group 54 and 58
// us, 4096 x 7168).  The widest column tile that gives every CU one: 64 rows of one
// group 52 us with 64, 40 with 32, 34 with 16 weight rows (7168 x 2048, where 224
// tiles of 32 are not one a CU: 18, 14 and 21 us).  Their row tiles are
// counted as the most that there can be, so that four groups of 16 rows each are
// left to the tiles (57 us; 34 in registers), as eight are (85 and 83).
inline Plan plan(const Shape& s, int64_t cus) {
  const int64_t avg = s.M_total / s.G;
  const int64_t rows = s.mode == kWgrad ? s.N : avg;
  const int64_t cols = s.mode == kPlain ? s.N : s.mode == kGlu ? 2 * s.N : s.K;
  auto rounds = [&](int64_t tile) { return parts(s.G * parts(rows, tile) * parts(cols, tile), cus); };
  const bool fits = !s.gather || s.A_rows * s.K < 0x7FF80000ll;  // 32-bit offsets into a gathered A
  const Plan tiles = fits && rounds(128) > 2 * rounds(256) ? kWide : kMid;
  if (s.mode >= kDgrad) return tiles;
  if (avg <= 16) {
    const int64_t n = m16(s) * n64(s);
    return n >= 2 * cus ? tiles : n >= cus ? kSplit16x64 : kSplit16x16;
  }
  if (s.G * parts(avg, 64) * parts(cols, 64) > cus) return tiles;
  if (m64(s) * n64(s) >= cus) return kSplit64x64;
  return s.mode != kGlu && m64(s) * n32(s) >= cus ? kSplit64x32 : kSplit64x16;
}

}  // namespace bf16
}  // namespace moe
