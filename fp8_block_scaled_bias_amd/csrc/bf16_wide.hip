// Grouped bf16 products in 256 x 256 tiles: four waves of 128 x 128,
// v_mfma_f32_32x32x16_bf16, every mode.
//
// The matrix cores take 4096 operations a clock and CU, so a K block of 64
// values of a tile takes 2048 clocks and 64 KB of operands.  LDS takes in the
// copies at 64 B a clock (1024 clocks) and, measured with four waves, gives a
// wave 16 B a lane in 4.3 clocks and transposed 8 B a lane in 6.2: the 128 KB
// that four waves of 128 x 128 read take 550 clocks, 1100 where one operand
// is transposed, 1600 where both are (waves of 128 x 64 would read half as much
// again).  On one group of 32768 rows, 4096 x 7168, the matrix cores are busy 86 %
// of the clocks, 65-71 % in an input gradient and 60 % in a weight gradient (1.28-
// 1.39, 1.15-1.27, 1.13-1.2 PFLOP/s, at 1.4 to 1.6 GHz by the chip's power).
// Hence one wave a SIMD, its accumulators in 256 AGPRs, the operands of a K
// block in 128 VGPRs, and
//  * two K blocks in LDS, in four regions of 16 KB each: tile rows 0..127 and
//    128..255 of P (A0, A1), the tile's two column halves of Q (B0, B1; gate and
//    up with kGlu).  A K block is worked on in four phases, A0 B0, A0 B1, A1 B0,
//    A1 B1, of 16 MFMAs (512 clocks) a wave.  Between its MFMAs a phase reads
//    the operands that the next one adds (B1, A1, then A0 and B0 of the next K
//    block) and copies into the region that the phase before read, for the K
//    block after the next: a copy has six phases to land.  A barrier ends each
//    phase.
//  * An operand whose contraction runs down its rows lies in 64 rows of 256 B
//    and is read transposed.
//  * Copies run on across tiles.  Persistent workgroups; those of an XCD share
//    a contiguous range of tiles (kWgrad: of equal work, its groups' lengths
//    differ), numbered in strips of 8 row tiles (kWgrad: 3), column tile by
//    column tile, so that the 32 tiles at work on an XCD read 8 row and 4 column
//    panels through its L2.
// Every copy goes through a buffer resource over the rows it may touch; lanes
// past a tile's or the contraction's end have an offset outside it.  What
// their slots hold is not used: such rows and columns are not stored, such
// contraction values are cleared in the registers of both operands.
#include "bf16_common.h"
#include "bf16_wide_waits.h"

namespace moe {
namespace bf16 {
namespace {

using gemm::barrier;
using gemm::build_group_tables;
using gemm::copy4;
using gemm::load_rsrc;
using gemm::MAXG;
using gemm::swz;
using gemm::wait_copies;

constexpr int WT = 256;
constexpr int REG = 128 * 128;      // a region: 16 KB
constexpr int STAGE = 4 * REG;      // A0, A1, B0, B1
constexpr int OFF_OUT = 2 * STAGE;  // per wave 32 rows x 128 B
constexpr int OFF_PREF = OFF_OUT + 4 * 4096;
constexpr int OFF_OFFS = OFF_PREF + 4112;
constexpr int OFF_IDX = OFF_OFFS + 4112;  // int [4][256]
constexpr int LDS = OFF_IDX + 4 * 1024;
static_assert((MAXG + 1) * 4 <= 4112 && LDS <= 160 * 1024 - 256, "LDS budget");

template <int V>
using ic = std::integral_constant<int, V>;

// Resources that change with the K block may have been put into vector registers:
// taken back where they were (FRESH: as in the weight gradient of gathered rows,
// between the load and which there have to be wait states).
template <bool FRESH>
__device__ __forceinline__ void copy_block16(const v4i& d, uint32_t voff, uint32_t soff, uint32_t m0) {
  v4i r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = __builtin_amdgcn_readfirstlane(d[i]);
  if (FRESH) gemm::copy16_fresh(r, voff, soff, m0);
  else gemm::copy16(r, voff, soff, m0);
}

__device__ __forceinline__ int64_t uniform(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((int)(uint32_t)v);
  return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32 | lo);
}

struct Tile {
  int g, n0, m0, rows;  // group, first column, first row, rows
  int kc, nkb;          // contraction values, K blocks (at least 2)
  int k0;               // kWgrad: the group's first row
};

template <int MODE, bool GATHER>
__global__ __launch_bounds__(WT, 1) void wide_kernel(Args a) {
  constexpr bool PT = MODE == kWgrad, QT = MODE >= kDgrad;  // contraction down the rows
  constexpr bool GLU = MODE == kGlu;
  __shared__ __attribute__((aligned(16))) uint8_t smem[LDS];
  __shared__ int s_red[4];
  __shared__ int s_carry;
  int* s_pref = reinterpret_cast<int*>(smem + OFF_PREF);
  int* s_offs = reinterpret_cast<int*>(smem + OFF_OFFS);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wv >> 1, wn = wv & 1;
  const int q = lane >> 5, l32 = lane & 31;
  const int G = a.G;
  const int64_t NC = QT ? a.K : a.N;              // columns of the output
  const uint32_t ldp = (uint32_t)(PT || QT ? a.N : a.K) * 2;  // bytes of a row of P, of Q
  const uint32_t ldq = (uint32_t)a.K * 2;
  constexpr int TN = GLU ? 128 : 256;             // output columns of a tile
  const int64_t ntiles = (NC + TN - 1) / TN;
  const int64_t q_rows = GLU ? 2 * a.N : a.N;     // weight rows of a group
  // Row tiles of a strip.  kWgrad: 32 tiles side by side are 3 x 11, so that what
  // they store at a time are long pieces of few rows (8192 tokens, 65 groups: 8
  // 4.02 ms, 4 3.90, 3 3.90, 2 3.94; 64 groups of 896 rows: 3.75, 3.63, 3.50, 3.52);
  // the other modes read less with squares (gate+up of the same: 8 3.04, 4 3.12, 3
  // 3.18 ms).
  constexpr int STRIP = MODE == kWgrad ? 3 : 8;
  const int64_t mtiles = (a.N + 255) / 256;       // kWgrad: row tiles of a group

  // kWgrad: s_pref counts the groups' K blocks and a tile's other work in them
  constexpr int BM = PT ? 64 : 256;
  build_group_tables<WT, BM>(a.offs, G, s_offs, s_pref, s_red, &s_carry);
  const int xcd = blockIdx.x & 7, jw = blockIdx.x >> 3, nper = gridDim.x >> 3;
  int64_t tlo, thi;
  if (PT) {
    constexpr int OVER = 3;  // a tile's stores, in K blocks (65 groups: 1 4.37, 2 4.10, 3 4.00, 5 4.14 ms)
    const int64_t per = mtiles * ntiles, cost = s_pref[G] + (int64_t)OVER * G;
    auto cut = [&](int x) -> int64_t {  // first tile of XCD x
      const int64_t c = cost * x;       // in eighths
      int lo = 0, hi = G;
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (8 * (s_pref[mid] + (int64_t)OVER * mid) <= c) lo = mid;
        else hi = mid;
      }
      const int64_t c0 = 8 * (s_pref[lo] + (int64_t)OVER * lo), own = 8 * (int64_t)(s_pref[lo + 1] - s_pref[lo] + OVER);
      return x == 8 ? G * per : lo * per + (c - c0) * per / own;
    };
    tlo = uniform(cut(xcd));
    thi = uniform(cut(xcd + 1));
  } else {
    const int64_t total = (int64_t)__builtin_amdgcn_readfirstlane(s_pref[G]) * ntiles;
    tlo = total * xcd / 8;
    thi = total * (xcd + 1) / 8;
  }
  const int64_t L0 = tlo + jw;
  if (L0 >= thi) return;
  const int my_n = __builtin_amdgcn_readfirstlane((int)((thi - L0 + nper - 1) / nper));

  // A place in the workgroup's tiles, every nper-th of the XCD's: the group and
  // the tile's number in it (past the last: the last).  The number of tiles is
  // far below 2^32, their results being in memory.
  struct Place {
    int left, g;
    uint32_t rem;
  };
  const uint32_t per = (uint32_t)(mtiles * ntiles);  // kWgrad: tiles of every group
  auto tiles_of = [&](int g) -> uint32_t {
    return PT ? per : (uint32_t)__builtin_amdgcn_readfirstlane(s_pref[g + 1] - s_pref[g]) * (uint32_t)ntiles;
  };
  auto settle = [&](Place& c) {
    uint32_t n = tiles_of(c.g);
    while (c.rem >= n) {
      c.rem -= n;
      n = tiles_of(++c.g);
    }
  };
  auto advance = [&](Place& c) {
    if (--c.left <= 0) return;
    c.rem += (uint32_t)nper;
    settle(c);
  };
  auto tile_at = [&](const Place& c) {
    Tile t;
    t.g = c.g;
    const int g0 = __builtin_amdgcn_readfirstlane(s_offs[t.g]), g1 = __builtin_amdgcn_readfirstlane(s_offs[t.g + 1]);
    const uint32_t cnt = PT ? (uint32_t)mtiles : (uint32_t)(g1 - g0 + 255) >> 8;
    const uint32_t strip = c.rem / (STRIP * (uint32_t)ntiles), r2 = c.rem - strip * (STRIP * (uint32_t)ntiles);
    const uint32_t w = min((uint32_t)STRIP, cnt - strip * STRIP), nt = r2 / w;
    const int mt = (int)(strip * STRIP + r2 - nt * w);
    t.n0 = __builtin_amdgcn_readfirstlane((int)(nt * TN));
    t.m0 = __builtin_amdgcn_readfirstlane((PT ? 0 : g0) + mt * 256);
    t.rows = min(256, (PT ? (int)a.N : g1) - t.m0);
    t.k0 = g0;
    t.kc = PT ? g1 - g0 : (int)(QT ? a.N : a.K);
    t.nkb = max(2, (t.kc + 63) >> 6);
    return t;
  };
  Place first{my_n, 0, 0};
  if (PT) {
    first.g = (int)uniform(L0 / per);
    first.rem = (uint32_t)(L0 - (int64_t)first.g * per);
  } else {
    int64_t rem = L0;
    while (rem >= (int64_t)tiles_of(first.g)) rem -= tiles_of(first.g++);
    first.rem = (uint32_t)rem;
  }
  // valid columns of a tile's half h
  auto cols_of = [&](const Tile& t, int h) -> int {
    return (int)min<int64_t>(128, max<int64_t>(0, GLU ? NC - t.n0 : NC - t.n0 - 128 * h));
  };

  // ---- copies, 1 KB each, four a wave and region.  Along the rows: rows 32 wv
  // + 8 c + lane / 8, slot lane % 8 <- chunk (lane % 8) ^ swz.  Down the rows:
  // rows 16 wv + 4 c + lane / 16, slot lane % 16 <- chunk (lane % 16) ^ 4 (row % 4).
  const uint32_t lds0 = (uint32_t)(uintptr_t)smem;
  const uint32_t m0_w = (uint32_t)__builtin_amdgcn_readfirstlane((int)(lds0 + (uint32_t)wv * 4096));
  constexpr uint32_t kOut = 0xFFFFFF00u;  // an offset outside every resource
  auto crow = [&](int c) -> int { return 32 * wv + 8 * c + (lane >> 3); };
  auto krow = [&](int c) -> int { return 16 * wv + 4 * c + (lane >> 4); };
  const uint32_t tchunk = (uint32_t)(((lane & 15) ^ (4 * ((lane >> 4) & 3))) << 4);
  const int tail = PT || QT ? 0 : (int)((a.K & 63) >> 3);  // chunks of the last K block, 0: all 8
  const int ptail = PT ? 0 : (int)(((QT ? a.N : a.K) & 63) >> 3);
  uint32_t vp[8], vq[4];  // lane offsets of the copies of A0 and A1, of a region of B
  bool cut_p[2], cut_q[2];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int chunk = (lane & 7) ^ swz(crow(c));
    vp[c] = PT ? (uint32_t)krow(c) * ldp + tchunk : (uint32_t)crow(c) * ldp + (uint32_t)(chunk << 4);
    vp[4 + c] = PT ? vp[c] + 256 : vp[c] + 128 * ldp;
    vq[c] = QT ? (uint32_t)krow(c) * ldq + tchunk : (uint32_t)crow(c) * ldq + (uint32_t)(chunk << 4);
    cut_p[c & 1] = ptail && chunk >= ptail;
    cut_q[c & 1] = tail && chunk >= tail;
  }
  const uint32_t a_last = (uint32_t)(a.A_rows - 1);

  // the copies' place: K block ck of tile ct, the co-th; the tile after it
  int co = 0, ck = 0;
  Place cp = first;
  Tile ct, cn = tile_at(cp);
  v4i rp[PT ? 2 : 1], rq[2];
  int* const s_idx = reinterpret_cast<int*>(smem + OFF_IDX);
  // kGlu, kPlain: the row indices of a tile into slot o % 4.  kWgrad: those of
  // a K block of 64 rows into the wave's own slot, counted over all blocks.
  auto index_copy = [&](const Tile& t, int o) {
    copy4(load_rsrc(a.index + t.m0, (uint32_t)t.rows * 4), (uint32_t)(64 * wv + lane) * 4,
          (uint32_t)__builtin_amdgcn_readfirstlane((int)(lds0 + OFF_IDX + (o & 3) * 1024 + wv * 256)));
  };
  auto index_of = [&](int o, int row) -> uint32_t {
    return min((uint32_t)s_idx[(o & 3) * 256 + row], a_last);
  };
  // kWgrad's index copies run two blocks ahead of the copies that use them: 32
  // copies are issued between, more than a phase's wait leaves on their way
  int xk = 0, xb = 0, cb = 0;
  Place xp = first;
  int x_k0 = 0, x_kc = 0;  // the group's rows
  auto index_group = [&]() {
    x_k0 = __builtin_amdgcn_readfirstlane(s_offs[xp.g]);
    x_kc = __builtin_amdgcn_readfirstlane(s_offs[xp.g + 1]) - x_k0;
  };
  auto index_block = [&]() {
    const int64_t r0 = (int64_t)x_k0 + 64 * xk;
    const int left = min(64, x_kc - 64 * xk);
    copy4(load_rsrc(a.index + (left > 0 ? r0 : 0), (uint32_t)max(left, 1) * 4), (uint32_t)lane * 4,
          (uint32_t)__builtin_amdgcn_readfirstlane((int)(lds0 + OFF_IDX + wv * 1024 + (xb & 3) * 256)));
    ++xb;
    if (++xk == max(2, (x_kc + 63) >> 6)) {
      xk = 0;
      advance(xp);
      index_group();
    }
  };
  // resources of the K block to be copied, where they move with it
  auto aim_block = [&]() {
    if (PT) {
      const int left = max(1, min(64, ct.kc - 64 * ck));
      const int64_t row = min<int64_t>((int64_t)ct.k0 + (ct.kc > 64 * ck ? 64 * ck : 0), a.M_total - 1);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // (a half without columns copies the other's)
        const int cols = min(128, ct.rows - 128 * h), hh = cols > 0 ? h : 0;
        rp[PT ? h : 0] = load_rsrc(a.P + row * a.N + ct.m0 + 128 * hh,
                              (uint32_t)(left - 1) * ldp + 2u * (uint32_t)(cols > 0 ? cols : min(128, ct.rows)));
        const int qc = cols_of(ct, h), qh = qc > 0 ? h : 0;
        if (!GATHER)
          rq[h] = load_rsrc(a.Q + row * a.K + ct.n0 + 128 * qh,
                       (uint32_t)(left - 1) * ldq + 2u * (uint32_t)(qc > 0 ? qc : cols_of(ct, 0)));
      }
      if (GATHER) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int r = krow(c);
          vq[c] = r < left && ct.kc > 64 * ck
                      ? min((uint32_t)s_idx[wv * 256 + (cb & 3) * 64 + r], a_last) * ldq + tchunk : kOut;
        }
      }
    } else if (QT) {
      const int left = max(1, min(64, ct.kc - 64 * ck));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int qc = cols_of(ct, h), qh = qc > 0 ? h : 0;
        rq[h] = load_rsrc(a.Q + ((int64_t)ct.g * q_rows + (ct.kc > 64 * ck ? 64 * ck : 0)) * a.K + ct.n0 + 128 * qh,
                     (uint32_t)(left - 1) * ldq + 2u * (uint32_t)(qc > 0 ? qc : cols_of(ct, 0)));
      }
    }
  };
  auto copy_tile = [&]() {  // sources of tile co
    ct = cn;
    advance(cp);
    cn = tile_at(cp);
    if (!QT) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int hh = h && cols_of(ct, 1) > 0;
        const int64_t row = (int64_t)ct.g * q_rows + ct.n0 + (GLU ? h * a.N : hh * 128);
        rq[h] = load_rsrc(a.Q + row * a.K, (uint32_t)cols_of(ct, hh) * ldq);
      }
    }
    if (PT) {
      if (GATHER)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int qc = cols_of(ct, h), qh = qc > 0 ? h : 0;
          const int64_t at = ct.n0 + 128 * qh;
          rq[h] = load_rsrc(a.Q + at, (uint32_t)a_last * ldq + 2u * (uint32_t)(qc > 0 ? qc : cols_of(ct, 0)));
        }
    } else if (GATHER) {
      rp[0] = load_rsrc(a.P, (uint32_t)a.A_rows * ldp);
      // (the lane's place passes through an empty asm so that what follows
      // is computed here and not kept in registers over the K loop)
      int ln = lane;
      asm volatile("" : "+v"(ln));
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        const int row = 128 * (p >> 2) + 32 * wv + 8 * (p & 3) + (ln >> 3);
        vp[p] = row < ct.rows ? index_of(co, row) * ldp + (uint32_t)(((ln & 7) ^ swz(row)) << 4) : kOut;
      }
      index_copy(cn, co + 1);
    } else {
      rp[0] = load_rsrc(a.P + (int64_t)ct.m0 * (ldp / 2), (uint32_t)ct.rows * ldp);
    }
    aim_block();
  };
  // copy c of region R (0, 1: A0, A1; 2, 3: B0, B1) of K block ck into stage st
  auto copy_rows = [&](auto R_, auto C_, uint32_t st) __attribute__((always_inline)) {
    constexpr int R = decltype(R_)::value, C = decltype(C_)::value;
    const uint32_t m = m0_w + st * STAGE + R * REG + C * 1024;
    if (R >= 2) {
      const bool past = !QT && (ck * 64 >= ct.kc || (ck == ct.nkb - 1 && cut_q[C & 1]));
      copy_block16<PT && GATHER>(rq[R & 1], past ? kOut : vq[C], QT ? 0 : (uint32_t)ck * 128, m);
    } else {
      const bool past = !PT && (ck * 64 >= ct.kc || (ck == ct.nkb - 1 && cut_p[C & 1]));
      copy_block16<PT && GATHER>(rp[PT ? R & 1 : 0], past ? kOut : vp[PT ? C : (4 * R + C) & 7], PT ? 0 : (uint32_t)ck * 128, m);
    }
  };
  auto copy_region = [&](auto R_, uint32_t st) __attribute__((always_inline)) {
    copy_rows(R_, ic<0>(), st);
    copy_rows(R_, ic<1>(), st);
    copy_rows(R_, ic<2>(), st);
    copy_rows(R_, ic<3>(), st);
  };
  auto copy_next = [&]() {  // to the next K block
    ++cb;
    if (PT && GATHER) index_block();
    if (++ck == ct.nkb) {
      ck = 0;
      ++co;
      copy_tile();
    } else {
      aim_block();
    }
  };

  // ---- operand reads: lane (q, l32) has 8 contraction values (16 ks + 8 q ..)
  // of row or column l32 of a 32-wide block.  The wave's two blocks of a
  // region begin at 32 wm and 64 further (P), at 64 wn and 32 further (Q: 64
  // columns, a whole line of bf16, are one wave's).
  uint32_t o[4];
#pragma unroll
  for (int ks = 0; ks < 4; ++ks)
    o[ks] = (uint32_t)(l32 * 128 + (((2 * ks + q) ^ swz(l32)) << 4));
  const uint32_t otr = tr_lane(lane);
  v4i fr[4][2][4];  // operands of A0, A1, B0, B1: [block][ks]
  auto read_one = [&](auto R_, int n, uint32_t st) __attribute__((always_inline)) {
    constexpr int R = decltype(R_)::value;
    const uint8_t* p = smem + st * STAGE + R * REG;
    const int w = R >= 2 ? 2 * wn + (n & 1) : wm + 2 * (n & 1);  // the 32-wide block
    if (R >= 2 ? QT : PT)
      fr[R][n & 1][n >> 1] = tr_read(p, otr, w, n >> 1);
    else
      fr[R][n & 1][n >> 1] = *reinterpret_cast<const v4i*>(p + w * 32 * 128 + o[n >> 1]);
  };
  auto clear_past = [&](auto R_, int left) __attribute__((always_inline)) {
    constexpr int R = decltype(R_)::value;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
      if (!PT || left < 16 * ks + 16) {
        fr[R][0][ks] = keep_first(fr[R][0][ks], left - 16 * ks - 8 * q);
        fr[R][1][ks] = keep_first(fr[R][1][ks], left - 16 * ks - 8 * q);
      }
  };

  v16f acc[2][2][2][2];  // [A half][B half][A block][B block]

  // ---- epilogue, between MFMAs: A0's results while the last K block works on
  // A1, A1's while the next tile's first works on A0, a half over 16 slots.
  // Lane (q, l32) holds row l32 of a 32 x 32 block and its columns 8 e + 4 q ..
  // +3; a panel of 32 rows by 128 bytes goes through the wave's own 4 KB of LDS
  // (16-byte chunk c of a row in slot c ^ row % 8) and comes back as 8 whole lines
  // a store: stores of 32 rows by 32 bytes drain at 34 B/ns a CU instead of 130.
  // Rows past the tile's end lie outside the store's resource, columns past it
  // are put outside: every panel issues all its stores.
  typedef uint32_t v4u __attribute__((ext_vector_type(4)));
  const uint32_t ldo = (uint32_t)(MODE == kDgradGlu ? 2 * NC : NC);  // columns of the output's rows
  // rows r0 .. of a tile in a tensor of `ld` columns a row, from column c0
  auto rows_at = [&](auto* base, const Tile& t, uint32_t ld, int64_t c0, int r0) __attribute__((always_inline)) {
    const int64_t row = (MODE == kWgrad ? (int64_t)t.g * a.N : 0) + t.m0 + r0;
    const int64_t left = max<int64_t>(0, (int64_t)(t.rows - r0) * ld - c0);
    return __builtin_amdgcn_make_buffer_rsrc((void*)(base + row * ld + c0), 0,
                                             (int)(uint32_t)(left * (int64_t)sizeof(*base)), 0x00020000);
  };
  const uint32_t l7 = l32 & 7;
  const uint32_t e_wr = OFF_OUT + wv * 4096 + l32 * 128;
  const uint32_t e_rd = OFF_OUT + wv * 4096 + (lane >> 3) * 128 + (((lane & 7) ^ (lane >> 3)) << 4);
  v4u lines[4];
  auto read_lines = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < 4; ++r) lines[r] = *reinterpret_cast<const v4u*>(smem + e_rd + r * 1024);
  };
  // A weight gradient is more than the caches hold: its stores are marked as not
  // reused, so that they do not push the operands' panels out of an XCD's 4 MB of
  // L2 (8192 tokens, 65 groups: 4.35 -> 4.10 ms; no difference for the other
  // modes, whose results the next call reads).
  constexpr int CACHE = MODE == kWgrad ? 2 : 0;
  // a panel's lines: rows r0 + 8 r + lane / 8, bytes 16 (lane % 8) of columns cc ..
  auto store_lines = [&](auto* base, const Tile& t, uint32_t ld, int64_t half, int r0, int cc) __attribute__((always_inline)) {
    constexpr int SZ = sizeof(*base), per = 16 / SZ;  // columns of a lane
    const auto out = rows_at(base, t, ld, half + t.n0, r0);
    const int c = cc + per * (lane & 7);
    const uint32_t off = t.n0 + c < NC ? ((lane >> 3) * ld + c) * SZ : kOut;
#pragma unroll
    for (int r = 0; r < 4; ++r)  // (past the rows' end stays past it: kOut + 24 rows is under 2^32)
      __builtin_amdgcn_raw_buffer_store_b128(lines[r], out, off == kOut ? off : off + 8 * r * ld * SZ, 0, CACHE);
  };
  auto put4 = [&](int chunk, const float* v) __attribute__((always_inline)) {  // 4 bf16 at 8 q of a chunk
    *reinterpret_cast<uint2*>(smem + e_wr + ((chunk ^ l7) << 4) + 8 * q) = pack4(v);
  };
  auto quad = [&](const v16f& c, int e, float (&v)[4]) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = c[4 * e + r];
  };
  // kDgradGlu: a block's gate and up values as its results are read back, rows
  // lane / 4 and + 16, columns 8 (lane % 4) ..; loaded a block ahead
  v4u gate[2][2], up[2][2];
  auto fetch = [&](auto K_, const Tile& t) __attribute__((always_inline)) {
    constexpr int K = decltype(K_)::value, H = K >> 3, B = (K >> 2) & 1, i = (K >> 1) & 1, j = K & 1;
    const int r0 = 128 * H + 64 * i + 32 * wm, c = 128 * B + 64 * wn + 32 * j + 8 * (lane & 3);
    const auto g = rows_at(a.gu_in, t, ldo, t.n0, r0), u = rows_at(a.gu_in, t, ldo, NC + t.n0, r0);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const uint32_t off = t.n0 + c < NC ? ((16 * r + (lane >> 2)) * ldo + c) * 2 : kOut;
      gate[K & 1][r] = __builtin_amdgcn_raw_buffer_load_b128(g, off, 0, 0);
      up[K & 1][r] = __builtin_amdgcn_raw_buffer_load_b128(u, off, 0, 0);
    }
  };
  // slot S (0..15) of half H's epilogue
  auto emit = [&](auto H_, auto S_, const Tile& t) __attribute__((always_inline)) {
    constexpr int H = decltype(H_)::value, S = decltype(S_)::value;
    float v[4], w[4];
    if constexpr (MODE == kWgrad) {
      // 8 panels, the 32 x 32 blocks; two slots each write half of its quads
      constexpr int K = S >> 1, B = K >> 2, i = (K >> 1) & 1, j = K & 1;
      auto store = [&](auto P_) __attribute__((always_inline)) {
        constexpr int P = decltype(P_)::value;
        read_lines();
        store_lines(static_cast<float*>(a.out), t, ldo, 0, 128 * H + 64 * ((P >> 1) & 1) + 32 * wm,
                    128 * (P >> 2) + 64 * wn + 32 * (P & 1));
      };
      if constexpr (S > 0 && S % 2 == 0) store(ic<K - 1>());
#pragma unroll
      for (int e = 2 * (S & 1); e < 2 * (S & 1) + 2; ++e) {
        quad(acc[H][B][i][j], e, v);
        *reinterpret_cast<float4*>(smem + e_wr + (((2 * e + q) ^ l7) << 4)) = make_float4(v[0], v[1], v[2], v[3]);
      }
      if constexpr (S == 15) store(ic<7>());
    } else if constexpr (MODE == kGlu) {
      // 2 row blocks; the kept gate and up panels in the first four slots, h's
      // quads in the last four
      constexpr int i = S >> 3, n = S & 7;
      const int r0 = 128 * H + 64 * i + 32 * wm;
      uint16_t* const h = static_cast<uint16_t*>(a.out);
      if constexpr (n == 0 && i == 1) {
        read_lines();
        store_lines(h, t, ldo, 0, r0 - 64, 64 * wn);
      }
      if constexpr (n < 4) {
        if (a.keep) {
          if constexpr (n == 2) {
            read_lines();
            store_lines(a.keep, t, 2 * ldo, 0, r0, 64 * wn);
          }
#pragma unroll
          for (int k = 4 * (n & 1); k < 4 * (n & 1) + 4; ++k) {
            quad(acc[H][n >> 1][i][k >> 2], k & 3, v);
            put4(k, v);
          }
        }
      } else {
        if constexpr (n == 4)
          if (a.keep) {
            read_lines();
            store_lines(a.keep, t, 2 * ldo, NC, r0, 64 * wn);
          }
#pragma unroll
        for (int k = 2 * (n - 4); k < 2 * (n - 4) + 2; ++k) {
          quad(acc[H][0][i][k >> 2], k & 3, v);
          quad(acc[H][1][i][k >> 2], k & 3, w);
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] = glu(v[r], w[r], a.act);
          put4(k, v);
        }
        if constexpr (S == 15) {
          read_lines();
          store_lines(h, t, ldo, 0, r0, 64 * wn);
        }
      }
    } else if constexpr (MODE == kDgradGlu) {
      // 8 blocks: dh through LDS as fp32, 8 columns a lane, in the first slot,
      // gradients in the second
      constexpr int K = S >> 1, B = K >> 2, i = (K >> 1) & 1, j = K & 1;
      if constexpr (S % 2 == 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          quad(acc[H][B][i][j], e, v);
          *reinterpret_cast<float4*>(smem + e_wr + (((2 * e + q) ^ l7) << 4)) = make_float4(v[0], v[1], v[2], v[3]);
        }
        if constexpr (8 * H + K + 1 < 16) fetch(ic<(8 * H + K + 1) & 15>(), t);
      } else {
        constexpr int F = K & 1;
        uint16_t* const out = static_cast<uint16_t*>(a.out);
        const int r0 = 128 * H + 64 * i + 32 * wm, c = 128 * B + 64 * wn + 32 * j + 8 * (lane & 3);
        const auto og = rows_at(out, t, ldo, t.n0, r0), ou = rows_at(out, t, ldo, NC + t.n0, r0);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = 16 * r + (lane >> 2);
          float d[8], dg[8], du[8];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const float4 f = *reinterpret_cast<const float4*>(smem + OFF_OUT + wv * 4096 + row * 128 +
                                                              (((2 * (lane & 3) + x) ^ (row & 7)) << 4));
            d[4 * x] = f.x, d[4 * x + 1] = f.y, d[4 * x + 2] = f.z, d[4 * x + 3] = f.w;
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t gw = gate[F][r][k >> 1], uw = up[F][r][k >> 1];
            glu_backward(bf16_to_f32(k & 1 ? gw >> 16 : gw & 0xFFFFu), bf16_to_f32(k & 1 ? uw >> 16 : uw & 0xFFFFu),
                         d[k], a.act, &dg[k], &du[k]);
          }
          const uint2 g0 = pack4(dg), g1 = pack4(dg + 4), u0 = pack4(du), u1 = pack4(du + 4);
          const uint32_t off = t.n0 + c < NC ? (row * ldo + c) * 2 : kOut;
          __builtin_amdgcn_raw_buffer_store_b128(v4u{g0.x, g0.y, g1.x, g1.y}, og, off, 0, 0);
          __builtin_amdgcn_raw_buffer_store_b128(v4u{u0.x, u0.y, u1.x, u1.y}, ou, off, 0, 0);
        }
      }
    } else {
      // 4 panels of two 32 x 32 blocks; four slots each write a quarter
      constexpr int K = S >> 2, B = K >> 1, i = K & 1, n = S & 3;
      auto store = [&](auto P_) __attribute__((always_inline)) {
        constexpr int P = decltype(P_)::value;
        read_lines();
        store_lines(static_cast<uint16_t*>(a.out), t, ldo, 0, 128 * H + 64 * (P & 1) + 32 * wm,
                    128 * (P >> 1) + 64 * wn);
      };
      if constexpr (S > 0 && n == 0) store(ic<K - 1>());
#pragma unroll
      for (int k = 2 * n; k < 2 * n + 2; ++k) {
        quad(acc[H][B][i][k >> 2], k & 3, v);
        put4(k, v);
      }
      if constexpr (S == 15) store(ic<3>());
    }
  };

  // ---- prologue: the first two K blocks, in the order they are read
  Place p = first;
  Tile t = cn;
  if (GATHER) {
    if (PT) {
      index_group();
      index_block();
      index_block();
      index_block();
    } else {
      index_copy(t, 0);
    }
    wait_copies<0>();
    barrier();
  }
  copy_tile();
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    copy_region(ic<0>(), s);
    copy_region(ic<2>(), s);
    copy_region(ic<3>(), s);
    copy_region(ic<1>(), s);
    if (s == 0) copy_next();
  }
  // (with an index, one or two of its copies are among the newest: a wait for
  // as many as there would be without them waits for more, never for less)
  wait_copies<24>();
  barrier();
#pragma unroll
  for (int n = 0; n < 8; ++n) {
    read_one(ic<0>(), n, 0);
    read_one(ic<2>(), n, 0);
  }
  wait_copies<PT && GATHER ? 0 : 24>();  // (the third block's indices too)
  barrier();
  copy_next();
  copy_region(ic<0>(), 0);  // A0 of the third
  // (the first tile's phases wait as every tile's do, for stores of a tile
  // before it that it does not have: both blocks have landed here)
  wait_copies<4>();
  barrier();

  // A phase: MFMAs of A half H and B half B; reads region R of stage rst for
  // the next one (early, so that the wait at its end finds them done), copies
  // region CR into stage cst.  FIRST: from zero.  PART 0, 1: part of the
  // epilogue of the other half of d.  W: the wait that ends the phase.
  auto phase = [&](auto H_, auto B_, auto R_, uint32_t rst, auto CR_, uint32_t cst, auto FIRST_, auto PART_, auto W_,
                   const Tile& d) __attribute__((always_inline)) {
    constexpr int H = decltype(H_)::value, B = decltype(B_)::value, PART = decltype(PART_)::value;
    constexpr bool FIRST = decltype(FIRST_)::value;
    auto slot = [&](auto N_) __attribute__((always_inline)) {
      constexpr int n = decltype(N_)::value;
      constexpr int i = n >> 2, ks = n & 3;  // block of A, K chunk
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const v16f zero = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
        acc[H][B][i][j] = mfma(fr[2 + B][j][ks], fr[H][i][ks], FIRST && ks == 0 ? zero : acc[H][B][i][j]);
      }
      if (n < 4) {
        read_one(R_, 2 * n, rst);
        read_one(R_, 2 * n + 1, rst);
      } else {
        copy_rows(CR_, ic<(n & 3)>(), cst);
      }
      if constexpr (PART >= 0) emit(ic<1 - H>(), ic<8 * (PART & 1) + n>(), d);
      __builtin_amdgcn_sched_barrier(0);
    };
    slot(ic<0>());
    slot(ic<1>());
    slot(ic<2>());
    slot(ic<3>());
    slot(ic<4>());
    slot(ic<5>());
    slot(ic<6>());
    slot(ic<7>());
    wait_copies<decltype(W_)::value>();
    __builtin_amdgcn_sched_barrier(0);
    barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  // Ends of phases: the phase's reads are in registers, the copies that the
  // next phase reads have landed (bf16_wide_waits.h).
  uint32_t st = 0;  // stage of the K block being multiplied
  Tile done = t;    // the tile before, whose A1 is still to be stored
  done.rows = 0;
  auto block = [&](auto FIRST_, auto LAST_, int left) __attribute__((always_inline)) {
    constexpr bool FIRST = decltype(FIRST_)::value, LAST = decltype(LAST_)::value;
    const bool cut = (FIRST || LAST) && left < 64;  // (those between are whole)
    if (cut) {
      clear_past(ic<0>(), left);
      clear_past(ic<2>(), left);
    }
    phase(ic<0>(), ic<0>(), ic<3>(), st, ic<2>(), st, FIRST_, ic<(FIRST ? 0 : -1)>(),
          ic<waits::phase(MODE, FIRST, LAST, 0)>(), done);
    if (cut) clear_past(ic<3>(), left);
    phase(ic<0>(), ic<1>(), ic<1>(), st, ic<3>(), st, FIRST_, ic<(FIRST ? 1 : -1)>(),
          ic<waits::phase(MODE, FIRST, LAST, 1)>(), done);
    if (cut) clear_past(ic<1>(), left);
    if constexpr (LAST) {
      done = t;
      if constexpr (MODE == kDgradGlu) {
        fetch(ic<0>(), done);
      }
    }
    phase(ic<1>(), ic<0>(), ic<0>(), st ^ 1, ic<1>(), st, FIRST_, ic<(LAST ? 0 : -1)>(),
          ic<waits::phase(MODE, FIRST, LAST, 2)>(), done);
    copy_next();
    phase(ic<1>(), ic<1>(), ic<2>(), st ^ 1, ic<0>(), st ^ 1, FIRST_, ic<(LAST ? 1 : -1)>(),
          ic<waits::phase(MODE, FIRST, LAST, 3)>(), done);
    st ^= 1;
  };
  for (; p.left > 0; advance(p), t = tile_at(p)) {
    block(ic<1>(), ic<0>(), t.kc);
    for (int k = 1; k < t.nkb - 1; ++k) block(ic<0>(), ic<0>(), 64);
    block(ic<0>(), ic<1>(), t.kc - 64 * (t.nkb - 1));
  }
  auto flush = [&](auto N_) __attribute__((always_inline)) {
    emit(ic<1>(), N_, done);
    __builtin_amdgcn_sched_barrier(0);
  };
  flush(ic<0>()); flush(ic<1>()); flush(ic<2>()); flush(ic<3>());
  flush(ic<4>()); flush(ic<5>()); flush(ic<6>()); flush(ic<7>());
  flush(ic<8>()); flush(ic<9>()); flush(ic<10>()); flush(ic<11>());
  flush(ic<12>()); flush(ic<13>()); flush(ic<14>()); flush(ic<15>());
  wait_copies<0>();  // what was copied past the last tile lands before the LDS is released
}

}  // namespace

void launch_wide(const Args& a, Mode m, hipStream_t st) {
  const dim3 grid(std::max(8, gemm::num_cus() / 8 * 8)), block(WT);
  switch (m) {
    case kPlain:
      if (a.index) wide_kernel<kPlain, true><<<grid, block, 0, st>>>(a);
      else wide_kernel<kPlain, false><<<grid, block, 0, st>>>(a);
      break;
    case kGlu:
      if (a.index) wide_kernel<kGlu, true><<<grid, block, 0, st>>>(a);
      else wide_kernel<kGlu, false><<<grid, block, 0, st>>>(a);
      break;
    case kDgrad: wide_kernel<kDgrad, false><<<grid, block, 0, st>>>(a); break;
    case kDgradGlu: wide_kernel<kDgradGlu, false><<<grid, block, 0, st>>>(a); break;
    case kWgrad:
      if (a.index) wide_kernel<kWgrad, true><<<grid, block, 0, st>>>(a);
      else wide_kernel<kWgrad, false><<<grid, block, 0, st>>>(a);
      break;
  }
}

}  // namespace bf16
}  // namespace moe
