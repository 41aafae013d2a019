// Grouped bf16 products in 256 x 256 tiles: four waves of 128 x 128,
// v_mfma_f32_32x32x16_bf16, every mode.
//
// The matrix cores take 4096 operations a clock and CU, so a K block of 64
// values of a tile takes 2048 clocks and 64 KB of operands.  LDS moves 128 B a
// clock: the 64 KB that come in and the 128 KB that four waves of 128 x 128
// read take 1536 of them (eight waves of 128 x 64 would fill them all).  Hence
// one wave a SIMD, its accumulators in 256 AGPRs, the operands of a K block in
// 128 VGPRs, and
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
//    differ), numbered in strips of 8 row tiles, column tile by column tile,
//    so that the 32 tiles at work on an XCD read 8 row and 4 column panels
//    through its L2.
// Every copy goes through a buffer resource over the rows it may touch; lanes
// past a tile's or the contraction's end have an offset outside it.  What
// their slots hold is not used: such rows and columns are not stored, such
// contraction values are cleared in the registers of both operands.
#include "bf16_common.h"

namespace moe {
namespace bf16 {
namespace {

using gemm::barrier;
using gemm::build_group_tables;
using gemm::MAXG;
using gemm::swz;

constexpr int WT = 256;
constexpr int REG = 128 * 128;      // a region: 16 KB
constexpr int STAGE = 4 * REG;      // A0, A1, B0, B1
constexpr int STRIP = 8;            // row tiles of a strip
constexpr int OFF_OUT = 2 * STAGE;  // per wave 32 x 32 results
constexpr int OFF_PREF = OFF_OUT + 4 * 4096;
constexpr int OFF_OFFS = OFF_PREF + 4112;
constexpr int OFF_IDX = OFF_OFFS + 4112;  // int [4][256]
constexpr int LDS = OFF_IDX + 4 * 1024;
static_assert((MAXG + 1) * 4 <= 4112 && LDS <= 160 * 1024 - 256, "LDS budget");

template <int V>
using ic = std::integral_constant<int, V>;

__device__ __forceinline__ v4i rsrc(const void* p, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  v4i r;
  r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)a);
  r[1] = __builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32));
  r[2] = __builtin_amdgcn_readfirstlane((int)bytes);
  r[3] = 0x00020000;
  return r;
}
// Lane i's 16 (4) bytes from offset voff + soff of the resource land at m0 +
// i * 16 (4); out of range: not read from memory.
// (resources that change with the K block may have been put into vector
// registers: taken back where they were, nothing where they were not)
__device__ __forceinline__ void copy16(const v4i& d, uint32_t voff, uint32_t soff, uint32_t m0) {
  v4i r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r[i] = __builtin_amdgcn_readfirstlane(d[i]);
  asm volatile("s_mov_b32 m0, %3\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
               ::"v"(voff), "s"(r), "s"(soff), "s"(m0) : "memory", "m0");
}
__device__ __forceinline__ void copy4(const v4i& r, uint32_t voff, uint32_t m0) {
  asm volatile("s_mov_b32 m0, %2\n\tbuffer_load_dword %0, %1, 0 offen lds"
               ::"v"(voff), "s"(r), "s"(m0) : "memory", "m0");
}
// s_waitcnt vmcnt(N) lgkmcnt(0)
template <int N>
__device__ __forceinline__ void wait_copies() {
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
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
  const int64_t mtiles = (a.N + 255) / 256;       // kWgrad: row tiles of a group

  // kWgrad: s_pref counts the groups' K blocks and a tile's other work in them
  constexpr int BM = PT ? 64 : 256;
  build_group_tables<WT, BM>(a.offs, G, s_offs, s_pref, s_red, &s_carry);
  const int xcd = blockIdx.x & 7, jw = blockIdx.x >> 3, nper = gridDim.x >> 3;
  int64_t tlo, thi;
  if (PT) {
    constexpr int OVER = 4;  // a tile's stores, in K blocks
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
  const int my_n = (int)((thi - L0 + nper - 1) / nper);

  // tile of ordinal o (past the last: the last); gh: group of the tile before
  auto tile_at = [&](int& gh, int o) {
    const int64_t L = L0 + (int64_t)min(o, my_n - 1) * nper;
    Tile t;
    uint32_t cnt, rem;
    if (PT) {
      const int64_t per = mtiles * ntiles;
      gh = t.g = __builtin_amdgcn_readfirstlane((int)(L / per));
      cnt = (uint32_t)mtiles;
      rem = (uint32_t)(L - t.g * per);
    } else {
      int g = gh;
      while (g + 1 < G && (int64_t)s_pref[g + 1] * ntiles <= L) ++g;
      gh = t.g = __builtin_amdgcn_readfirstlane(g);
      cnt = (uint32_t)(s_pref[t.g + 1] - s_pref[t.g]);
      rem = (uint32_t)(L - (int64_t)s_pref[t.g] * ntiles);
    }
    const uint32_t strip = rem / (STRIP * (uint32_t)ntiles), r2 = rem - strip * (STRIP * (uint32_t)ntiles);
    const uint32_t w = min((uint32_t)STRIP, cnt - strip * STRIP), nt = r2 / w;
    const int mt = (int)(strip * STRIP + r2 - nt * w);
    t.n0 = __builtin_amdgcn_readfirstlane((int)(nt * TN));
    const int g0 = s_offs[t.g], g1 = s_offs[t.g + 1];
    t.m0 = __builtin_amdgcn_readfirstlane((PT ? 0 : g0) + mt * 256);
    t.rows = __builtin_amdgcn_readfirstlane(min(256, (PT ? (int)a.N : g1) - t.m0));
    t.k0 = __builtin_amdgcn_readfirstlane(g0);
    t.kc = __builtin_amdgcn_readfirstlane(PT ? g1 - g0 : (int)(QT ? a.N : a.K));
    t.nkb = max(2, (t.kc + 63) >> 6);
    return t;
  };
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

  // the copies' place: K block ck of the tile of ordinal co
  int co = 0, ck = 0, cg = 0;
  Tile ct;
  v4i rp[PT ? 2 : 1], rq[2];
  int* const s_idx = reinterpret_cast<int*>(smem + OFF_IDX);
  // kGlu, kPlain: the row indices of a tile into slot o % 4.  kWgrad: those of
  // a K block of 64 rows into the wave's own slot, counted over all blocks.
  auto index_copy = [&](const Tile& t, int o) {
    copy4(rsrc(a.index + t.m0, (uint32_t)t.rows * 4), (uint32_t)(64 * wv + lane) * 4,
          (uint32_t)__builtin_amdgcn_readfirstlane((int)(lds0 + OFF_IDX + (o & 3) * 1024 + wv * 256)));
  };
  auto index_of = [&](int o, int row) -> uint32_t {
    return min((uint32_t)s_idx[(o & 3) * 256 + row], a_last);
  };
  // kWgrad's index copies run two blocks ahead of the copies that use them: 32
  // copies are issued between, more than a phase's wait leaves on their way
  int xo = 0, xk = 0, xg = 0, xb = 0, cb = 0;
  Tile xt;
  auto index_block = [&]() {
    const int64_t r0 = (int64_t)xt.k0 + 64 * xk;
    const int left = min(64, xt.kc - 64 * xk);
    copy4(rsrc(a.index + (left > 0 ? r0 : 0), (uint32_t)max(left, 1) * 4), (uint32_t)lane * 4,
          (uint32_t)__builtin_amdgcn_readfirstlane((int)(lds0 + OFF_IDX + wv * 1024 + (xb & 3) * 256)));
    ++xb;
    if (++xk == xt.nkb) {
      xk = 0;
      xt = tile_at(xg, ++xo);
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
        rp[PT ? h : 0] = rsrc(a.P + row * a.N + ct.m0 + 128 * hh,
                              (uint32_t)(left - 1) * ldp + 2u * (uint32_t)(cols > 0 ? cols : min(128, ct.rows)));
        const int qc = cols_of(ct, h), qh = qc > 0 ? h : 0;
        if (!GATHER)
          rq[h] = rsrc(a.Q + row * a.K + ct.n0 + 128 * qh,
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
        rq[h] = rsrc(a.Q + ((int64_t)ct.g * q_rows + (ct.kc > 64 * ck ? 64 * ck : 0)) * a.K + ct.n0 + 128 * qh,
                     (uint32_t)(left - 1) * ldq + 2u * (uint32_t)(qc > 0 ? qc : cols_of(ct, 0)));
      }
    }
  };
  auto copy_tile = [&]() {  // sources of tile co
    ct = tile_at(cg, co);
    if (!QT) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int hh = h && cols_of(ct, 1) > 0;
        const int64_t row = (int64_t)ct.g * q_rows + ct.n0 + (GLU ? h * a.N : hh * 128);
        rq[h] = rsrc(a.Q + row * a.K, (uint32_t)cols_of(ct, hh) * ldq);
      }
    }
    if (PT) {
      if (GATHER)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int qc = cols_of(ct, h), qh = qc > 0 ? h : 0;
          const int64_t at = ct.n0 + 128 * qh;
          rq[h] = rsrc(a.Q + at, (uint32_t)a_last * ldq + 2u * (uint32_t)(qc > 0 ? qc : cols_of(ct, 0)));
        }
    } else if (GATHER) {
      rp[0] = rsrc(a.P, (uint32_t)a.A_rows * ldp);
      // (the lane's place passes through an empty asm so that what follows
      // is computed here and not kept in registers over the K loop)
      int ln = lane;
      asm volatile("" : "+v"(ln));
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        const int row = 128 * (p >> 2) + 32 * wv + 8 * (p & 3) + (ln >> 3);
        vp[p] = row < ct.rows ? index_of(co, row) * ldp + (uint32_t)(((ln & 7) ^ swz(row)) << 4) : kOut;
      }
      int g2 = cg;
      index_copy(tile_at(g2, co + 1), co + 1);
    } else {
      rp[0] = rsrc(a.P + (int64_t)ct.m0 * (ldp / 2), (uint32_t)ct.rows * ldp);
    }
    aim_block();
  };
  // copy c of region R (0, 1: A0, A1; 2, 3: B0, B1) of K block ck into stage st
  auto copy_rows = [&](auto R_, auto C_, uint32_t st) __attribute__((always_inline)) {
    constexpr int R = decltype(R_)::value, C = decltype(C_)::value;
    const uint32_t m = m0_w + st * STAGE + R * REG + C * 1024;
    if (R >= 2) {
      const bool past = !QT && (ck * 64 >= ct.kc || (ck == ct.nkb - 1 && cut_q[C & 1]));
      copy16(rq[R & 1], past ? kOut : vq[C], QT ? 0 : (uint32_t)ck * 128, m);
    } else {
      const bool past = !PT && (ck * 64 >= ct.kc || (ck == ct.nkb - 1 && cut_p[C & 1]));
      copy16(rp[PT ? R & 1 : 0], past ? kOut : vp[PT ? C : (4 * R + C) & 7], PT ? 0 : (uint32_t)ck * 128, m);
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
  // region begin at 32 wm (P), 32 wn (Q) and 64 further.
  uint32_t o[4];
#pragma unroll
  for (int ks = 0; ks < 4; ++ks)
    o[ks] = (uint32_t)(l32 * 128 + (((2 * ks + q) ^ swz(l32)) << 4));
  const uint32_t otr = tr_lane(lane);
  v4i fr[4][2][4];  // operands of A0, A1, B0, B1: [block][ks]
  auto read_one = [&](auto R_, int n, uint32_t st) __attribute__((always_inline)) {
    constexpr int R = decltype(R_)::value;
    const uint8_t* p = smem + st * STAGE + R * REG;
    const int w = R >= 2 ? wn : wm;
    if (R >= 2 ? QT : PT)
      fr[R][n & 1][n >> 1] = tr_read(p, otr, w + 2 * (n & 1), n >> 1);
    else
      fr[R][n & 1][n >> 1] = *reinterpret_cast<const v4i*>(p + w * 32 * 128 + o[n >> 1] + (n & 1) * 64 * 128);
  };
  auto clear_past = [&](auto R_, int left) __attribute__((always_inline)) {
    constexpr int R = decltype(R_)::value;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      fr[R][0][ks] = keep_first(fr[R][0][ks], left - 16 * ks - 8 * q);
      fr[R][1][ks] = keep_first(fr[R][1][ks], left - 16 * ks - 8 * q);
    }
  };

  v16f acc[2][2][2][2];  // [A half][B half][A block][B block]

  // ---- epilogue.  Lane (q, l32) holds row l32 of a block and its columns 8 e
  // + 4 q .. +3; through the wave's own 4 KB of LDS (16-byte chunk c of a
  // row in slot c ^ row % 8) a lane gets 8 columns of rows lane / 4 and + 16.
  const uint32_t e_wr = OFF_OUT + wv * 4096 + l32 * 128;
  const uint32_t e_rd = OFF_OUT + wv * 4096 + (lane >> 2) * 128;
  auto turn = [&](const v16f& c, float (&v)[2][8]) __attribute__((always_inline)) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      *reinterpret_cast<float4*>(smem + e_wr + (((2 * e + q) ^ (l32 & 7)) << 4)) =
          make_float4(c[4 * e], c[4 * e + 1], c[4 * e + 2], c[4 * e + 3]);
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 w = *reinterpret_cast<const float4*>(
            smem + e_rd + r * 2048 + (((2 * (lane & 3) + h) ^ ((lane >> 2) & 7)) << 4));
        v[r][4 * h] = w.x, v[r][4 * h + 1] = w.y, v[r][4 * h + 2] = w.z, v[r][4 * h + 3] = w.w;
      }
  };
  typedef uint32_t v4u __attribute__((ext_vector_type(4)));
  auto pack8 = [](const float* v) {
    return v4u{f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]), f32x2_to_bf16x2(v[4], v[5]),
               f32x2_to_bf16x2(v[6], v[7])};
  };
  auto unpack8 = [](const v4u& w, float* v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = bf16_to_f32(w[i] & 0xFFFFu), v[2 * i + 1] = bf16_to_f32(w[i] >> 16);
  };
  auto finish = [&](const Tile& t) __attribute__((always_inline)) {
#pragma unroll
    for (int H = 0; H < 2; ++H)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int B = 0; B < (GLU ? 1 : 2); ++B)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int r0 = 128 * H + 64 * i + 32 * wm + (lane >> 2);
            const int64_t c = t.n0 + 128 * B + 64 * j + 32 * wn + 8 * (lane & 3);
            float v[2][8], w[2][8];
            turn(acc[H][B][i][j], v);
            if (GLU) turn(acc[H][1][i][j], w);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              if (r0 + 16 * r >= t.rows || c >= NC) continue;
              const int64_t row = (int64_t)t.m0 + r0 + 16 * r;
              if (MODE == kWgrad) {
                float4* out = reinterpret_cast<float4*>(static_cast<float*>(a.out) + ((int64_t)t.g * a.N + row) * NC + c);
                out[0] = make_float4(v[r][0], v[r][1], v[r][2], v[r][3]);
                out[1] = make_float4(v[r][4], v[r][5], v[r][6], v[r][7]);
              } else if (MODE == kGlu) {
                if (a.keep) {
                  *reinterpret_cast<v4u*>(a.keep + row * 2 * NC + c) = pack8(v[r]);
                  *reinterpret_cast<v4u*>(a.keep + row * 2 * NC + NC + c) = pack8(w[r]);
                }
#pragma unroll
                for (int k = 0; k < 8; ++k) v[r][k] = glu(v[r][k], w[r][k], a.act);
                *reinterpret_cast<v4u*>(static_cast<uint16_t*>(a.out) + row * NC + c) = pack8(v[r]);
              } else if (MODE == kDgradGlu) {
                float g[8], u[8];
                unpack8(*reinterpret_cast<const v4u*>(a.gu_in + row * 2 * NC + c), g);
                unpack8(*reinterpret_cast<const v4u*>(a.gu_in + row * 2 * NC + NC + c), u);
#pragma unroll
                for (int k = 0; k < 8; ++k) glu_backward(g[k], u[k], v[r][k], a.act, &v[r][k], &w[r][k]);
                uint16_t* out = static_cast<uint16_t*>(a.out) + row * 2 * NC + c;
                *reinterpret_cast<v4u*>(out) = pack8(v[r]);
                *reinterpret_cast<v4u*>(out + NC) = pack8(w[r]);
              } else {
                *reinterpret_cast<v4u*>(static_cast<uint16_t*>(a.out) + row * NC + c) = pack8(v[r]);
              }
            }
          }
  };

  // ---- prologue: the first two K blocks, in the order they are read
  int t_g = 0, to = 0;
  Tile t = tile_at(t_g, 0);
  if (GATHER) {
    if (PT) {
      xt = t;
      xg = t_g;
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
  wait_copies<20>();
  barrier();

  // A phase: MFMAs of A half H and B half B; reads region R of stage rst for
  // the next one (early, so that the wait at its end finds them done), copies
  // region CR into stage cst.  FIRST: from zero.  The wait that ends it leaves
  // the newest 24 on their way, the copies of six phases: what the next phase
  // reads was copied before them.  Stores and index copies among them make
  // the wait stricter.
  auto phase = [&](auto H_, auto B_, auto R_, uint32_t rst, auto CR_, uint32_t cst, auto FIRST_)
                   __attribute__((always_inline)) {
    constexpr int H = decltype(H_)::value, B = decltype(B_)::value;
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
    wait_copies<24>();
    __builtin_amdgcn_sched_barrier(0);
    barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  uint32_t st = 0;  // stage of the K block being multiplied
  auto block = [&](auto FIRST_, int left) __attribute__((always_inline)) {
    if (left < 64) {
      clear_past(ic<0>(), left);
      clear_past(ic<2>(), left);
    }
    phase(ic<0>(), ic<0>(), ic<3>(), st, ic<2>(), st, FIRST_);
    if (left < 64) clear_past(ic<3>(), left);
    phase(ic<0>(), ic<1>(), ic<1>(), st, ic<3>(), st, FIRST_);
    if (left < 64) clear_past(ic<1>(), left);
    phase(ic<1>(), ic<0>(), ic<0>(), st ^ 1, ic<1>(), st, FIRST_);
    copy_next();
    phase(ic<1>(), ic<1>(), ic<2>(), st ^ 1, ic<0>(), st ^ 1, FIRST_);
    st ^= 1;
  };
  for (; to < my_n; t = tile_at(t_g, ++to)) {
    block(ic<1>(), t.kc);
    for (int k = 1; k < t.nkb; ++k) block(ic<0>(), t.kc - 64 * k);
    finish(t);
  }
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
