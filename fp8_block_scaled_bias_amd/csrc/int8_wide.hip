// Grouped int8 product for groups of many rows: 256 x 256 output tiles, four
// waves of 128 x 128, v_mfma_i32_32x32x32_i8, bf16 or SwiGLU epilogue.
//
// The matrix cores take 8192 operations a clock and CU, so a 128-byte K block
// of a tile (2 * 256 * 256 * 128 operations) takes 2048 clocks and 64 KB of
// operands: at full rate a CU reads 32 B a clock from L2, and a copy has to
// be on its way for as long as L2 and HBM take under that load.  LDS moves 128
// B a clock: the 64 KB that come in and the 128 KB that four waves of 128 x
// 128 read take 1536 of the 2048 clocks (eight waves of 128 x 64 would read
// 192 KB and fill them all).  Hence:
//  * One wave a SIMD with the accumulators in its 256 AGPRs and the operands
//    of a K block, 128 registers, in its VGPRs.
//  * LDS holds two K blocks in four regions each (tile rows 0..127 and
//    128..255 of A: A0, A1; weight rows of the tile's two column halves: B0,
//    B1 - gate and up with SwiGLU).  A K block is worked on in four phases,
//    A0 B0, A0 B1, A1 B0, A1 B1, of 16 MFMAs (512 clocks) a wave.  Between
//    its MFMAs a phase reads the operands that the next one adds (B1, A1,
//    then A0 and B0 of the next K block), and copies into the region that
//    the phase before read, for the K block after the next: a copy has six
//    phases, a K block and a half, to land.  A barrier ends each phase; the last MFMA
//    covers it.
//  * Copies run on across tiles: the next tile's first two K blocks load
//    while the last ones of this tile are multiplied.
//  * Persistent workgroups; those of an XCD (blockIdx % 8) share a contiguous
//    range of tiles.  A group's tiles are numbered in strips of 8 M tiles, N
//    tile by N tile, so that the 32 tiles at work on an XCD read 8 row and 4
//    weight panels through its L2.
//  * The epilogue runs between MFMAs too: A0's results while the last K block
//    works on A1, A1's while the next tile's first works on A0.
// Every copy goes through a buffer resource over the rows it may touch; lanes
// with nothing to read (rows past a tile's end, the last K block past a row's
// end) have an offset outside it, and what their slots hold is not used: such
// rows are not stored, such K positions are cleared in A's registers.
//
// Measured (two cards): 8192 x 8192 x 8192 in 414 to 428 us, 2.6 POP/s, the
// matrix cores busy 74 to 78 % of the cycles at the 1.56 GHz that the power
// allows; 256 groups of 512 rows, N = 7168, K = 2048 in 1.84 to 1.90 ms, 2.0 to
// 2.1 POP/s (65 %); the same with SwiGLU, I = 2048, K = 7168, gathered, in 3.34
// to 3.48 ms, 2.2 to 2.3 POP/s.
#include "int8_common.h"
#include "int8_wide_waits.h"

namespace moe {
namespace int8 {
namespace {

using gemm::barrier;
using gemm::build_group_tables;
using gemm::copy16;
using gemm::copy4;
using gemm::load_rsrc;
using gemm::MAXG;
using gemm::swz;
using gemm::wait_copies;

constexpr int WT = 256;
constexpr int REG = 128 * 128;      // a region: 128 rows x 128 B
constexpr int STAGE = 4 * REG;      // A0, A1, B0, B1
constexpr int STRIP = 8;            // M tiles of a strip
constexpr int OFF_OUT = 2 * STAGE;  // per wave 32 rows x 64 B
constexpr int OFF_PREF = OFF_OUT + 4 * 2048;
constexpr int OFF_OFFS = OFF_PREF + 4112;
constexpr int OFF_IDX = OFF_OFFS + 4112;    // int [4 tiles][256]
constexpr int OFF_SC = OFF_IDX + 4 * 1024;  // float [2][sa 256, sb 256]
constexpr int LDS = OFF_SC + 2 * 2048;
static_assert((MAXG + 1) * 4 <= 4112 && LDS <= 160 * 1024 - 256, "LDS budget");

template <int V>
using ic = std::integral_constant<int, V>;

struct Tile {
  int g, n0, m0, rows;
};

template <bool SWIGLU, bool GATHER>
__global__ __launch_bounds__(WT, 1) void wide_kernel(Args a) {
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
  const int64_t N = a.N;
  const uint32_t K = (uint32_t)a.K;
  const int nkb = (int)((K + 127) >> 7);
  constexpr int TN = SWIGLU ? 128 : 256;  // output columns of a tile
  const int64_t ntiles = (N + TN - 1) / TN;
  const int64_t b_rows = SWIGLU ? 2 * N : N;  // weight rows of a group
  const int64_t b_half = SWIGLU ? N : 128;    // from B0's rows to B1's

  build_group_tables<WT, 256>(a.offs, G, s_offs, s_pref, s_red, &s_carry);
  const int64_t total = (int64_t)s_pref[G] * ntiles;
  const int xcd = blockIdx.x & 7, jw = blockIdx.x >> 3, nper = gridDim.x >> 3;
  const int64_t tlo = total * xcd / 8, thi = total * (xcd + 1) / 8;
  const int64_t L0 = tlo + jw;
  if (L0 >= thi) return;
  const int my_n = (int)((thi - L0 + nper - 1) / nper);

  // tile of ordinal o (past the last: the last); gh: group of the tile before
  auto tile_at = [&](int& gh, int o) {
    const int64_t L = L0 + (int64_t)min(o, my_n - 1) * nper;
    int g = gh;
    while (g + 1 < G && (int64_t)s_pref[g + 1] * ntiles <= L) ++g;
    gh = g = __builtin_amdgcn_readfirstlane(g);
    const uint32_t cnt = (uint32_t)(s_pref[g + 1] - s_pref[g]);
    const uint32_t rem = (uint32_t)(L - (int64_t)s_pref[g] * ntiles);
    const uint32_t strip = rem / (STRIP * (uint32_t)ntiles), r2 = rem - strip * (STRIP * (uint32_t)ntiles);
    const uint32_t w = min((uint32_t)STRIP, cnt - strip * STRIP), nt = r2 / w;
    Tile t;
    t.g = g;
    t.n0 = __builtin_amdgcn_readfirstlane((int)(nt * TN));
    t.m0 = __builtin_amdgcn_readfirstlane(s_offs[g] + (int)(strip * STRIP + r2 - nt * w) * 256);
    t.rows = __builtin_amdgcn_readfirstlane(min(256, s_offs[g + 1] - t.m0));
    return t;
  };
  // valid weight rows of a tile's column half h
  auto cols_of = [&](const Tile& t, int h) -> int {
    return (int)min<int64_t>(128, max<int64_t>(0, SWIGLU ? N - t.n0 : N - t.n0 - 128 * h));
  };

  // ---- copies.  Wave wv moves rows 32 wv .. +31 of a region, 8 rows a copy:
  // lane -> row + lane / 8, LDS slot lane % 8 <- 16-byte chunk (lane % 8) ^ swz
  const uint32_t lds0 = (uint32_t)(uintptr_t)smem;
  const uint32_t m0_w = (uint32_t)__builtin_amdgcn_readfirstlane((int)(lds0 + (uint32_t)wv * 4096));
  auto crow = [&](int c) -> int { return 32 * wv + 8 * c + (lane >> 3); };
  const int tail = (int)((K & 127) >> 4);  // 16-byte chunks of the last K block, 0: all 8
  constexpr uint32_t kOut = 0xFFFFFF00u;   // an offset outside every resource
  uint32_t vb[4];     // lane offsets of the four copies of a region of B
  uint32_t va[8];     // of A0's and A1's copies
  bool cut[2];        // even, odd copies: the lane's chunk lies past the row's end in the last K block
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const int chunk = (lane & 7) ^ swz(crow(c));
    vb[c] = (uint32_t)crow(c) * K + (uint32_t)(chunk << 4);
    va[c] = vb[c];
    va[4 + c] = vb[c] + 128 * K;
    cut[c & 1] = tail && chunk >= tail;
  }
  const uint32_t a_last = (uint32_t)(a.A_rows - 1);

  // the copies' place: K block ck of the tile of ordinal co
  int co = 0, ck = 0, cg = 0;
  v4i ra, rb[2];
  auto index_copy = [&](const Tile& t, int o) {  // the row indices of a tile into slot o & 3
    copy4(load_rsrc(a.index + t.m0, (uint32_t)t.rows * 4), (uint32_t)(64 * wv + lane) * 4,
          (uint32_t)__builtin_amdgcn_readfirstlane((int)(lds0 + OFF_IDX + (o & 3) * 1024 + wv * 256)));
  };
  auto index_of = [&](int o, int row) -> uint32_t {
    return min((uint32_t)reinterpret_cast<const int*>(smem + OFF_IDX)[(o & 3) * 256 + row], a_last);
  };
  auto copy_tile = [&]() {  // sources of tile co
    const Tile t = tile_at(cg, co);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // (a half without columns copies the other's rows; K offsets never lie
      // past a resource's end)
      const int hh = h && cols_of(t, 1) > 0;
      rb[h] = load_rsrc(a.B + ((int64_t)t.g * b_rows + t.n0 + hh * b_half) * K, (uint32_t)cols_of(t, hh) * K);
    }
    if (GATHER) {
      ra = load_rsrc(a.A, (uint32_t)a.A_rows * K);
      // (the lane's place passes through an empty asm so that what follows
      // is computed here and not kept in registers over the K loop)
      int ln = lane;
      asm volatile("" : "+v"(ln));
#pragma unroll
      for (int p = 0; p < 8; ++p) {
        const int row = 128 * (p >> 2) + 32 * wv + 8 * (p & 3) + (ln >> 3);
        va[p] = row < t.rows ? index_of(co, row) * K + (uint32_t)(((ln & 7) ^ swz(row)) << 4) : kOut;
      }
      int g2 = cg;
      index_copy(tile_at(g2, co + 1), co + 1);
    } else {
      ra = load_rsrc(a.A + (int64_t)t.m0 * K, (uint32_t)t.rows * K);
    }
  };
  // copy c of region R (0, 1: A0, A1; 2, 3: B0, B1) of K block ck into stage st
  auto copy_rows = [&](auto R_, auto C_, uint32_t st) __attribute__((always_inline)) {
    constexpr int R = decltype(R_)::value, C = decltype(C_)::value;
    const uint32_t v = R >= 2 ? vb[C] : va[4 * (R & 1) + C];
    copy16(R >= 2 ? rb[R & 1] : ra, ck == nkb - 1 && cut[C & 1] ? kOut : v, (uint32_t)ck * 128,
           m0_w + st * STAGE + R * REG + C * 1024);
  };
  auto copy_region = [&](auto R_, uint32_t st) __attribute__((always_inline)) {
    copy_rows(R_, ic<0>(), st);
    copy_rows(R_, ic<1>(), st);
    copy_rows(R_, ic<2>(), st);
    copy_rows(R_, ic<3>(), st);
  };
  auto copy_next = [&]() {  // to the next K block
    if (++ck == nkb) {
      ck = 0;
      ++co;
      copy_tile();
    }
  };

  // ---- operand reads: lane (q, l32) has 16 bytes (chunk 2 ks + q) of row
  // l32 of a 32-row block; blocks start at multiples of 32 rows.  The wave's
  // two blocks of a region begin at rows 32 wm (A), 32 wn (B) and 64 further.
  uint32_t o[4];
#pragma unroll
  for (int ks = 0; ks < 4; ++ks)
    o[ks] = (uint32_t)(l32 * 128 + (((2 * ks + q) ^ swz(l32)) << 4));
  v4i fr[4][2][4];  // operands of A0, A1, B0, B1: [block][ks]
  auto read_one = [&](auto R_, int n, uint32_t st) __attribute__((always_inline)) {
    constexpr int R = decltype(R_)::value;
    const uint8_t* p = smem + st * STAGE + R * REG + (R >= 2 ? wn : wm) * 32 * 128;
    fr[R][n & 1][n >> 1] = *reinterpret_cast<const v4i*>(p + o[n >> 1] + (n & 1) * 64 * 128);
  };
  auto clear_tail = [&](auto R_) __attribute__((always_inline)) {
    constexpr int R = decltype(R_)::value;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
      if (2 * ks + q >= tail) {
        fr[R][0][ks] = v4i{0, 0, 0, 0};
        fr[R][1][ks] = v4i{0, 0, 0, 0};
      }
  };

  v16i acc[2][2][2][2];  // [A half][B half][A block][B block]

  // ---- the tile being multiplied
  int t_g = 0, to = 0;
  Tile t = tile_at(t_g, 0);
  auto scale_copy = [&]() {  // its scales: rows and columns 64 wv .. +63
    const uint32_t m = (uint32_t)__builtin_amdgcn_readfirstlane(
        (int)(lds0 + OFF_SC + (to & 1) * 2048 + wv * 256));
    int ln = lane;
    asm volatile("" : "+v"(ln));
    const int row = 64 * wv + ln;
    if (GATHER)
      copy4(load_rsrc(a.sa, (uint32_t)a.A_rows * 4), row < t.rows ? index_of(to, row) * 4 : kOut, m);
    else
      copy4(load_rsrc(a.sa + t.m0, (uint32_t)t.rows * 4), (uint32_t)row * 4, m);
    const int h = wv >> 1;
    copy4(load_rsrc(a.sb + (int64_t)t.g * b_rows + t.n0 + h * b_half, (uint32_t)cols_of(t, h) * 4),
          (uint32_t)(64 * (wv & 1) + ln) * 4, m + 1024);
  };

  // ---- epilogue.  Lane (q, l32) holds token row l32 of a block (i, j) of A
  // half H and B half B (SwiGLU: gate in B0, up in B1) and its columns 8 g +
  // 4 q .. +3 (g = 0..3).  They go through the wave's own 2 KB of LDS (16-byte
  // chunk c of row r in slot c ^ (r / 2) % 4) into rows of 64 bytes.  The fp32
  // result is rounded once, to bf16.  Blocks are taken in the order E = 0 ..
  // NE-1.  Every block is stored, rows and columns past the tile's end to
  // offsets that the hardware drops, so that a phase always issues the same
  // number of stores.
  constexpr int NE = SWIGLU ? 4 : 8;  // blocks of a half
  typedef uint32_t v4u __attribute__((ext_vector_type(4)));
  struct Done {
    Tile t;
    int slot;  // of its scales
  };
  // lane parts of the epilogue's addresses: the scales of a row block and of 4
  // columns, its own rows of LDS written and read, the output
  const uint32_t e_row = OFF_SC + (32 * wm + l32) * 4, e_col = OFF_SC + 1024 + (32 * wn + 4 * q) * 4;
  const uint32_t e_wr = OFF_OUT + wv * 2048 + l32 * 64 + (((l32 >> 1) & 3) << 4) + 8 * q;
  const uint32_t e_rd = OFF_OUT + wv * 2048 + (lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 3) & 3)) << 4);
  const uint32_t e_lcol = 32 * wn + 8 * (lane & 3);
  const uint32_t e_st = ((32 * wm + (lane >> 2)) * (uint32_t)N + e_lcol) * 2;
  // Scales of the 8 results of a slot: gate and up columns of one g with
  // SwiGLU, the columns of two g without; read a slot ahead.
  struct Scales {
    float row;
    float4 col[2];
  };
  auto emit_scales = [&](auto H_, auto S_, const Done& d, Scales& e) __attribute__((always_inline)) {
    constexpr int H = decltype(H_)::value, S = decltype(S_)::value;  // slot 0..15 of a half
    constexpr int per = 16 / NE, E = S / per;
    constexpr int B = E >> 2, i = (E >> 1) & 1, j = E & 1, g = SWIGLU ? S % 4 : 2 * (S % 2);
    const uint8_t* base = smem + d.slot * 2048;
    e.row = *reinterpret_cast<const float*>(base + e_row + (128 * H + 64 * i) * 4);
    const uint8_t* c = base + e_col + (128 * B + 64 * j + 8 * g) * 4;
    e.col[0] = *reinterpret_cast<const float4*>(c);
    e.col[1] = *reinterpret_cast<const float4*>(c + (SWIGLU ? 128 : 8) * 4);
  };
  auto emit_math = [&](auto H_, auto S_, const Scales& e) __attribute__((always_inline)) {
    constexpr int H = decltype(H_)::value, S = decltype(S_)::value;
    constexpr int per = 16 / NE, E = S / per;
    constexpr int B = E >> 2, i = (E >> 1) & 1, j = E & 1, g = SWIGLU ? S % 4 : 2 * (S % 2);
    float v[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float w[4] = {e.col[h].x, e.col[h].y, e.col[h].z, e.col[h].w};
#pragma unroll
      for (int r = 0; r < 4; ++r)
        v[h][r] = (float)(SWIGLU ? acc[H][h][i][j][4 * g + r] : acc[H][B][i][j][4 * (g + h) + r]) * (e.row * w[r]);
    }
    if (SWIGLU) {
#pragma unroll
      for (int r = 0; r < 4; ++r) v[0][r] = silu_mul(v[0][r], v[1][r]);
    }
#pragma unroll
    for (int h = 0; h < (SWIGLU ? 1 : 2); ++h)
      *reinterpret_cast<uint2*>(smem + (e_wr ^ ((g + h) << 4))) =
          make_uint2(f32x2_to_bf16x2(v[h][0], v[h][1]), f32x2_to_bf16x2(v[h][2], v[h][3]));
  };
  auto emit_read = [&](v4u (&w)[2]) __attribute__((always_inline)) {
#pragma unroll
    for (int r = 0; r < 2; ++r) w[r] = *reinterpret_cast<const v4u*>(smem + e_rd + r * 1024);
  };
  // (a resource from the block's first row and column to the tile's last row:
  // offsets of rows past it are outside; columns past N are put outside)
  auto emit_store = [&](auto H_, auto E_, const v4u (&w)[2], const Done& d) __attribute__((always_inline)) {
    constexpr int H = decltype(H_)::value, E = decltype(E_)::value;
    constexpr int B = E >> 2, i = (E >> 1) & 1, j = E & 1;
    const uint32_t c0 = (uint32_t)d.t.n0 + 128 * B + 64 * j;
    const uint32_t off = e_st | (c0 + e_lcol < (uint32_t)N ? 0u : kOut);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int r0 = 128 * H + 64 * i + 16 * r;
      const int bytes = max(0, (d.t.rows - r0) * (int)N - (int)c0) * 2;
      __builtin_amdgcn_raw_buffer_store_b128(
          w[r], __builtin_amdgcn_make_buffer_rsrc(a.C + (int64_t)(d.t.m0 + r0) * N + c0, 0, bytes, 0x00020000),
          off, 0, 0);
    }
  };
  // slot n (0..7) of the first (PART 0) or second (1) phase of a half's epilogue
  Scales es;
  auto emit_slot = [&](auto H_, auto PART_, auto N_, const Done& d) __attribute__((always_inline)) {
    constexpr int PART = decltype(PART_)::value, n = decltype(N_)::value, S = 8 * PART + n;
    constexpr int per = 16 / NE;  // slots of a block
    constexpr int E = S / per, part = S % per;
    constexpr bool stores = part == 0 && E > 0;
    v4u w[2];
    if (S == 0) emit_scales(H_, ic<0>(), d, es);
    if (stores) emit_read(w);
    Scales next;
    if (S < 15) emit_scales(H_, ic<(S < 15 ? S + 1 : 0)>(), d, next);
    emit_math(H_, ic<S>(), es);
    es = next;
    if (stores) emit_store(H_, ic<(stores ? E - 1 : 0)>(), w, d);
    if (S == 15) {
      emit_read(w);
      emit_store(H_, ic<NE - 1>(), w, d);
    }
  };

  // ---- prologue: the first two K blocks, in the order they are read
  if (GATHER) {
    index_copy(t, 0);
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
  wait_copies<waits::prologue(0)>();
  barrier();
#pragma unroll
  for (int n = 0; n < 8; ++n) {
    read_one(ic<0>(), n, 0);
    read_one(ic<2>(), n, 0);
  }
  wait_copies<waits::prologue(1)>();
  barrier();
  copy_next();
  copy_region(ic<0>(), 0);  // A0 of the third
  wait_copies<waits::prologue(2)>();
  barrier();

  // A phase: MFMAs of A half H and B half B; reads region R of stage rst for
  // the next one (early, so that the wait at its end finds them done), copies
  // region CR into stage cst.  FIRST: from zero.  PART 0, 1: part of the
  // epilogue of the other half of d.  W: the wait that ends the phase.
  auto phase = [&](auto H_, auto B_, auto R_, uint32_t rst, auto CR_, uint32_t cst, auto FIRST_,
                   auto PART_, auto W_, const Done& d) __attribute__((always_inline)) {
    constexpr int H = decltype(H_)::value, B = decltype(B_)::value;
    constexpr bool FIRST = decltype(FIRST_)::value;
    auto slot = [&](auto N_) __attribute__((always_inline)) {
      constexpr int n = decltype(N_)::value;
      constexpr int i = n >> 2, ks = n & 3;  // block of A, K chunk
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const v16i zero = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
        acc[H][B][i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(
            fr[2 + B][j][ks], fr[H][i][ks], FIRST && ks == 0 ? zero : acc[H][B][i][j], 0, 0, 0);
      }
      if (n < 4) {
        read_one(R_, 2 * n, rst);
        read_one(R_, 2 * n + 1, rst);
      } else {
        copy_rows(CR_, ic<(n & 3)>(), cst);
      }
      if (decltype(PART_)::value >= 0) emit_slot(ic<1 - H>(), ic<(decltype(PART_)::value & 1)>(), N_, d);
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
  // next phase reads have landed (int8_wide_waits.h).
  uint32_t st = 0;  // stage of the K block being multiplied
  Done done{t, 0};  // the tile before, whose A1 is still to be stored
  done.t.rows = 0;
  auto block = [&](auto FIRST_, auto LAST_) __attribute__((always_inline)) {
    constexpr bool FIRST = decltype(FIRST_)::value, LAST = decltype(LAST_)::value;
    if (FIRST) scale_copy();
    if (LAST && tail) clear_tail(ic<0>());
    phase(ic<0>(), ic<0>(), ic<3>(), st, ic<2>(), st, FIRST_, ic<(FIRST ? 0 : -1)>(),
          ic<waits::phase(SWIGLU, FIRST, LAST, 0)>(), done);
    phase(ic<0>(), ic<1>(), ic<1>(), st, ic<3>(), st, FIRST_, ic<(FIRST ? 1 : -1)>(),
          ic<waits::phase(SWIGLU, FIRST, LAST, 1)>(), done);
    if (LAST) {
      if (tail) clear_tail(ic<1>());
      done = Done{t, to & 1};
    }
    phase(ic<1>(), ic<0>(), ic<0>(), st ^ 1, ic<1>(), st, FIRST_, ic<(LAST ? 0 : -1)>(),
          ic<waits::phase(SWIGLU, FIRST, LAST, 2)>(), done);
    copy_next();
    phase(ic<1>(), ic<1>(), ic<2>(), st ^ 1, ic<0>(), st ^ 1, FIRST_, ic<(LAST ? 1 : -1)>(),
          ic<waits::phase(SWIGLU, FIRST, LAST, 3)>(), done);
    st ^= 1;
  };
  for (; to < my_n; t = tile_at(t_g, ++to)) {
    block(ic<1>(), ic<0>());
    for (int k = 1; k < nkb - 1; ++k) block(ic<0>(), ic<0>());
    block(ic<0>(), ic<1>());
  }
  auto flush = [&](auto N_) __attribute__((always_inline)) {
    emit_slot(ic<1>(), ic<(decltype(N_)::value >> 3)>(), ic<(decltype(N_)::value & 7)>(), done);
    __builtin_amdgcn_sched_barrier(0);
  };
  flush(ic<0>()); flush(ic<1>()); flush(ic<2>()); flush(ic<3>());
  flush(ic<4>()); flush(ic<5>()); flush(ic<6>()); flush(ic<7>());
  flush(ic<8>()); flush(ic<9>()); flush(ic<10>()); flush(ic<11>());
  flush(ic<12>()); flush(ic<13>()); flush(ic<14>()); flush(ic<15>());
  wait_copies<0>();  // what was copied past the last tile lands before the LDS is released
}

}  // namespace

void launch_wide(const Args& a, bool swiglu, hipStream_t st) {
  const dim3 grid(std::max(8, (gemm::num_cus() / 8) * 8)), block(WT);
  if (swiglu) {
    if (a.index) wide_kernel<true, true><<<grid, block, 0, st>>>(a);
    else wide_kernel<true, false><<<grid, block, 0, st>>>(a);
  } else {
    if (a.index) wide_kernel<false, true><<<grid, block, 0, st>>>(a);
    else wide_kernel<false, false><<<grid, block, 0, st>>>(a);
  }
}

}  // namespace int8
}  // namespace moe
