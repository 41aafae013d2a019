// Grouped int8 product for groups of many rows: 256 x 256 output tiles, eight
// waves, v_mfma_i32_32x32x32_i8, bf16 or SwiGLU epilogue.
//
// The matrix cores take 8192 operations a clock and CU, so a 128-byte K block
// of a tile (2 * 256 * 256 * 128 operations) takes 2048 clocks and 64 KB of
// operands: at full rate a CU reads 32 B a clock from L2, and a copy has to
// be on its way for as long as L2 and HBM take under that load.  Hence:
//  * LDS holds two K blocks in four regions each (tile rows 0..127 and
//    128..255 of A: A0, A1; weight rows of the tile's two column halves: B0,
//    B1 - gate and up with SwiGLU).  A K block is worked on in four phases,
//    A0 B0, A0 B1, A1 B0, A1 B1 (8 MFMAs of a wave each).  A region is free
//    as soon as every wave has its operands in registers, one phase after it
//    was read, and is then filled for the K block after the next: a copy has
//    seven phases, most of two K blocks, to land.
//  * The two waves of a SIMD take turns: while one multiplies (a slot of 8
//    MFMAs, 256 clocks) the other reads its next operands from LDS, issues
//    two copies and waits for what it reads next; a barrier ends each slot.
//    Waves 4..7 run one slot behind waves 0..3.
//  * Copies run on across tiles: the next tile's first two K blocks load
//    while the last ones of this tile are multiplied, and the epilogue of a
//    half (A0, A1) follows the phase that completes it.
//  * Persistent workgroups; those of an XCD (blockIdx % 8) share a contiguous
//    range of tiles, M tiles of one weight panel next to each other, so they
//    share its L2.
// Every copy goes through a buffer resource over the rows it may touch; lanes
// with nothing to read (rows past a tile's end, the last K block past a row's
// end) have an offset outside it, and what their slots hold is not used: such
// rows are not stored, such K positions are cleared in A's registers.
#include "int8_common.h"

namespace moe {
namespace int8 {
namespace {

using gemm::barrier;
using gemm::build_group_tables;
using gemm::MAXG;
using gemm::swz;

constexpr int WT = 512;
constexpr int REG = 128 * 128;      // a region: 128 rows x 128 B
constexpr int STAGE = 4 * REG;      // A0, A1, B0, B1
constexpr int OFF_OUT = 2 * STAGE;  // per wave 32 rows x 64 B
constexpr int OFF_PREF = OFF_OUT + 8 * 2048;
constexpr int OFF_OFFS = OFF_PREF + 4112;
constexpr int OFF_IDX = OFF_OFFS + 4112;    // int [2][256]
constexpr int OFF_SC = OFF_IDX + 2 * 1024;  // float [2][sa 256, sb 256]
constexpr int LDS = OFF_SC + 2 * 2048;
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
__device__ __forceinline__ void copy16(const v4i& r, uint32_t voff, uint32_t soff, uint32_t m0) {
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

struct Tile {
  int g, n0, m0, rows;
};

template <bool SWIGLU, bool GATHER>
__global__ __launch_bounds__(WT, 1) void wide_kernel(Args a) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[LDS];
  __shared__ int s_red[8];
  __shared__ int s_carry;
  int* s_pref = reinterpret_cast<int*>(smem + OFF_PREF);
  int* s_offs = reinterpret_cast<int*>(smem + OFF_OFFS);
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wv >> 2, wn = wv & 3;
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
    const uint32_t nt = rem / cnt;
    Tile t;
    t.g = g;
    t.n0 = __builtin_amdgcn_readfirstlane((int)(nt * TN));
    t.m0 = __builtin_amdgcn_readfirstlane(s_offs[g] + (int)(rem - nt * cnt) * 256);
    t.rows = __builtin_amdgcn_readfirstlane(min(256, s_offs[g + 1] - t.m0));
    return t;
  };
  // valid weight rows of a tile's column half h
  auto cols_of = [&](const Tile& t, int h) -> int {
    return (int)min<int64_t>(128, max<int64_t>(0, SWIGLU ? N - t.n0 : N - t.n0 - 128 * h));
  };

  // ---- copies.  Wave wv moves rows 16 wv .. +15 of a region, 8 rows a copy:
  // lane -> row + lane / 8, LDS slot lane % 8 <- 16-byte chunk (lane % 8) ^ swz
  const uint32_t lds0 = (uint32_t)(uintptr_t)smem;
  const uint32_t m0_w = (uint32_t)__builtin_amdgcn_readfirstlane((int)(lds0 + (uint32_t)wv * 2048));
  auto crow = [&](int c) -> int { return 16 * wv + 8 * c + (lane >> 3); };
  const int tail = (int)((K & 127) >> 4);  // 16-byte chunks of the last K block, 0: all 8
  constexpr uint32_t kOut = 0xFFFFFF00u;   // an offset outside every resource
  uint32_t vb[2];     // lane offsets of the two copies of a region of B
  uint32_t va[4];     // of A0's and A1's copies
  bool cut[2];        // the lane's chunk lies past the row's end in the last K block
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const int chunk = (lane & 7) ^ swz(crow(c));
    vb[c] = (uint32_t)crow(c) * K + (uint32_t)(chunk << 4);
    va[c] = vb[c];
    va[2 + c] = vb[c] + 128 * K;
    cut[c] = tail && chunk >= tail;
  }
  const uint32_t a_last = (uint32_t)(a.A_rows - 1);

  // the copies' place: K block ck of the tile of ordinal co
  int co = 0, ck = 0, cg = 0;
  v4i ra, rb[2];
  auto index_copy = [&](const Tile& t, int o) {  // the row indices of a tile into slot o & 1
    if (wv < 4)
      copy4(rsrc(a.index + t.m0, (uint32_t)t.rows * 4), (uint32_t)(64 * wv + lane) * 4,
            (uint32_t)__builtin_amdgcn_readfirstlane((int)(lds0 + OFF_IDX + (o & 1) * 1024 + wv * 256)));
  };
  auto index_of = [&](int o, int row) -> uint32_t {
    return min((uint32_t)reinterpret_cast<const int*>(smem + OFF_IDX)[(o & 1) * 256 + row], a_last);
  };
  auto copy_tile = [&]() {  // sources of tile co
    const Tile t = tile_at(cg, co);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      // (a half without columns copies the other's rows; K offsets never lie
      // past a resource's end)
      const int hh = h && cols_of(t, 1) > 0;
      rb[h] = rsrc(a.B + ((int64_t)t.g * b_rows + t.n0 + hh * b_half) * K, (uint32_t)cols_of(t, hh) * K);
    }
    if (GATHER) {
      ra = rsrc(a.A, (uint32_t)a.A_rows * K);
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const int row = 128 * (p >> 1) + crow(p & 1);
        va[p] = row < t.rows
                    ? index_of(co, row) * K + (uint32_t)(((lane & 7) ^ swz(row)) << 4)
                    : kOut;
      }
      int g2 = cg;
      index_copy(tile_at(g2, co + 1), co + 1);
    } else {
      ra = rsrc(a.A + (int64_t)t.m0 * K, (uint32_t)t.rows * K);
    }
  };
  // region R (0, 1: A0, A1; 2, 3: B0, B1) of K block ck into stage st
  auto copy_region = [&](auto R_, uint32_t st) __attribute__((always_inline)) {
    constexpr int R = decltype(R_)::value;
    const uint32_t so = (uint32_t)ck * 128;
    const uint32_t m = m0_w + st * STAGE + R * REG;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const uint32_t v = R >= 2 ? vb[c] : va[2 * (R & 1) + c];
      copy16(R >= 2 ? rb[R & 1] : ra, ck == nkb - 1 && cut[c] ? kOut : v, so, m + c * 1024);
    }
  };
  auto copy_next = [&]() {  // to the next K block
    if (++ck == nkb) {
      ck = 0;
      ++co;
      copy_tile();
    }
  };

  // ---- operand reads: lane (q, l32) has 16 bytes (chunk 2 ks + q) of row
  // l32 of a 32-row block; blocks start at multiples of 32 rows
  uint32_t o[4];
#pragma unroll
  for (int ks = 0; ks < 4; ++ks)
    o[ks] = (uint32_t)(l32 * 128 + (((2 * ks + q) ^ swz(l32)) << 4));
  v4i fa[2][4], fb[2][4];
  auto read_a = [&](int h, uint32_t st) __attribute__((always_inline)) {
    const uint8_t* p = smem + st * STAGE + h * REG + wm * 32 * 128;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
        fa[i][ks] = *reinterpret_cast<const v4i*>(p + o[ks] + i * 64 * 128);
  };
  auto read_b = [&](auto H_, uint32_t st) __attribute__((always_inline)) {
    constexpr int H = decltype(H_)::value;
    const uint8_t* p = smem + st * STAGE + (2 + H) * REG + wn * 32 * 128;
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) fb[H][ks] = *reinterpret_cast<const v4i*>(p + o[ks]);
  };
  auto clear_tail = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
      if (2 * ks + q >= tail) {
        fa[0][ks] = v4i{0, 0, 0, 0};
        fa[1][ks] = v4i{0, 0, 0, 0};
      }
  };

  v16i acc[2][2][2];  // [A half][B half][32-row block]
  auto clear = [&](int h) __attribute__((always_inline)) {
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[h][b][i][r] = 0;
  };
  clear(0);
  clear(1);

  // ---- the tile being multiplied
  int t_g = 0, to = 0, tk = 0;
  Tile t = tile_at(t_g, 0);
  auto scale_copy = [&]() {  // its scales: 64 a wave, rows from waves 0..3
    const uint32_t m = (uint32_t)__builtin_amdgcn_readfirstlane(
        (int)(lds0 + OFF_SC + (to & 1) * 2048 + wv * 256));
    if (wv < 4) {
      const int row = 64 * wv + lane;
      if (GATHER)
        copy4(rsrc(a.sa, (uint32_t)a.A_rows * 4), row < t.rows ? index_of(to, row) * 4 : kOut, m);
      else
        copy4(rsrc(a.sa + t.m0, (uint32_t)t.rows * 4), (uint32_t)row * 4, m);
    } else {
      const int h = (wv >> 1) & 1;
      copy4(rsrc(a.sb + (int64_t)t.g * b_rows + t.n0 + h * b_half, (uint32_t)cols_of(t, h) * 4),
            (uint32_t)(64 * (wv & 1) + lane) * 4, m);
    }
  };
  // rows 128 h + 64 i + 32 wm .. +31 (i = 0, 1) of the tile
  auto live = [&](int h, int i) { return 128 * h + 64 * i + 32 * wm < t.rows; };

  // Results of A half h: lane (q, l32) holds token row l32 of a block and the
  // columns 8 g + 4 q .. +3 (g = 0..3) of its 32.  Through the wave's own 2 KB
  // of LDS (16-byte chunk c of row r in slot c ^ (r / 2) % 4) into rows of 64
  // bytes.  The fp32 result is rounded once, to bf16.
  auto epilogue = [&](auto H_, auto B_) __attribute__((always_inline)) {
    constexpr int H = decltype(H_)::value, B = decltype(B_)::value;
    const float* sc = reinterpret_cast<const float*>(smem + OFF_SC + (to & 1) * 2048);
    uint8_t* out = smem + OFF_OUT + wv * 2048;
    const __amdgpu_buffer_rsrc_t rc = __builtin_amdgcn_make_buffer_rsrc(
        a.C + (int64_t)t.m0 * N, 0, (int)((uint32_t)t.rows * (uint32_t)N * 2), 0x00020000);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (!live(H, i)) continue;
      const int row0 = 128 * H + 64 * i + 32 * wm;
      const float sa = sc[row0 + l32];
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const float4 s0 = *reinterpret_cast<const float4*>(sc + 256 + (SWIGLU ? 0 : 128 * B) + 32 * wn + 8 * g + 4 * q);
        const float w0[4] = {s0.x, s0.y, s0.z, s0.w};
        float v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = (float)acc[H][SWIGLU ? 0 : B][i][4 * g + r] * (sa * w0[r]);
        if (SWIGLU) {
          const float4 s1 = *reinterpret_cast<const float4*>(sc + 256 + 128 + 32 * wn + 8 * g + 4 * q);
          const float w1[4] = {s1.x, s1.y, s1.z, s1.w};
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] = silu_mul(v[r], (float)acc[H][1][i][4 * g + r] * (sa * w1[r]));
        }
        *reinterpret_cast<uint2*>(out + l32 * 64 + ((g ^ ((l32 >> 1) & 3)) << 4) + 8 * q) =
            make_uint2(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]));
      }
      const int col = t.n0 + (SWIGLU ? 0 : 128 * B) + 32 * wn + 8 * (lane & 3);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = 16 * r + (lane >> 2);
        const uint4 d = *reinterpret_cast<const uint4*>(out + row * 64 + (((lane & 3) ^ ((row >> 1) & 3)) << 4));
        typedef uint32_t v4u __attribute__((ext_vector_type(4)));
        const v4u w = {d.x, d.y, d.z, d.w};
        if (col < N)
          __builtin_amdgcn_raw_buffer_store_b128(w, rc, ((row0 + row) * (int)N + col) * 2, 0, 0);
      }
    }
  };

  // ---- prologue: the first two K blocks, in the order they are read
  if (GATHER) {
    index_copy(t, 0);
    wait_copies<0>();
    barrier();
  }
  copy_tile();
  copy_region(ic<2>(), 0);
  copy_region(ic<0>(), 0);
  copy_region(ic<3>(), 0);
  copy_region(ic<1>(), 0);
  copy_next();
  copy_region(ic<2>(), 1);
  copy_region(ic<0>(), 1);
  copy_region(ic<3>(), 1);
  copy_region(ic<1>(), 1);
  wait_copies<12>();
  barrier();
  read_b(ic<0>(), 0);
  wait_copies<12>();
  barrier();
  if (wm) barrier();  // waves 4..7: one slot behind

  auto multiply = [&](auto H_, auto B_) __attribute__((always_inline)) {
    constexpr int H = decltype(H_)::value, B = decltype(B_)::value;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (live(H, i)) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          acc[H][B][i] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[B][ks], fa[i][ks], acc[H][B][i], 0, 0, 0);
      }
  };
  // end of a slot: this slot's reads are in registers, the copies that the
  // next phase reads have landed (six phases of two copies come after them)
  auto slot_read = [&]() __attribute__((always_inline)) {
    wait_copies<12>();
    __builtin_amdgcn_sched_barrier(0);
    barrier();
    __builtin_amdgcn_s_setprio(1);
  };
  auto slot_multiply = [&]() __attribute__((always_inline)) {
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
    barrier();
    __builtin_amdgcn_sched_barrier(0);
  };

  uint32_t st = 0;  // stage of the K block being multiplied
  const int blocks = my_n * nkb;
  for (int blk = 0; blk < blocks; ++blk) {
    const bool last = tk == nkb - 1;
    // A0 B0; copies of K block + 2 begin
    read_a(0, st);
    if (tk == 0) scale_copy();  // before copy_next: it reads the index slot that a next tile may take
    copy_next();
    copy_region(ic<2>(), st);
    if (last && tail) clear_tail();
    slot_read();
    multiply(ic<0>(), ic<0>());
    slot_multiply();
    // A0 B1
    read_b(ic<1>(), st);
    copy_region(ic<0>(), st);
    slot_read();
    multiply(ic<0>(), ic<1>());
    slot_multiply();
    // A1 B0
    if (last) {
      if (!SWIGLU) epilogue(ic<0>(), ic<0>());
      epilogue(ic<0>(), ic<1>());
      clear(0);
    }
    read_a(1, st);
    copy_region(ic<3>(), st);
    if (last && tail) clear_tail();
    slot_read();
    multiply(ic<1>(), ic<0>());
    slot_multiply();
    // A1 B1; B0 of the next K block
    read_b(ic<0>(), st ^ 1);
    copy_region(ic<1>(), st);
    slot_read();
    multiply(ic<1>(), ic<1>());
    slot_multiply();
    st ^= 1;
    if (last) {
      if (!SWIGLU) epilogue(ic<1>(), ic<0>());
      epilogue(ic<1>(), ic<1>());
      clear(1);
      tk = 0;
      t = tile_at(t_g, ++to);
    } else {
      ++tk;
    }
  }
  if (!wm) barrier();
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
