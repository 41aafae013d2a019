// Grouped int8 product with too few 256 x 256 tiles for the CUs: 128 x 128
// tiles, four waves of 64 x 64, v_mfma_i32_32x32x32_i8.
//
// Bound by the latency of each K block, where a tile or two a CU is all there
// is: so the 128-byte K blocks of both operands go through a ring of four
// stages in LDS, three of them on their way (copies straight into LDS), on
// across a workgroup's tiles; one barrier a K block.  One group of 1024 rows, N
// = 4096, K = 7168: 45 to 50 us (65 with 256 x 256 tiles).
#include "int8_common.h"

namespace moe {
namespace int8 {
namespace {

using gemm::barrier;
using gemm::build_group_tables;
using gemm::MAXG;
using gemm::swz;

constexpr int MT = 256;
constexpr int BM = 128, BN = 128;
constexpr int S = 4;                           // stages
constexpr int STAGE = (BM + BN) * 128;
constexpr int AC = BM / 32, BC = BN / 32;      // copies of a wave and K block
constexpr int MI = BM / 64;                    // row blocks of a wave

__device__ __forceinline__ v4i rsrc(const void* p, uint32_t bytes) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  v4i r;
  r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)a);
  r[1] = __builtin_amdgcn_readfirstlane((int)(uint32_t)(a >> 32));
  r[2] = __builtin_amdgcn_readfirstlane((int)bytes);
  r[3] = 0x00020000;
  return r;
}
// Lane i's 16 bytes from offset voff + soff of the resource land at m0 + 16 i;
// out of range: not read from memory.
__device__ __forceinline__ void copy16(const v4i& r, uint32_t voff, uint32_t soff, uint32_t m0) {
  asm volatile("s_mov_b32 m0, %3\n\tbuffer_load_dwordx4 %0, %1, %2 offen lds"
               ::"v"(voff), "s"(r), "s"(soff), "s"(m0) : "memory", "m0");
}
template <int N>
__device__ __forceinline__ void wait_copies() {
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4));
}

template <bool SWIGLU>
__global__ __launch_bounds__(MT, 1) void mid_kernel(Args a) {
  constexpr int TN = SWIGLU ? BN / 2 : BN;
  __shared__ __attribute__((aligned(16))) uint8_t smem[S * STAGE];
  __shared__ int s_offs[MAXG + 1];
  __shared__ int s_pref[MAXG + 1];
  __shared__ int s_red[4];
  __shared__ int s_carry;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wv >> 1, wn = wv & 1, q = lane >> 5, l32 = lane & 31;
  const int64_t N = a.N;
  const uint32_t K = (uint32_t)a.K;
  const int nkb = (int)((K + 127) >> 7);
  const int64_t ntiles = (N + TN - 1) / TN;
  const int64_t b_rows = SWIGLU ? 2 * N : N;
  build_group_tables<MT, BM>(a.offs, a.G, s_offs, s_pref, s_red, &s_carry);
  const int64_t total = (int64_t)s_pref[a.G] * ntiles;
  // an XCD's workgroups (blockIdx % 8) take a contiguous range of tiles, the
  // row tiles of one weight panel next to each other
  const int nper = gridDim.x >> 3;
  const int64_t tlo = total * (blockIdx.x & 7) / 8, thi = total * ((blockIdx.x & 7) + 1) / 8;
  const int64_t L0 = tlo + (blockIdx.x >> 3);
  if (L0 >= thi) return;
  const int my_n = (int)((thi - L0 + nper - 1) / nper);
  struct Place {
    int g, m0, rows, n0;
  };
  auto place = [&](int o) {  // (past the last: the last)
    const gemm::Tile t =
        gemm::decode_tile(s_pref, s_offs, a.G, ntiles, L0 + (int64_t)min(o, my_n - 1) * nper, BM);
    Place p;
    p.g = __builtin_amdgcn_readfirstlane(t.g);
    p.m0 = __builtin_amdgcn_readfirstlane(t.m0);
    p.rows = __builtin_amdgcn_readfirstlane(min(BM, t.m1 - t.m0));
    p.n0 = __builtin_amdgcn_readfirstlane((int)t.nt * TN);
    return p;
  };
  auto source = [&](int row) -> int64_t {
    return a.index ? (int64_t)min((uint32_t)a.index[row], (uint32_t)(a.A_rows - 1)) : row;
  };

  // ---- copies: 8 rows each, lane -> row + lane / 8, LDS slot lane % 8 <-
  // 16-byte chunk (lane % 8) ^ swz.  Wave wv moves rows (BM / 4) wv .. of A and
  // 32 wv .. of B.  Lanes past the tile's rows and columns repeat the last
  // ones'; those past a row's end in the last K block read its last bytes,
  // and their K positions are cleared in A's registers.
  const uint32_t lds0 = (uint32_t)(uintptr_t)smem;
  const int tail = (int)((K & 127) >> 4);  // 16-byte chunks of the last K block, 0: all 8
  int co = 0, ck = 0;
  uint32_t cs = 0;
  v4i ra, rb;
  uint32_t va[AC], vb[BC];
  auto aim = [&]() {
    const Place p = place(co);
    const int64_t cols = N - p.n0 < TN ? N - p.n0 : TN;
    rb = rsrc(a.B + ((int64_t)p.g * b_rows + (SWIGLU && wv >= 2 ? N : 0) + p.n0) * K, (uint32_t)(cols * K));
    ra = a.index ? rsrc(a.A, (uint32_t)a.A_rows * K) : rsrc(a.A + (int64_t)p.m0 * K, (uint32_t)p.rows * K);
#pragma unroll
    for (int c = 0; c < BC; ++c) {
      const int row = 32 * wv + 8 * c + (lane >> 3);
      const int col = SWIGLU ? row & (TN - 1) : row;
      vb[c] = (uint32_t)min<int64_t>(col, cols - 1) * K + (uint32_t)(((lane & 7) ^ swz(row)) << 4);
    }
#pragma unroll
    for (int c = 0; c < AC; ++c) {
      const int row = (BM / 4) * wv + 8 * c + (lane >> 3);
      const int64_t src = source(p.m0 + min(row, p.rows - 1));
      va[c] = (uint32_t)(a.index ? src : src - p.m0) * K + (uint32_t)(((lane & 7) ^ swz(row)) << 4);
    }
  };
  auto copy_block = [&]() __attribute__((always_inline)) {
    const bool last = ck == nkb - 1 && tail;
    const uint32_t so = (uint32_t)ck * 128;
    const uint32_t m = lds0 + cs * STAGE;
#pragma unroll
    for (int c = 0; c < AC; ++c) {
      const int row = (BM / 4) * wv + 8 * c + (lane >> 3), chunk = (lane & 7) ^ swz(row);
      copy16(ra, last && chunk >= tail ? va[c] - (uint32_t)((chunk - tail + 1) << 4) : va[c], so,
             m + (uint32_t)(((BM / 4) * wv + 8 * c) * 128));
    }
#pragma unroll
    for (int c = 0; c < BC; ++c) {
      const int row = 32 * wv + 8 * c + (lane >> 3), chunk = (lane & 7) ^ swz(row);
      copy16(rb, last && chunk >= tail ? vb[c] - (uint32_t)((chunk - tail + 1) << 4) : vb[c], so,
             m + (uint32_t)(BM * 128 + (32 * wv + 8 * c) * 128));
    }
    cs = cs + 1 == S ? 0 : cs + 1;
    if (++ck == nkb) {
      ck = 0;
      ++co;
      aim();
    }
  };

  uint32_t o[4];  // lane (q, l32): chunk 2 ks + q of row l32 of a 32-row block
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) o[ks] = (uint32_t)(l32 * 128 + (((2 * ks + q) ^ swz(l32)) << 4));
  v16i acc[MI][2];
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0;
  };
  // lane (q, l32): token row l32 of a block, columns 8 g + 4 q .. +3 of a block
  auto finish = [&](const Place& p) __attribute__((always_inline)) {
    const float* sb = a.sb + (int64_t)p.g * b_rows + p.n0;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int row = 32 * wm + 64 * i + l32;
      if (row >= p.rows) continue;
      const float sa = a.sa[source(p.m0 + row)];
      uint16_t* out = a.C + (int64_t)(p.m0 + row) * N + p.n0;
#pragma unroll
      for (int j = 0; j < (SWIGLU ? 1 : 2); ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int c = (BN / 2) * j + 32 * wn + 8 * g + 4 * q;
          if (p.n0 + c >= N) continue;
          float v[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            v[r] = (float)acc[i][j][4 * g + r] * (sa * sb[c + r]);
            if (SWIGLU) v[r] = silu_mul(v[r], (float)acc[i][1][4 * g + r] * (sa * sb[N + c + r]));
          }
          *reinterpret_cast<uint2*>(out + c) = make_uint2(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]));
        }
    }
  };

  aim();
#pragma unroll
  for (int s = 0; s < S - 1; ++s) copy_block();
  clear();
  int t_o = 0, t_k = 0;
  Place p = place(0);
  uint32_t st = 0;
  const int blocks = my_n * nkb;
  for (int blk = 0; blk < blocks; ++blk) {
    // this block's copies have landed (those of S - 2 blocks come after them),
    // and everyone is past the block whose stage is filled next
    wait_copies<(S - 2) * (AC + BC)>();
    barrier();
    copy_block();
    const uint8_t* pa = smem + st * STAGE + wm * 32 * 128;
    const uint8_t* pb = smem + st * STAGE + BM * 128 + wn * 32 * 128;
    const bool last = t_k == nkb - 1;
    v4i fa[MI][4], fb[2][4];
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
#pragma unroll
      for (int j = 0; j < 2; ++j) fb[j][ks] = *reinterpret_cast<const v4i*>(pb + o[ks] + j * (BN / 2) * 128);
#pragma unroll
      for (int i = 0; i < MI; ++i) fa[i][ks] = *reinterpret_cast<const v4i*>(pa + o[ks] + i * 64 * 128);
    }
    if (last && tail)
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
        if (2 * ks + q >= tail)
#pragma unroll
          for (int i = 0; i < MI; ++i) fa[i][ks] = v4i{0, 0, 0, 0};
#pragma unroll
    for (int ks = 0; ks < 4; ++ks)
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[j][ks], fa[i][ks], acc[i][j], 0, 0, 0);
    st = st + 1 == S ? 0 : st + 1;
    if (last) {
      finish(p);
      clear();
      t_k = 0;
      p = place(++t_o);
    } else {
      ++t_k;
    }
  }
  wait_copies<0>();  // what was copied past the last tile lands before the LDS is released
}

}  // namespace

void launch_mid(const Args& a, bool swiglu, hipStream_t st) {
  const dim3 grid(std::max(8, gemm::num_cus() / 8 * 8)), block(MT);
  if (swiglu) mid_kernel<true><<<grid, block, 0, st>>>(a);
  else mid_kernel<false><<<grid, block, 0, st>>>(a);
}

}  // namespace int8
}  // namespace moe
