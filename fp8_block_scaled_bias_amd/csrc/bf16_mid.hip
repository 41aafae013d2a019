// Grouped bf16 products in 128 x 128 tiles: four waves of 64 x 64,
// v_mfma_f32_32x32x16_bf16, every mode and size.
//
// A K block of 64 values of both operands (32 KB) goes through a ring of four
// stages in LDS (copies straight into LDS), on across a workgroup's tiles, and
// from there into registers a block before it is multiplied, so that its stage
// is free for the block four further: three are on their way.  One barrier a K
// block.  An operand whose
// contraction runs along its rows lies in 128 rows of 128 B, one whose
// contraction runs down its rows (the weights of an input gradient, both
// operands of a weight gradient) in 64 rows of 256 B, and is read transposed.
// Copies of rows and columns past the ends repeat the last ones; contraction
// values past the end are cleared in the registers of both operands.
#include "bf16_common.h"

namespace moe {
namespace bf16 {
namespace {

using gemm::barrier;
using gemm::build_group_tables;
using gemm::dma16;
using gemm::MAXG;
using gemm::swz;
using gemm::wait_copies;

constexpr int MT = 256;
constexpr int BM = 128, BN = 128;
constexpr int S = 4;                  // stages
constexpr int REG = 128 * 128;        // an operand's K block
constexpr int STAGE = 2 * REG;
constexpr int COPIES = 4;             // of a wave, operand and K block

template <int MODE>
__global__ __launch_bounds__(MT, 1) void mid_kernel(Args a) {
  constexpr bool PT = MODE == kWgrad, QT = MODE >= kDgrad;  // contraction down the rows
  constexpr bool GLU = MODE == kGlu;
  constexpr int TN = GLU ? BN / 2 : BN;
  __shared__ __attribute__((aligned(16))) uint8_t smem[S * STAGE];
  __shared__ int s_offs[MAXG + 1];
  __shared__ int s_pref[MAXG + 1];
  __shared__ int s_red[4];
  __shared__ int s_carry;
  __shared__ int s_idx[PT ? 4 * 4 * 64 : 1];  // kWgrad: a wave's row indices of four K blocks
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wv >> 1, wn = wv & 1, q = lane >> 5, l32 = lane & 31;
  // columns of the output, its row tiles (kWgrad), the contraction's length
  const int64_t NC = MODE == kDgrad || MODE == kDgradGlu || MODE == kWgrad ? a.K : a.N;
  const int64_t ntiles = (NC + TN - 1) / TN, mtiles = (a.N + BM - 1) / BM;
  const int64_t q_rows = (GLU ? 2 : 1) * a.N;  // weight rows of a group
  build_group_tables<MT, BM>(a.offs, a.G, s_offs, s_pref, s_red, &s_carry);
  const int64_t total = PT ? (int64_t)a.G * mtiles * ntiles : (int64_t)s_pref[a.G] * ntiles;
  // an XCD's workgroups (blockIdx % 8) take a contiguous range of tiles, the
  // row tiles of one weight panel next to each other
  const int nper = gridDim.x >> 3;
  const int64_t tlo = total * (blockIdx.x & 7) / 8, thi = total * ((blockIdx.x & 7) + 1) / 8;
  const int64_t L0 = tlo + (blockIdx.x >> 3);
  if (L0 >= thi) return;
  const int my_n = (int)((thi - L0 + nper - 1) / nper);
  struct Place {
    int g, m0, rows, n0;  // group, first row, rows, first column of the tile
    int kc, nkb;          // contraction values, blocks
  };
  auto place = [&](int o) {  // (past the last: the last)
    const int64_t L = L0 + (int64_t)min(o, my_n - 1) * nper;
    Place p;
    if (PT) {
      const int64_t per = mtiles * ntiles, g = L / per, r = L - g * per, nt = r / mtiles;
      p.g = __builtin_amdgcn_readfirstlane((int)g);
      p.m0 = __builtin_amdgcn_readfirstlane((int)(r - nt * mtiles) * BM);
      p.rows = (int)min<int64_t>(BM, a.N - p.m0);
      p.n0 = __builtin_amdgcn_readfirstlane((int)nt * TN);
      p.kc = s_offs[p.g + 1] - s_offs[p.g];
    } else {
      const gemm::Tile t = gemm::decode_tile(s_pref, s_offs, a.G, ntiles, L, BM);
      p.g = __builtin_amdgcn_readfirstlane(t.g);
      p.m0 = __builtin_amdgcn_readfirstlane(t.m0);
      p.rows = min(BM, t.m1 - t.m0);
      p.n0 = __builtin_amdgcn_readfirstlane((int)t.nt * TN);
      p.kc = (int)(QT ? a.N : a.K);
    }
    p.rows = __builtin_amdgcn_readfirstlane(p.rows);
    p.kc = __builtin_amdgcn_readfirstlane(p.kc);
    p.nkb = max(1, (p.kc + 63) >> 6);  // (a group without rows: one block, cleared)
    return p;
  };
  auto source = [&](int64_t row) -> int64_t {
    return a.index ? (int64_t)min((uint32_t)a.index[row], (uint32_t)(a.A_rows - 1)) : row;
  };

  // ---- copies.  Along the rows: 8 rows each, lane -> row + lane / 8, slot
  // lane % 8 <- chunk (lane % 8) ^ swz.  Down the rows: 4 rows each, lane -> row
  // + lane / 16, slot lane % 16 <- chunk (lane % 16) ^ 4 (row % 4).
  const uint32_t lds0 = (uint32_t)(uintptr_t)smem;
  int co = 0, ck = 0;
  uint32_t cs = 0;
  Place cp = place(0);
  // A lane's places in the K block to be copied; they move by a block's bytes.
  const uint8_t* pp[COPIES];
  const uint8_t* pq[COPIES];
  const int64_t step_p = PT ? 128 * a.N : 128, step_q = QT ? 128 * a.K : 128;
  auto aim = [&]() {
    const int64_t cols = min<int64_t>(TN, NC - cp.n0);
    const int64_t k0 = PT ? min<int64_t>(s_offs[cp.g], a.M_total - 1) : 0;
#pragma unroll
    for (int c = 0; c < COPIES; ++c) {
      const int row = 32 * wv + 8 * c + (lane >> 3), along = 8 * ((lane & 7) ^ swz(row));
      const int krow = 16 * wv + 4 * c + (lane >> 4), chunk = (lane & 15) ^ (4 * (krow & 3));
      if (PT)
        pp[c] = reinterpret_cast<const uint8_t*>(a.P + (k0 + krow) * a.N + cp.m0 + min(8 * chunk, cp.rows - 8));
      else
        pp[c] = reinterpret_cast<const uint8_t*>(
            a.P + source((int64_t)cp.m0 + min(row, cp.rows - 1)) * (QT ? a.N : a.K) + along);
      if (QT) {
        // (gathered rows: from the indices, block by block)
        const int64_t at = PT ? (a.index ? 0 : k0 + krow) : (int64_t)cp.g * q_rows + krow;
        pq[c] = reinterpret_cast<const uint8_t*>(a.Q + at * a.K + cp.n0 + min<int64_t>(8 * chunk, cols - 8));
      } else {
        const int64_t col = GLU ? (row & (TN - 1)) : row;
        const int64_t at = (int64_t)cp.g * q_rows + (GLU && row >= TN ? a.N : 0) + cp.n0 + min(col, cols - 1);
        pq[c] = reinterpret_cast<const uint8_t*>(a.Q + at * a.K + along);
      }
    }
  };
  // kWgrad's indices are copied three blocks ahead of the copies that use them
  int xo = 0, xk = 0, xb = 0, cb = 0;
  Place xp = cp;
  auto index_block = [&]() {
    const int64_t row = min<int64_t>((int64_t)s_offs[xp.g] + 64 * xk + lane, a.M_total - 1);
    gemm::dma4(a.index + row, (uint32_t)(uintptr_t)s_idx + (uint32_t)((wv * 4 + (xb & 3)) * 256));
    ++xb;
    if (++xk == xp.nkb) {
      xk = 0;
      xp = place(++xo);
    }
  };
  // copies 2 N and 2 N + 1 of a K block's eight
  uint32_t m_copy = 0;
  int c_left = 0;
  auto copy_begin = [&]() __attribute__((always_inline)) {
    if (PT && a.index) index_block();
    m_copy = lds0 + cs * STAGE + (uint32_t)wv * 4096;
    c_left = max(1, cp.kc - 64 * ck);
  };
  auto copy_pair = [&](int c) __attribute__((always_inline)) {
    const uint8_t *p = pp[c], *w = pq[c];
    const int krow = 16 * wv + 4 * c + (lane >> 4);
    if (PT && a.index)
      w += (int64_t)min((uint32_t)s_idx[(wv * 4 + (cb & 3)) * 64 + krow], (uint32_t)(a.A_rows - 1)) * (2 * a.K);
    if (c_left < 64) {  // what lies past the end: the last values again
      const int row = 32 * wv + 8 * c + (lane >> 3);
      const int along = max(0, 8 * ((lane & 7) ^ swz(row)) - (c_left - 8)) * 2, down = max(0, krow - (c_left - 1));
      p -= PT ? down * (2 * a.N) : along;
      if (!(PT && a.index)) w -= QT ? down * (2 * a.K) : along;
    }
    dma16(p, m_copy + c * 1024);
    dma16(w, m_copy + REG + c * 1024);
    pp[c] += step_p;
    if (!(PT && a.index)) pq[c] += step_q;
  };
  auto copy_end = [&]() __attribute__((always_inline)) {
    ++cb;
    cs = cs + 1 == S ? 0 : cs + 1;
    if (++ck == cp.nkb) {
      ck = 0;
      cp = place(++co);
      aim();
    }
  };
  auto copy_block = [&]() {
    copy_begin();
#pragma unroll
    for (int c = 0; c < COPIES; ++c) copy_pair(c);
    copy_end();
  };

  uint32_t o[4];  // lane (q, l32): chunk 2 ks + q of row l32 of a 32-row block
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) o[ks] = (uint32_t)(l32 * 128 + (((2 * ks + q) ^ swz(l32)) << 4));
  const uint32_t otr = tr_lane(lane);
  v16f acc[2][2];
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  };
  // lane (q, l32): row l32 of a block, columns 8 g + 4 q .. +3 of a block
  auto finish = [&](const Place& p) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = 32 * wm + 64 * i + l32;
      if (row >= p.rows) continue;
      const int64_t r = (int64_t)p.m0 + row;
#pragma unroll
      for (int j = 0; j < (GLU ? 1 : 2); ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int64_t c = p.n0 + (BN / 2) * j + 32 * wn + 8 * e + 4 * q;
          if (c >= NC) continue;
          float v[4], w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] = acc[i][j][4 * e + k];
          if (MODE == kWgrad) {
            *reinterpret_cast<float4*>(static_cast<float*>(a.out) + ((int64_t)p.g * a.N + r) * NC + c) =
                make_float4(v[0], v[1], v[2], v[3]);
          } else if (MODE == kGlu) {
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = acc[i][1][4 * e + k];
            if (a.keep) {
              *reinterpret_cast<uint2*>(a.keep + r * 2 * NC + c) = pack4(v);
              *reinterpret_cast<uint2*>(a.keep + r * 2 * NC + NC + c) = pack4(w);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = glu(v[k], w[k], a.act);
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + r * NC + c) = pack4(v);
          } else if (MODE == kDgradGlu) {
            float g[4], u[4];
            unpack4(*reinterpret_cast<const uint2*>(a.gu_in + r * 2 * NC + c), g);
            unpack4(*reinterpret_cast<const uint2*>(a.gu_in + r * 2 * NC + NC + c), u);
#pragma unroll
            for (int k = 0; k < 4; ++k) glu_backward(g[k], u[k], v[k], a.act, &v[k], &w[k]);
            uint16_t* out = static_cast<uint16_t*>(a.out) + r * 2 * NC + c;
            *reinterpret_cast<uint2*>(out) = pack4(v);
            *reinterpret_cast<uint2*>(out + NC) = pack4(w);
          } else {
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + r * NC + c) = pack4(v);
          }
        }
    }
  };

  if (PT && a.index) {
#pragma unroll
    for (int i = 0; i < 3; ++i) index_block();
    wait_copies<0>();
  }
  aim();
#pragma unroll
  for (int s = 0; s < S; ++s) {
    copy_block();
    if (PT && a.index) wait_copies<0>();  // (the first blocks' indices are not so far ahead)
  }
  v4i fp[2][2][4], fq[2][2][4];  // operands: [block in turn][32 rows][ks]
  uint32_t st = 0;
  auto read_ks = [&](v4i (&xp)[2][4], v4i (&xq)[2][4], int ks) __attribute__((always_inline)) {
    const uint8_t* tp = smem + st * STAGE;
    const uint8_t* tq = tp + REG;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      xq[i][ks] = QT ? tr_read(tq, otr, wn + 2 * i, ks)
                     : *reinterpret_cast<const v4i*>(tq + o[ks] + (32 * wn + 64 * i) * 128);
      xp[i][ks] = PT ? tr_read(tp, otr, wm + 2 * i, ks)
                     : *reinterpret_cast<const v4i*>(tp + o[ks] + (32 * wm + 64 * i) * 128);
    }
  };
  wait_copies<(S - 1) * 2 * COPIES>();
  barrier();
#pragma unroll
  for (int ks = 0; ks < 4; ++ks) read_ks(fp[0], fq[0], ks);
  st = 1;
  clear();
  int t_o = 0, t_k = 0;
  Place p = place(0);
  auto step = [&](v4i (&xp)[2][4], v4i (&xq)[2][4], v4i (&np)[2][4], v4i (&nq)[2][4]) __attribute__((always_inline)) {
    // the next block's copies have landed (those of two blocks come after
    // them), and everyone has this block in registers
    wait_copies<(S - 2) * 2 * COPIES>();
    barrier();
    const int left = p.kc - 64 * t_k;
    if (left < 64)
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          xq[i][ks] = keep_first(xq[i][ks], left - 16 * ks - 8 * q);
          xp[i][ks] = keep_first(xp[i][ks], left - 16 * ks - 8 * q);
        }
    copy_begin();
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = mfma(xq[j][ks], xp[i][ks], acc[i][j]);
      read_ks(np, nq, ks);
      copy_pair(ks);
      __builtin_amdgcn_sched_barrier(0);
    }
    copy_end();
    st = st + 1 == S ? 0 : st + 1;
    if (++t_k == p.nkb) {
      finish(p);
      clear();
      t_k = 0;
      p = place(++t_o);
    }
  };
  while (t_o < my_n) {
    step(fp[0], fq[0], fp[1], fq[1]);
    if (t_o == my_n) break;
    step(fp[1], fq[1], fp[0], fq[0]);
  }
  wait_copies<0>();  // what was copied past the last tile lands before the LDS is released
}

}  // namespace

void launch_mid(const Args& a, Mode m, hipStream_t st) {
  const dim3 grid(std::max(8, gemm::num_cus() / 8 * 8)), block(MT);
  switch (m) {
    case kPlain: mid_kernel<kPlain><<<grid, block, 0, st>>>(a); break;
    case kGlu: mid_kernel<kGlu><<<grid, block, 0, st>>>(a); break;
    case kDgrad: mid_kernel<kDgrad><<<grid, block, 0, st>>>(a); break;
    case kDgradGlu: mid_kernel<kDgradGlu><<<grid, block, 0, st>>>(a); break;
    case kWgrad: mid_kernel<kWgrad><<<grid, block, 0, st>>>(a); break;
  }
}

}  // namespace bf16
}  // namespace moe
