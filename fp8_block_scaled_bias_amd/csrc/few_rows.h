// Grouped products for groups of few rows: the weights are read once, straight
// into registers, as bytes; E is the elements' type, with the matrix
// instruction, what a sum is scaled by, and the output.
//
// Bound by the weights' stream (a row tile does 2 * rows operations a weight
// and far fewer than the matrix cores need for one), so nothing passes through
// LDS: a lane loads 16 bytes of a weight row and of a token row where a 16 x 16
// matrix instruction of 64 bytes wants them (lane l: row l % 16, bytes
// 16 (l / 16) .. +15; both operands permute K alike), D blocks of 128 bytes
// ahead.
//  * flow_kernel, where there are tiles enough for every wave: each wave works
//    on tiles of its own, 16 MB rows x 64 weight rows over the whole of K, and
//    its loads run on from tile to tile.
//  * split_kernel, where there are not: a workgroup of four waves takes 16 MB
//    rows x 16 NJ weight rows, its waves every fourth K block; their sums meet
//    in LDS.  The K loop's end reads nothing past it: with the last block read
//    again for every block ahead that is not there, one row of N = 16384, K =
//    4096 bytes took 21 us instead of 12.
#pragma once

#include "gemm_common.h"

namespace moe {
namespace few_rows {

using gemm::build_group_tables;
using gemm::decode_tile;
using gemm::MAXG;
typedef int v4i __attribute__((ext_vector_type(4)));

constexpr int ST = 256;

template <class E, int NJ, int MB, int D, bool GLU>
__global__ __launch_bounds__(ST) void split_kernel(typename E::Args a) {
  constexpr bool HALF = GLU && NJ == 1;  // 8 gate and 8 up columns in one block
  constexpr int NO = GLU && !HALF ? NJ / 2 : NJ;  // 16-column blocks of the output
  constexpr int TN = HALF ? 8 : 16 * NO;
  constexpr int W = ST / 64, PITCH = 16 * NJ + 4;
  __shared__ int s_offs[MAXG + 1];
  __shared__ int s_pref[MAXG + 1];
  __shared__ int s_red[W];
  __shared__ int s_carry;
  __shared__ __attribute__((aligned(16))) typename E::Sum red[W][16][PITCH];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, q = lane >> 4;
  const int64_t N = a.N, K = E::row_bytes(a);
  const int nkb = (int)((K + 127) >> 7);
  const int64_t ntiles = (N + TN - 1) / TN;
  const int64_t b_rows = GLU ? 2 * N : N;
  // one group whose rows fit a tile: the loads need not wait for its offsets
  const bool lone = a.G == 1 && a.M_total <= 16 * MB;
  if (!lone) build_group_tables<ST, 16 * MB>(a.offs, a.G, s_offs, s_pref, s_red, &s_carry);
  const int64_t total = lone ? ntiles : (int64_t)s_pref[a.G] * ntiles;
  // an XCD's workgroups (blockIdx % 8) take a contiguous range of tiles, the
  // row tiles of one weight panel next to each other
  const int nper = gridDim.x >> 3;
  const int64_t chunk = (total + 7) >> 3;
  const int64_t lo = (blockIdx.x & 7) * chunk, hi = min(total, lo + chunk);
  for (int64_t L = lo + (blockIdx.x >> 3); L < hi; L += nper) {
    gemm::Tile t{};
    if (lone) {
      t.nt = L;
      t.m1 = (int)a.M_total;
    } else {
      t = decode_tile(s_pref, s_offs, a.G, ntiles, L, 16 * MB);
    }
    const int g = __builtin_amdgcn_readfirstlane(t.g);
    const int m0 = __builtin_amdgcn_readfirstlane(t.m0), m1 = __builtin_amdgcn_readfirstlane(t.m1);
    const int64_t n0 = (int64_t)__builtin_amdgcn_readfirstlane((int)t.nt) * TN;
    const uint8_t* pb = E::B(a) + ((int64_t)g * b_rows + n0) * K;
    uint32_t vb[NO];  // lane offsets of the weight rows (past N: the last)
#pragma unroll
    for (int j = 0; j < NO; ++j)
      vb[j] = (uint32_t)(min<int64_t>(HALF ? r16 & 7 : 16 * j + r16, N - 1 - n0) * K);
    if (HALF && r16 >= 8) pb += N * K;
    const uint8_t* pa[MB];
    int64_t src[MB];
#pragma unroll
    for (int i = 0; i < MB; ++i) {
      const int row = min(m0 + 16 * i + r16, m1 - 1);
      src[i] = a.index ? (int64_t)min((uint32_t)a.index[row], (uint32_t)(a.A_rows - 1)) : row;
      pa[i] = E::A(a) + src[i] * K;
    }
    const int mb = min(MB, (m1 - m0 + 15) >> 4);  // row blocks with rows

    v4i fa[D][MB][2], fb[D][NJ][2];
    typename E::Acc acc[MB][NJ];
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = typename E::Acc{0, 0, 0, 0};
    auto load = [&](v4i (&xa)[MB][2], v4i (&xb)[NJ][2], int kb) __attribute__((always_inline)) {
      // (bytes past the row's end: read within it, cleared below)
      const uint32_t k0 = (uint32_t)kb * 128 + 16 * q;
      uint32_t o[2];
      o[0] = min(k0, (uint32_t)K - 16);
      o[1] = min(k0 + 64, (uint32_t)K - 16);
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          xb[j][h] = *reinterpret_cast<const v4i*>(pb + (j >= NO ? N * K : 0) + (vb[j % NO] + o[h]));
#pragma unroll
      for (int i = 0; i < MB; ++i)
        if (i == 0 || i < mb)
#pragma unroll
          for (int h = 0; h < 2; ++h) xa[i][h] = *reinterpret_cast<const v4i*>(pa[i] + o[h]);
    };
    auto multiply = [&](v4i (&xa)[MB][2], v4i (&xb)[NJ][2], int kb) __attribute__((always_inline)) {
      if ((int64_t)kb * 128 + 128 > K) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (kb * 128 + 64 * h + 16 * q >= (int)K) {
#pragma unroll
            for (int i = 0; i < MB; ++i) xa[i][h] = v4i{0, 0, 0, 0};
            if (E::kClearB)
#pragma unroll
              for (int j = 0; j < NJ; ++j) xb[j][h] = v4i{0, 0, 0, 0};
          }
      }
#pragma unroll
      for (int i = 0; i < MB; ++i)
        if (i == 0 || i < mb)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < NJ; ++j)
              acc[i][j] = E::mfma(xa[i][h], xb[j][h], acc[i][j]);
    };
#pragma unroll
    for (int d = 0; d < D - 1; ++d)
      if (wv + W * d < nkb) load(fa[d], fb[d], wv + W * d);
    int kb = wv;
    for (; kb + 2 * W * (D - 1) < nkb; kb += W * D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        load(fa[(d + D - 1) % D], fb[(d + D - 1) % D], kb + W * (d + D - 1));
        multiply(fa[d], fb[d], kb + W * d);
      }
    }
    for (; kb < nkb; kb += W * D) {  // the last blocks: nothing is read twice
#pragma unroll
      for (int d = 0; d < D; ++d) {
        const int cur = kb + W * d, next = cur + W * (D - 1);
        if (next < nkb) load(fa[(d + D - 1) % D], fb[(d + D - 1) % D], next);
        if (cur < nkb) multiply(fa[d], fb[d], cur);
      }
    }
    // lane: rows 4 q + r of a row block, column r16 of a column block
    for (int i = 0; i < mb; ++i) {
      __syncthreads();
#pragma unroll
      for (int ii = 0; ii < MB; ++ii)
        if (ii == i)
#pragma unroll
          for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r) red[wv][4 * q + r][16 * j + r16] = acc[ii][j][r];
      __syncthreads();
      const int lr = tid >> 4, row = m0 + 16 * i + lr, c0 = (tid & 15) * NO;
      if (row >= (lone ? a.offs[1] : m1) || n0 + c0 >= N || (HALF && c0 >= 8)) continue;
      const int64_t sr = a.index ? (int64_t)min((uint32_t)a.index[row], (uint32_t)(a.A_rows - 1)) : row;
      const typename E::Row rs = E::row(a, sr);
      float v[NO];
#pragma unroll
      for (int c = 0; c < NO; ++c) {
        auto sum = [&](int col) { return (red[0][lr][col] + red[1][lr][col]) + (red[2][lr][col] + red[3][lr][col]); };
        const int64_t at = n0 + c0 + c;
        v[c] = E::value(sum(c0 + c), rs, E::col(a, (int64_t)g * b_rows + at));
        if (GLU)
          v[c] = E::glu(a, row, at, v[c], E::value(sum(TN + c0 + c), rs, E::col(a, (int64_t)g * b_rows + N + at)));
      }
      uint16_t* out = E::out(a) + (int64_t)row * N + n0 + c0;
      if (NO == 4)
        *reinterpret_cast<uint2*>(out) = make_uint2(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2 % NO], v[3 % NO]));
      else if (NO == 2)
        *reinterpret_cast<uint32_t*>(out) = f32x2_to_bf16x2(v[0], v[1 % NO]);
      else
        *out = (uint16_t)f32_to_bf16_rne(v[0]);
    }
    __syncthreads();
  }
}

template <class E, int MB, int D, bool GLU>
__global__ __launch_bounds__(ST) void flow_kernel(typename E::Args a) {
  constexpr int NJ = 4, NO = GLU ? 2 : 4;
  static_assert(!E::kClearB, "what is past a row's end is cleared in one operand only");
  __shared__ int s_offs[MAXG + 1];
  __shared__ int s_pref[MAXG + 1];
  __shared__ int s_red[4];
  __shared__ int s_carry;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, q = lane >> 4;
  const int64_t N = a.N, K = E::row_bytes(a);
  const int nkb = (int)((K + 127) >> 7);
  const int64_t ntiles = (N + 16 * NO - 1) / (16 * NO);
  const int64_t b_rows = GLU ? 2 * N : N;
  build_group_tables<ST, 16 * MB>(a.offs, a.G, s_offs, s_pref, s_red, &s_carry);
  const int64_t total = (int64_t)s_pref[a.G] * ntiles;
  // an XCD's waves take a contiguous range of tiles (the row tiles of one
  // weight panel next to each other), every nper-th each
  const int64_t nper = (int64_t)(gridDim.x >> 3) * 4;
  const int64_t lo = total * (blockIdx.x & 7) / 8, hi = total * ((blockIdx.x & 7) + 1) / 8;
  const int64_t L0 = lo + (int64_t)(blockIdx.x >> 3) * 4 + wv;
  if (L0 >= hi) return;
  const int my_n = (int)((hi - L0 + nper - 1) / nper);

  struct Place {
    int g, m0, m1, mb;
    int64_t n0;
  };
  auto place = [&](int o) {
    const gemm::Tile t = decode_tile(s_pref, s_offs, a.G, ntiles, L0 + (int64_t)min(o, my_n - 1) * nper, 16 * MB);
    Place p;
    p.g = __builtin_amdgcn_readfirstlane(t.g);
    p.m0 = __builtin_amdgcn_readfirstlane(t.m0);
    p.m1 = __builtin_amdgcn_readfirstlane(t.m1);
    p.n0 = (int64_t)__builtin_amdgcn_readfirstlane((int)t.nt) * (16 * NO);
    p.mb = min(MB, (p.m1 - p.m0 + 15) >> 4);  // row blocks with rows
    return p;
  };
  auto source = [&](int row) -> int64_t {
    return a.index ? (int64_t)min((uint32_t)a.index[row], (uint32_t)(a.A_rows - 1)) : row;
  };

  // ---- loads: K block lk of tile lo_
  int l_o = 0, l_k = 0, l_mb = 0;
  const uint8_t* pb = nullptr;
  uint32_t vb[NO];
  const uint8_t* pa[MB];
  auto aim = [&]() {
    const Place p = place(l_o);
    pb = E::B(a) + ((int64_t)p.g * b_rows + p.n0) * K;
    l_mb = p.mb;
#pragma unroll
    for (int j = 0; j < NO; ++j)  // (weight rows past N: the last)
      vb[j] = (uint32_t)(min<int64_t>(16 * j + r16, N - 1 - p.n0) * K);
#pragma unroll
    for (int i = 0; i < MB; ++i) pa[i] = E::A(a) + source(min(p.m0 + 16 * i + r16, p.m1 - 1)) * K;
  };
  v4i fa[D][MB][2], fb[D][NJ][2];
  typename E::Acc acc[MB][NJ];
  auto load = [&](v4i (&xa)[MB][2], v4i (&xb)[NJ][2]) __attribute__((always_inline)) {
    // (bytes past a row's end: read within it, cleared below)
    const uint32_t k0 = (uint32_t)(l_k * 128 + 16 * q);
    const uint32_t end = (uint32_t)K - 16u;
    const uint32_t o[2] = {std::min(k0, end), std::min(k0 + 64u, end)};
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        xb[j][h] = *reinterpret_cast<const v4i*>(pb + (j >= NO ? N * K : 0) + (vb[j % NO] + o[h]));
#pragma unroll
    for (int i = 0; i < MB; ++i)
      if (i == 0 || i < l_mb)
#pragma unroll
        for (int h = 0; h < 2; ++h) xa[i][h] = *reinterpret_cast<const v4i*>(pa[i] + o[h]);
    if (++l_k == nkb) {
      l_k = 0;
      if (++l_o < my_n) aim();
    }
  };
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < MB; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[i][j] = typename E::Acc{0, 0, 0, 0};
  };
  // lane: rows 4 q + r of a row block, column r16 of a column block
  auto finish = [&](const Place& p) __attribute__((always_inline)) {
    typename E::Col w[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int64_t c = p.n0 + min<int64_t>(16 * (j % NO) + r16, N - 1 - p.n0);
      w[j] = E::col(a, (int64_t)p.g * b_rows + (j >= NO ? N : 0) + c);
    }
#pragma unroll
    for (int i = 0; i < MB; ++i)
      if (i == 0 || i < p.mb)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = p.m0 + 16 * i + 4 * q + r;
          if (row >= p.m1) continue;
          const typename E::Row rs = E::row(a, source(row));
          uint16_t* out = E::out(a) + (int64_t)row * N + p.n0 + r16;
#pragma unroll
          for (int j = 0; j < NO; ++j) {
            if (p.n0 + 16 * j + r16 >= N) continue;
            float v = E::value(acc[i][j][r], rs, w[j]);
            if (GLU)
              v = E::glu(a, row, p.n0 + 16 * j + r16, v, E::value(acc[i][NO % NJ + j][r], rs, w[NO % NJ + j]));
            out[16 * j] = (uint16_t)f32_to_bf16_rne(v);
          }
        }
  };

  aim();
#pragma unroll
  for (int d = 0; d < D - 1; ++d)
    if (l_o < my_n) load(fa[d], fb[d]);
  clear();
  int c_o = 0, c_k = 0;
  Place p = place(0);
  while (c_o < my_n) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (l_o < my_n) load(fa[(d + D - 1) % D], fb[(d + D - 1) % D]);
      if (c_o < my_n) {
        v4i(&xa)[MB][2] = fa[d];
        v4i(&xb)[NJ][2] = fb[d];
        if ((int64_t)c_k * 128 + 128 > K) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (c_k * 128 + 64 * h + 16 * q >= (int)K) {
#pragma unroll
              for (int i = 0; i < MB; ++i) xa[i][h] = v4i{0, 0, 0, 0};
            }
        }
#pragma unroll
        for (int i = 0; i < MB; ++i)
          if (i == 0 || i < p.mb)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int j = 0; j < NJ; ++j)
                acc[i][j] = E::mfma(xa[i][h], xb[j][h], acc[i][j]);
        if (++c_k == nkb) {
          finish(p);
          clear();
          c_k = 0;
          if (++c_o < my_n) p = place(c_o);
        }
      }
    }
  }
}

template <class E, int MB, int D, bool GLU>
void launch_flow(const typename E::Args& a, hipStream_t st) {
  const unsigned grid = (unsigned)(2 * gemm::num_cus() / 8 * 8);
  flow_kernel<E, MB, D, GLU><<<dim3(std::max(8u, grid)), dim3(ST), 0, st>>>(a);
}

template <class E, int NJ, int MB, int D, bool GLU>
void launch_split(const typename E::Args& a, int64_t tiles, hipStream_t st) {
  const int64_t most = 4 * (int64_t)gemm::num_cus() / 8 * 8;
  const unsigned grid = (unsigned)std::min<int64_t>(most, ceil_div(tiles, 8) * 8);
  split_kernel<E, NJ, MB, D, GLU><<<dim3(grid), dim3(ST), 0, st>>>(a);
}

}  // namespace few_rows
}  // namespace moe
