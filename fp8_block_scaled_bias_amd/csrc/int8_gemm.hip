// Grouped product of 8-bit integers with a scale for each token and one for
// each output channel (the experts' products of a quantised layer; one group
// is a plain linear layer), plain or with SwiGLU over gate and up columns.
//
//   C[r, n] = bf16( (sa[r] * sb[g, n]) * sum_k a[r, k] b[g, n, k] )
//
// The sum is exact in 32 bits (K < 2^17 codes of at most 2^7 in size), so the
// order of the products does not matter; it is rounded to fp32 once.
#include "int8_common.h"

namespace moe {
namespace int8 {
namespace {

constexpr int T8 = 256;     // threads: four waves
constexpr int BM8 = 64;     // rows of a tile, 16 to a wave
constexpr int BN8 = 64;     // output columns of a tile
constexpr int KB8 = 64;     // bytes of K a step
constexpr int P8 = KB8 + 16;

// The group and first row of the m-th row tile; false past the last.
__device__ __forceinline__ bool find_tile(const Args& a, int64_t m, int* g, int* r0, int* r1) {
  const int lane = threadIdx.x & 63;
  int64_t before = 0;
  for (int g0 = 0; g0 < a.G; g0 += 64) {
    const int gi = g0 + lane;
    const int lo = gi < a.G ? a.offs[gi] : 0, hi = gi < a.G ? a.offs[gi + 1] : 0;
    const int tiles = hi > lo ? (hi - lo + BM8 - 1) / BM8 : 0;
    int v = tiles;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const int n = __shfl_up(v, o, 64);
      if (lane >= o) v += n;
    }
    const int64_t end = before + v;
    const uint64_t here = __ballot(m < end);
    if (here) {
      const int l = __ffsll((unsigned long long)here) - 1;
      const int first = __shfl(v - tiles, l, 64);
      *g = g0 + l;
      *r0 = __shfl(lo, l, 64) + (int)(m - before - first) * BM8;
      *r1 = __shfl(hi, l, 64);
      return true;
    }
    before = __shfl(end, 63, 64);
  }
  return false;
}

template <bool SWIGLU>
__global__ __launch_bounds__(T8) void int8_tile_kernel(Args a) {
  constexpr int NB = SWIGLU ? 2 : 1;
  __shared__ __attribute__((aligned(16))) int8_t sA[BM8][P8];
  __shared__ __attribute__((aligned(16))) int8_t sB[NB * BN8][P8];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int64_t n0 = (int64_t)blockIdx.x * BN8;
  int g, r0, r1;
  for (int64_t m = blockIdx.y; find_tile(a, m, &g, &r0, &r1); m += gridDim.y) {
  // copies: thread -> row tid / 4, 16 bytes (tid % 4)
  const int cr = tid >> 2, cc = (tid & 3) * 16;
  int64_t arow = min(r0 + cr, r1 - 1);
  if (a.index) arow = min((uint32_t)a.index[arow], (uint32_t)(a.A_rows - 1));
  const int8_t* pa = a.A + arow * a.K;
  const int64_t bn = min<int64_t>(n0 + cr, a.N - 1);
  const int8_t* pb = a.B + ((int64_t)g * NB * a.N + bn) * a.K;
  v4i acc[NB][4];
#pragma unroll
  for (int h = 0; h < NB; ++h)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[h][j] = v4i{0, 0, 0, 0};
  for (int64_t k0 = 0; k0 < a.K; k0 += KB8) {
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const bool in = k0 + cc < a.K;
    const uint4 va = in ? *reinterpret_cast<const uint4*>(pa + k0 + cc) : zero;
    uint4 vb[NB];
#pragma unroll
    for (int h = 0; h < NB; ++h)
      vb[h] = in ? *reinterpret_cast<const uint4*>(pb + h * a.N * a.K + k0 + cc) : zero;
    __syncthreads();
    *reinterpret_cast<uint4*>(&sA[cr][cc]) = va;
#pragma unroll
    for (int h = 0; h < NB; ++h) *reinterpret_cast<uint4*>(&sB[h * BN8 + cr][cc]) = vb[h];
    __syncthreads();
    const v4i fa = *reinterpret_cast<const v4i*>(&sA[16 * wv + (lane & 15)][16 * (lane >> 4)]);
#pragma unroll
    for (int h = 0; h < NB; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const v4i fb = *reinterpret_cast<const v4i*>(&sB[h * BN8 + 16 * j + (lane & 15)][16 * (lane >> 4)]);
        acc[h][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fa, fb, acc[h][j], 0, 0, 0);
      }
  }
  const float* sb = a.sb + (int64_t)g * NB * a.N;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int row = r0 + 16 * wv + 4 * (lane >> 4) + r;
    if (row >= r1) continue;
    const int64_t src = a.index ? min((uint32_t)a.index[row], (uint32_t)(a.A_rows - 1)) : row;
    const float s = a.sa[src];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t n = n0 + 16 * j + (lane & 15);
      if (n >= a.N) continue;
      float v = (float)acc[0][j][r] * (s * sb[n]);
      if (SWIGLU) v = silu_mul(v, (float)acc[NB - 1][j][r] * (s * sb[a.N + n]));
      a.C[(int64_t)row * a.N + n] = (uint16_t)f32_to_bf16_rne(v);
    }
  }
  }
}

int int8_gemm(const char* who, bool swiglu, const int8_t* A, const float* A_scale,
              const int32_t* a_row_index, int64_t A_rows, const int8_t* B, const float* B_scale,
              const int32_t* group_offsets, int32_t G, int64_t M_total, int64_t N, int64_t K, void* C,
              hipStream_t st) {
  MOE_INVALID(G >= 1, "%s: G=%d must be >= 1", who, (int)G);
  MOE_UNSUPPORTED(G <= 1024, "%s: G=%d > 1024 groups is not supported", who, (int)G);
  MOE_INVALID(M_total >= 0 && M_total < (1ll << 31), "%s: M_total=%lld out of range", who,
              (long long)M_total);
  MOE_INVALID(N > 0 && N % 8 == 0, "%s: %s=%lld must be a positive multiple of 8", who,
              swiglu ? "I" : "N", (long long)N);
  MOE_INVALID(K > 0 && K % 16 == 0, "%s: K=%lld must be a positive multiple of 16", who, (long long)K);
  MOE_UNSUPPORTED(K < 131072 && N <= (1 << 21), "%s: K=%lld >= 131072 or %s=%lld > 2097152 is not supported",
                  who, (long long)K, swiglu ? "I" : "N", (long long)N);
  if (M_total == 0) return MOE_OK;
  MOE_INVALID(A_rows >= (a_row_index ? 1 : M_total) && A_rows < (1ll << 31),
              "%s: A_rows=%lld must be in [%s, 2^31)", who, (long long)A_rows,
              a_row_index ? "1" : "M_total");
  MOE_INVALID(A && A_scale && B && B_scale && group_offsets && C, "%s: null pointer", who);
  MOE_INVALID(((uintptr_t)A & 15) == 0 && ((uintptr_t)B & 15) == 0 && ((uintptr_t)C & 15) == 0 &&
                  ((uintptr_t)A_scale & 3) == 0 && ((uintptr_t)B_scale & 3) == 0 &&
                  ((uintptr_t)a_row_index & 3) == 0 && ((uintptr_t)group_offsets & 3) == 0,
              "%s: A, B and the output must be 16-byte aligned, scales and indices 4-byte", who);
  const Args a{A, A_scale, a_row_index, A_rows, B, B_scale, group_offsets, G, M_total, N, K,
                   static_cast<uint16_t*>(C)};
  const int64_t mtiles = std::min<int64_t>({M_total, G + M_total / BM8, 65535});
  const dim3 grid((unsigned)ceil_div(N, BN8), (unsigned)mtiles);
  if (M_total / G >= 32 && K > 128 && (!a_row_index || A_rows * K < 0xFFF00000ll)) launch_wide(a, swiglu, st);
  else if (swiglu) int8_tile_kernel<true><<<grid, dim3(T8), 0, st>>>(a);
  else int8_tile_kernel<false><<<grid, dim3(T8), 0, st>>>(a);
  return check_launch(who);
}

}  // namespace
}  // namespace int8
}  // namespace moe

using namespace moe;
using namespace moe::int8;

extern "C" int grouped_int8_gemm(const int8_t* A, const float* A_scale, const int32_t* a_row_index,
                                 int64_t A_rows, const int8_t* B, const float* B_scale,
                                 const int32_t* group_offsets, int32_t G, int64_t M_total, int64_t N,
                                 int64_t K, void* C_bf16, void* stream) {
  clear_error();
  return int8_gemm("grouped_int8_gemm", false, A, A_scale, a_row_index, A_rows, B, B_scale,
                   group_offsets, G, M_total, N, K, C_bf16, as_stream(stream));
}

extern "C" int grouped_int8_gemm_swiglu(const int8_t* A, const float* A_scale,
                                        const int32_t* a_row_index, int64_t A_rows, const int8_t* B,
                                        const float* B_scale, const int32_t* group_offsets, int32_t G,
                                        int64_t M_total, int64_t I, int64_t K, void* H_bf16,
                                        void* stream) {
  clear_error();
  return int8_gemm("grouped_int8_gemm_swiglu", true, A, A_scale, a_row_index, A_rows, B, B_scale,
                   group_offsets, G, M_total, I, K, H_bf16, as_stream(stream));
}
