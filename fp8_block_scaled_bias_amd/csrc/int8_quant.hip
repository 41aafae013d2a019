// Quantisation to 8-bit integers with one scale a row: a token's activations
// (bf16) or an output channel's weights (fp32).
//
//   s = max |v| * fp32(1 / 127) (1 if that is 0),  code = v / s rounded to the
//   nearest whole number (ties to even), from the exact quotient
//
// HBM bound: 2 B (bf16) or 4 B (fp32) in and 1 B out per element.  Measured:
// 147456 x 2048 bf16 159 us (5.7 TB/s), 135168 x 7168 fp32 897 us (5.4 TB/s),
// 128 x 7168 bf16 3.6 us.
#include "common.h"

namespace moe {
namespace {

constexpr int QT = 256;

// The code of v for scale s, y = 1 / s: an estimate q within one of v / s, its
// remainder v - q s (exact as one FMA: v and q s are multiples of s's last
// place, and |remainder| < s) decides.
__device__ __forceinline__ float settle(float q, float v, float s) {
  const float r = fmaf(-q, s, v), h = 0.5f * s, m = fabsf(r);
  return m > h || (m == h && ((int)q & 1)) ? q + copysignf(1.0f, r) : q;
}

// 8 codes in two words.  The estimate is v y rounded to a whole number by an
// addition of 1.5 * 2^23, which leaves it in the sum's low bits; where no
// remainder reaches half a scale, all eight are right.
__device__ __forceinline__ uint2 codes8(const float* v, float s, float y) {
  const float big = 12582912.0f;
  float t[8], most = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    t[i] = fmaf(v[i], y, big);
    most = fmaxf(most, fabsf(fmaf(big - t[i], s, v[i])));
  }
  if (most >= 0.5f * s) {
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = settle(t[i] - big, v[i], s) + big;
  }
  auto word = [&](const float* f) -> uint32_t {
    // low bytes of four words
    const uint32_t ab = __builtin_amdgcn_perm(__float_as_uint(f[1]), __float_as_uint(f[0]), 0x0C0C0400u);
    const uint32_t cd = __builtin_amdgcn_perm(__float_as_uint(f[3]), __float_as_uint(f[2]), 0x04000C0Cu);
    return ab | cd;
  };
  return make_uint2(word(t), word(t + 4));
}

// scales too small or too large for the above: the quotient in 64 bits,
// which tells every quotient of two fp32 numbers from a tie
__device__ __attribute__((noinline)) uint2 codes8_wide(float v0, float v1, float v2, float v3, float v4,
                                                       float v5, float v6, float v7, float s) {
  const float v[8] = {v0, v1, v2, v3, v4, v5, v6, v7};
  uint32_t w[2] = {0, 0};
  for (int i = 0; i < 8; ++i) {
    const int q = (int)fmin(fmax(rint((double)v[i] / (double)s), -127.0), 127.0);
    w[i >> 2] |= (uint32_t)(q & 0xFF) << (8 * (i & 3));
  }
  return make_uint2(w[0], w[1]);
}

// 8 elements as they lie in memory
struct Bf16x8 {
  uint4 a;
  __device__ __forceinline__ void load(const uint16_t* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float* v) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
};
struct F32x8 {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float* v) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};

__device__ __forceinline__ float scale_of(float amax) {
  const float s = amax * (1.0f / 127.0f);
  return s == 0.f ? 1.0f : s;
}
template <typename X>
__device__ __forceinline__ uint2 quantise(const X& x, float s, float y) {
  float v[8];
  x.get(v);
  if (recip_ok(s)) return codes8(v, s, y);
  return codes8_wide(v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7], s);
}

// A row by WPR waves (1, or the workgroup's 4 or 16), R runs of 8 elements a lane,
// in registers between the maximum and the codes: read from memory once.
template <typename D, typename X, int WPR, int R>
__global__ __launch_bounds__(WPR == 1 ? QT : 64 * WPR) void int8_rows_kernel(
    const D* __restrict__ in, int64_t M, int K, int64_t ld, int8_t* __restrict__ out,
    float* __restrict__ scales) {
  __shared__ float red[2][WPR];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int c0 = 8 * (WPR > 1 ? (int)threadIdx.x : lane);
  int turn = 0;
  const int64_t per = WPR > 1 ? 1 : 4;
  for (int64_t r = (int64_t)blockIdx.x * per + (WPR > 1 ? 0 : wv); r < M; r += (int64_t)gridDim.x * per) {
    X x[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int c = c0 + i * 512 * WPR;
      if (c < K) x[i].load(in + r * ld + c);
      else x[i].zero();
    }
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float v[8];
      x[i].get(v);
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(v[j]));
    }
    amax = wave_max_xor(amax, 64);
    if (WPR > 1) {
      if (lane == 0) red[turn][wv] = amax;
      __syncthreads();
      amax = red[turn][0];
#pragma unroll
      for (int w = 1; w < WPR; ++w) amax = fmaxf(amax, red[turn][w]);
      turn ^= 1;  // (the other half: nobody waits for its readers)
    }
    const float s = scale_of(amax), y = 1.0f / s;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int c = c0 + i * 512 * WPR;
      if (c < K) *reinterpret_cast<uint2*>(out + r * (int64_t)K + c) = quantise(x[i], s, y);
    }
    if ((WPR > 1 ? threadIdx.x : lane) == 0) scales[r] = s;
  }
}

// rows longer than that, read twice
template <typename D, typename X>
__global__ __launch_bounds__(QT) void int8_long_rows_kernel(const D* __restrict__ in, int64_t M, int K,
                                                            int64_t ld, int8_t* __restrict__ out,
                                                            float* __restrict__ scales) {
  __shared__ float red[4];
  for (int64_t r = blockIdx.x; r < M; r += gridDim.x) {
    const D* row = in + r * ld;
    float amax = 0.f;
    for (int c = threadIdx.x * 8; c < K; c += QT * 8) {
      X x;
      x.load(row + c);
      float v[8];
      x.get(v);
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
    }
    amax = wave_max_xor(amax, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = amax;
    __syncthreads();
    const float s = scale_of(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]))), y = 1.0f / s;
    for (int c = threadIdx.x * 8; c < K; c += QT * 8) {
      X x;
      x.load(row + c);
      *reinterpret_cast<uint2*>(out + r * (int64_t)K + c) = quantise(x, s, y);
    }
    if (threadIdx.x == 0) scales[r] = s;
  }
}

template <typename D, typename X>
int rows_launch(const char* who, const D* in, int64_t M, int64_t K64, int64_t ld, int8_t* out,
                float* scales, hipStream_t st) {
  MOE_INVALID(in && out && scales, "%s: null pointer", who);
  MOE_INVALID(((uintptr_t)in & 15) == 0 && ((uintptr_t)out & 7) == 0 && ((uintptr_t)scales & 3) == 0,
              "%s: in must be 16-byte, out 8-byte, scales 4-byte aligned", who);
  const int K = (int)K64;
  const dim3 block(QT);
  const dim3 one((unsigned)std::min<int64_t>(M, 1 << 20)), four((unsigned)std::min<int64_t>(ceil_div(M, 4), 1 << 20));
#define MOE_ROWS(WPR, R, GRID)                                                              \
  int8_rows_kernel<D, X, WPR, R><<<GRID, dim3(WPR == 1 ? QT : 64 * WPR), 0, st>>>(in, M, K, ld, \
                                                                                  out, scales)
  // a wave a row where it holds one and there are rows enough for the CUs'
  // waves, else a workgroup; of 16 waves where there is about a row a CU (128
  // x 7168: 3.6 us, 5.2 with 4 waves; 500 x 4096: 4.6 and 4.2)
  if (K <= 512) MOE_ROWS(1, 1, four);
  else if (K <= 1024 && M >= 2048) MOE_ROWS(1, 2, four);
  else if (K <= 2048 && M >= 2048) MOE_ROWS(1, 4, four);
  else if (K <= 2048) MOE_ROWS(4, 1, one);
  else if (K <= 8192 && M <= (K <= 4096 ? 256 : 512)) MOE_ROWS(16, 1, one);
  else if (K > 8192 && K <= 16384 && M <= 512) MOE_ROWS(16, 2, one);
  else if (K <= 4096) MOE_ROWS(4, 2, one);
  else if (K <= 8192) MOE_ROWS(4, 4, one);
  else if (K <= 16384) MOE_ROWS(4, 8, one);
  else int8_long_rows_kernel<D, X><<<one, block, 0, st>>>(in, M, K, ld, out, scales);
#undef MOE_ROWS
  return check_launch(who);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int int8_quant_rows(const void* in_bf16, int64_t M, int64_t K, int64_t ld_in,
                               int8_t* out_int8, float* scales, void* stream) {
  clear_error();
  MOE_INVALID(M >= 0, "int8_quant_rows: M=%lld < 0", (long long)M);
  MOE_INVALID(K > 0 && K % 8 == 0, "int8_quant_rows: K=%lld must be a positive multiple of 8",
              (long long)K);
  MOE_INVALID(ld_in % 8 == 0 && ld_in >= K, "int8_quant_rows: ld_in=%lld must be a multiple of 8 and >= %lld",
              (long long)ld_in, (long long)K);
  MOE_UNSUPPORTED(K <= (1 << 24) && M < (1ll << 31), "int8_quant_rows: too large");
  if (M == 0) return MOE_OK;
  return rows_launch<uint16_t, Bf16x8>("int8_quant_rows", static_cast<const uint16_t*>(in_bf16), M, K, ld_in, out_int8,
                     scales, as_stream(stream));
}

extern "C" int int8_quant_channels(const float* w_f32, int64_t G, int64_t N, int64_t K,
                                   int8_t* out_int8, float* scales, void* stream) {
  clear_error();
  MOE_INVALID(G >= 0 && N > 0, "int8_quant_channels: G=%lld must be >= 0 and N=%lld > 0", (long long)G,
              (long long)N);
  MOE_INVALID(K > 0 && K % 8 == 0, "int8_quant_channels: K=%lld must be a positive multiple of 8",
              (long long)K);
  MOE_UNSUPPORTED(K <= (1 << 24) && G < (1ll << 31) && N < (1ll << 31) && G * N < (1ll << 31),
                  "int8_quant_channels: too large");
  if (G == 0) return MOE_OK;
  return rows_launch<float, F32x8>("int8_quant_channels", w_f32, G * N, K, K, out_int8, scales, as_stream(stream));
}
