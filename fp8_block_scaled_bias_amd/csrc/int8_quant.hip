// Quantisation to 8-bit integers with one scale a row: a token's activations
// (bf16) or an output channel's weights (fp32).
//
//   s = max |v| * fp32(1 / 127) (1 if that is 0),  code = v / s rounded to the
//   nearest whole number (ties to even), from the exact quotient
//
// HBM bound: 2 B (bf16) or 4 B (fp32) in and 1 B out per element.
#include "common.h"

namespace moe {
namespace {

constexpr int QT = 256;

// The code of v for scale s, y = 1 / s: the rounded estimate v * y lies
// within one of v / s, its remainder v - q s is exact as one FMA (v and q s
// are multiples of s's last place, and |remainder| < s), and decides.
__device__ __forceinline__ int int8_code(float v, float s, float y) {
  float q = rintf(v * y);
  const float r = fmaf(-q, s, v), h = 0.5f * s, m = fabsf(r);
  if (m > h || (m == h && ((int)q & 1))) q += copysignf(1.0f, r);
  return (int)q;
}

// scales too small or too large for the above: the quotient in 64 bits,
// which tells every quotient of two fp32 numbers from a tie
__device__ __forceinline__ int int8_code_wide(float v, float s) {
  return (int)fmin(fmax(rint((double)v / (double)s), -127.0), 127.0);
}

__device__ __forceinline__ void load8(const uint16_t* p, float* v) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_to_f32(w[i] & 0xFFFFu);
    v[2 * i + 1] = bf16_to_f32(w[i] >> 16);
  }
}
__device__ __forceinline__ void load8(const float* p, float* v) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

template <typename D>
__global__ __launch_bounds__(QT) void int8_rows_kernel(const D* __restrict__ in, int64_t M, int64_t K,
                                                       int64_t ld, int8_t* __restrict__ out,
                                                       float* __restrict__ scales) {
  __shared__ float red[QT / 64];
  for (int64_t r = blockIdx.x; r < M; r += gridDim.x) {
    const D* row = in + r * ld;
    float amax = 0.f;
    for (int64_t c = threadIdx.x * 8; c < K; c += QT * 8) {
      float v[8];
      load8(row + c, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(v[i]));
    }
    amax = wave_max_xor(amax, 64);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = amax;
    __syncthreads();
    amax = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    float s = amax * (1.0f / 127.0f);
    s = s == 0.f ? 1.0f : s;
    const float y = 1.0f / s;
    const bool near_one = recip_ok(s);
    for (int64_t c = threadIdx.x * 8; c < K; c += QT * 8) {
      float v[8];
      load8(row + c, v);
      uint32_t w[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int q = near_one ? int8_code(v[i], s, y) : int8_code_wide(v[i], s);
        w[i >> 2] |= (uint32_t)(q & 0xFF) << (8 * (i & 3));
      }
      *reinterpret_cast<uint2*>(out + r * K + c) = make_uint2(w[0], w[1]);
    }
    if (threadIdx.x == 0) scales[r] = s;
  }
}

template <typename D>
int rows_launch(const char* who, const D* in, int64_t M, int64_t K, int64_t ld, int8_t* out,
                float* scales, hipStream_t st) {
  MOE_INVALID(in && out && scales, "%s: null pointer", who);
  MOE_INVALID(((uintptr_t)in & 15) == 0 && ((uintptr_t)out & 7) == 0 && ((uintptr_t)scales & 3) == 0,
              "%s: in must be 16-byte, out 8-byte, scales 4-byte aligned", who);
  const int64_t blocks = std::min<int64_t>(M, 1 << 20);
  int8_rows_kernel<D><<<dim3((unsigned)blocks), dim3(QT), 0, st>>>(in, M, K, ld, out, scales);
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
  return rows_launch("int8_quant_rows", static_cast<const uint16_t*>(in_bf16), M, K, ld_in, out_int8,
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
  return rows_launch("int8_quant_channels", w_f32, G * N, K, K, out_int8, scales, as_stream(stream));
}
