// Arguments and pieces shared by the kernels of the grouped bf16 products.
#pragma once

#include "bf16_plan.h"
#include "gemm_common.h"

namespace moe {
namespace bf16 {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));

// A product D[m, n] = sum_k P[m, k] Q[n, k] of each group.
//   kPlain, kGlu         P: the group's rows of A (gathered by index),
//                        Q: its weights B [N, K] (kGlu: gate, then up rows)
//   kDgrad, kDgradGlu    P: the group's rows of dC [rows, N], Q: W [N, K]
//                        transposed - the contraction runs over its rows
//   kWgrad               P: dY's columns, Q: A's (rows gathered by index): the
//                        contraction runs over the group's rows
struct Args {
  const uint16_t* P;
  const uint16_t* Q;
  const int32_t* index;  // source rows of A, or null
  int64_t A_rows;
  const int32_t* offs;
  int G;
  int64_t M_total;
  int64_t N, K;          // of the weights; kGlu: N = I; kDgradGlu: K = I
  int act;
  const uint16_t* gu_in; // kDgradGlu: the forward's gate and up outputs
  void* out;
  uint16_t* keep;        // kGlu: gate and up outputs, or null
};

__device__ __forceinline__ v16f mfma(const v4i& x, const v4i& y, const v16f& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, x), __builtin_bit_cast(v8bf, y),
                                                 c, 0, 0, 0);
}

// The gate's activation, g times the logistic function of z: z = g (SiLU), or
// twice the argument of the tanh form of GELU, 2 sqrt(2/pi) (g + 0.044715 g^3).
// There g is held to +-16, past which the logistic function is 0 or 1 in
// fp32, so that the slope stays finite for every finite g.  The exponential and
// the reciprocal are the hardware's (an ulp each: what the rounding of z itself
// does to the exponential is more): their exact forms made the epilogue of a 256
// x 256 tile of gate and up 128 x 30 instructions long instead of 128 x 8.
constexpr float kGeluR = 1.5957691216057308f, kGeluC = 0.044715f;
__device__ __forceinline__ float logistic(float g, int act, float* dz) {
  float z = g;
  *dz = 1.0f;
  if (act == MOE_ACT_GELU) {
    const float c = __builtin_amdgcn_fmed3f(g, -16.0f, 16.0f), c2 = c * c;
    z = kGeluR * c * fmaf(kGeluC, c2, 1.0f);
    *dz = kGeluR * fmaf(3.0f * kGeluC, c2, 1.0f);
  }
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * z));
}
__device__ __forceinline__ float glu(float g, float u, int act) {
  float dz;
  return g * logistic(g, act, &dz) * u;
}
// dg and du of h = act(g) u for the gradient d of h
__device__ __forceinline__ void glu_backward(float g, float u, float d, int act, float* dg, float* du) {
  float dz;
  const float s = logistic(g, act, &dz);
  *dg = d * u * fmaf(g * s * (1.0f - s), dz, s);
  *du = d * (g * s);
}

__device__ __forceinline__ uint2 pack4(const float* v) {
  return make_uint2(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]));
}
__device__ __forceinline__ void unpack4(const uint2& w, float* v) {
  v[0] = bf16_to_f32(w.x & 0xFFFFu);
  v[1] = bf16_to_f32(w.x >> 16);
  v[2] = bf16_to_f32(w.y & 0xFFFFu);
  v[3] = bf16_to_f32(w.y >> 16);
}

// 8 consecutive contraction values of an operand, of which the first n count:
// the others' bits are cleared (what lies there may be anything).
__device__ __forceinline__ v4i keep_first(v4i f, int n) {
#pragma unroll
  for (int d = 0; d < 4; ++d)
    f[d] &= n >= 2 * d + 2 ? -1 : n == 2 * d + 1 ? 0xFFFF : 0;
  return f;
}

// An operand tile whose contraction runs down its rows lies in LDS as 64 rows of
// 128 columns, 256 B each; 16-byte chunk c of row r in slot c ^ 4 (r % 4).
// Lane (q, l32) gets the 8 contraction values 16 ks + 8 q .. of column l32 of a
// 32-column block by two transposing reads, each of 4 rows by 16 columns for
// 16 lanes (lane i of them addresses row i / 4, columns 4 (i % 4) ..): the
// four rows of a read lie in four different quarters of the banks.
__device__ __forceinline__ uint32_t tr_lane(int lane) {  // of block 0, ks 0
  const int i = lane & 15, row = 8 * (lane >> 5) + (i >> 2);
  const int chunk = 2 * ((lane >> 4) & 1) + ((i & 3) >> 1);
  return (uint32_t)(row * 256 + ((chunk ^ (4 * (row & 3))) << 4) + 8 * (i & 1));
}
typedef short v4s __attribute__((ext_vector_type(4)));
// block: which 32 columns of the tile (its bits move the quarter of the row)
__device__ __forceinline__ v4i tr_read(const uint8_t* tile, uint32_t lane_off, int block, int ks) {
  typedef __attribute__((address_space(3))) v4s lds_v4s;
  const __attribute__((address_space(3))) uint8_t* p =
      (const __attribute__((address_space(3))) uint8_t*)tile + (lane_off ^ (uint32_t)(block << 6)) + ks * 16 * 256;
  const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)p);
  const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s*)(p + 4 * 256));
  typedef int v2i __attribute__((ext_vector_type(2)));
  const v2i a = __builtin_bit_cast(v2i, lo), b = __builtin_bit_cast(v2i, hi);
  return v4i{a[0], a[1], b[0], b[1]};
}

void launch_zero(float* p, int64_t n, hipStream_t st);  // n a multiple of 4

// 256 x 256 tiles (bf16_wide.hip).  Requires, with an index, A_rows * K < 2^31.
void launch_wide(const Args& a, Mode m, hipStream_t st);

// The weights straight into registers (bf16_stream.hip): kPlain and kGlu, any size.
void launch_stream(const Args& a, Mode m, Plan p, hipStream_t st);

// 128 x 128 tiles (bf16_mid.hip): any size.
void launch_mid(const Args& a, Mode m, hipStream_t st);

}  // namespace bf16
}  // namespace moe
