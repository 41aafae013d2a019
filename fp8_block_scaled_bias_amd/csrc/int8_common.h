// Arguments shared by the kernels of the grouped int8 products.
#pragma once

#include "gemm_common.h"
#include "int8_plan.h"

namespace moe {
namespace int8 {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));

struct Args {
  const int8_t* A;
  const float* sa;
  const int32_t* index;  // source rows of A, or null
  int64_t A_rows;
  const int8_t* B;
  const float* sb;
  const int32_t* offs;
  int G;
  int64_t M_total;
  int64_t N;    // columns of the output; B has N rows a group, or 2N with SwiGLU
  int64_t K;
  uint16_t* C;  // bf16 [M_total, N]
};

// silu(g) * u
__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.0f + expf(-g)) * u; }

// 256 x 256 tiles (int8_wide.hip).  Requires K > 128 and, with an index,
// A_rows * K < 2^32.
void launch_wide(const Args& a, bool swiglu, hipStream_t st);

// 128 x 128 tiles (int8_mid.hip).  Requires, with an index, A_rows * K < 2^32.
void launch_mid(const Args& a, bool swiglu, hipStream_t st);

// The weights straight into registers (int8_stream.hip): any size.
void launch_stream(const Args& a, Plan p, bool swiglu, hipStream_t st);

}  // namespace int8
}  // namespace moe
