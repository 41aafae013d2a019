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
  const Plan p = plan(Shape{swiglu, a_row_index != nullptr, A_rows, G, M_total, N, K}, gemm::num_cus());
  if (p == kWide) launch_wide(a, swiglu, st);
  else if (p == kMid) launch_mid(a, swiglu, st);
  else launch_stream(a, p, swiglu, st);
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
