// Grouped bf16 products: the experts' projections, their input gradients and
// weight gradients, with the gated activation or its backward in the epilogue
// (one group is a dense layer).  Sums are taken in fp32 by the matrix cores;
// a result is rounded once, when it is stored.
#include "bf16_common.h"

namespace moe {
namespace bf16 {
namespace {

bool aligned16(const void* p) { return ((uintptr_t)p & 15) == 0; }

// Checks shared by every mode, then the launch.  n_name, k_name: what the
// header calls the two sizes.
int run(const char* who, Mode m, const Args& a, const char* n_name, const char* k_name, hipStream_t st) {
  MOE_INVALID(a.G >= 1, "%s: G=%d must be >= 1", who, a.G);
  MOE_UNSUPPORTED(a.G <= gemm::MAXG, "%s: G=%d > %d groups is not supported", who, a.G, gemm::MAXG);
  MOE_INVALID(a.M_total >= 0 && a.M_total < (1ll << 31), "%s: M_total=%lld out of range", who,
              (long long)a.M_total);
  MOE_UNSUPPORTED(a.M_total <= gemm::kMaxRows, "%s: M_total=%lld > 2^31 - 256 is not supported", who,
                  (long long)a.M_total);
  MOE_INVALID(a.N > 0 && a.N % 8 == 0, "%s: %s=%lld must be a positive multiple of 8", who, n_name,
              (long long)a.N);
  MOE_INVALID(a.K > 0 && a.K % 8 == 0, "%s: %s=%lld must be a positive multiple of 8", who, k_name,
              (long long)a.K);
  MOE_UNSUPPORTED(a.N <= (1 << 21) && a.K <= (1 << 21), "%s: %s=%lld or %s=%lld > 2097152 is not supported",
                  who, n_name, (long long)a.N, k_name, (long long)a.K);
  const bool glu = m == kGlu || m == kDgradGlu;
  MOE_INVALID(!glu || a.act == MOE_ACT_SILU || a.act == MOE_ACT_GELU,
              "%s: act=%d must be MOE_ACT_SILU or MOE_ACT_GELU", who, a.act);
  if (a.M_total == 0 && m != kWgrad) return MOE_OK;
  MOE_INVALID(a.out && aligned16(a.out) && aligned16(a.keep), "%s: outputs must be non-null and 16-byte aligned",
              who);
  if (a.M_total == 0) {  // every group is empty: the gradient is zero
    launch_zero(static_cast<float*>(a.out), (int64_t)a.G * a.N * a.K, st);
    return check_launch(who);
  }
  MOE_INVALID(a.A_rows >= (a.index ? 1 : a.M_total) && a.A_rows < (1ll << 31),
              "%s: A_rows=%lld must be in [%s, 2^31)", who, (long long)a.A_rows, a.index ? "1" : "M_total");
  MOE_INVALID(a.P && a.Q && a.offs && (m != kDgradGlu || a.gu_in), "%s: null pointer", who);
  MOE_INVALID(aligned16(a.P) && aligned16(a.Q) && aligned16(a.gu_in) && ((uintptr_t)a.index & 3) == 0 &&
                  ((uintptr_t)a.offs & 3) == 0,
              "%s: operands must be 16-byte aligned, indices 4-byte", who);
  MOE_INVALID(a.out != a.P && a.out != a.Q && a.out != a.gu_in && (!a.keep || a.keep != a.out),
              "%s: outputs must not alias inputs or each other", who);
  const Plan p = plan(Shape{m, a.index != nullptr, a.A_rows, a.G, a.M_total, a.N, a.K}, gemm::num_cus());
  if (p == kWide) launch_wide(a, m, st);
  else if (p == kMid) launch_mid(a, m, st);
  else launch_stream(a, m, p, st);
  return check_launch(who);
}

__global__ __launch_bounds__(256) void zero_kernel(float4* p, int64_t n) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
    p[i] = make_float4(0.f, 0.f, 0.f, 0.f);
}

}  // namespace

void launch_zero(float* p, int64_t n, hipStream_t st) {
  const int64_t blocks = std::min<int64_t>(ceil_div(n / 4, 256), 4096);
  zero_kernel<<<dim3((unsigned)blocks), dim3(256), 0, st>>>(reinterpret_cast<float4*>(p), n / 4);
}

}  // namespace bf16
}  // namespace moe

using namespace moe;
using namespace moe::bf16;

static const uint16_t* u16(const void* p) { return static_cast<const uint16_t*>(p); }

extern "C" int grouped_bf16_gemm(const void* A_bf16, const int32_t* a_row_index, int64_t A_rows,
                                 const void* B_bf16, const int32_t* group_offsets, int32_t G,
                                 int64_t M_total, int64_t N, int64_t K, void* C_bf16, void* stream) {
  clear_error();
  const Args a{u16(A_bf16), u16(B_bf16), a_row_index, A_rows, group_offsets, G, M_total, N, K, 0, nullptr,
               C_bf16, nullptr};
  return run("grouped_bf16_gemm", kPlain, a, "N", "K", as_stream(stream));
}

extern "C" int grouped_bf16_gemm_glu(const void* A_bf16, const int32_t* a_row_index, int64_t A_rows,
                                     const void* B_bf16, const int32_t* group_offsets, int32_t G,
                                     int64_t M_total, int64_t I, int64_t K, int32_t act, void* H_bf16,
                                     void* GU_bf16, void* stream) {
  clear_error();
  const Args a{u16(A_bf16), u16(B_bf16), a_row_index, A_rows, group_offsets, G, M_total, I, K, act, nullptr,
               H_bf16, static_cast<uint16_t*>(GU_bf16)};
  return run("grouped_bf16_gemm_glu", kGlu, a, "I", "K", as_stream(stream));
}

extern "C" int grouped_bf16_gemm_dgrad(const void* dC_bf16, const void* W_bf16, const int32_t* group_offsets,
                                       int32_t G, int64_t M_total, int64_t N, int64_t K, void* dA_bf16,
                                       void* stream) {
  clear_error();
  const Args a{u16(dC_bf16), u16(W_bf16), nullptr, M_total, group_offsets, G, M_total, N, K, 0, nullptr,
               dA_bf16, nullptr};
  return run("grouped_bf16_gemm_dgrad", kDgrad, a, "N", "K", as_stream(stream));
}

extern "C" int grouped_bf16_gemm_dgrad_glu(const void* dC_bf16, const void* W_bf16, const void* GU_bf16,
                                           const int32_t* group_offsets, int32_t G, int64_t M_total,
                                           int64_t N, int64_t I, int32_t act, void* dGU_bf16, void* stream) {
  clear_error();
  const Args a{u16(dC_bf16), u16(W_bf16), nullptr, M_total, group_offsets, G, M_total, N, I, act, u16(GU_bf16),
               dGU_bf16, nullptr};
  return run("grouped_bf16_gemm_dgrad_glu", kDgradGlu, a, "N", "I", as_stream(stream));
}

extern "C" int grouped_bf16_wgrad(const void* dY_bf16, const void* A_bf16, const int32_t* a_row_index,
                                  int64_t A_rows, const int32_t* group_offsets, int32_t G, int64_t M_total,
                                  int64_t N, int64_t K, float* dW, void* stream) {
  clear_error();
  const Args a{u16(dY_bf16), u16(A_bf16), a_row_index, A_rows, group_offsets, G, M_total, N, K, 0, nullptr,
               dW, nullptr};
  return run("grouped_bf16_wgrad", kWgrad, a, "N", "K", as_stream(stream));
}
