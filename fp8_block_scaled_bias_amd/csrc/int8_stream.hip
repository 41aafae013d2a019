// Grouped int8 product for groups of few rows, or too few tiles for the wide
// kernel (few_rows.h: the weights read once, straight into registers), with
// v_mfma_i32_16x16x64_i8.  The waves' sums are whole numbers: their order does
// not matter.
//
// flow_kernel: 256 groups of 4 rows, N = 7168, K = 2048 (3.76 GB of weights):
// 635 us, 5.9 TB/s.  split_kernel: one row, N = 4096, K = 7168 (29 MB): 7.6 us,
// most of it the launch and the first loads' latency; 64 rows 19.4 us.
#include "int8_common.h"
#include "few_rows.h"

namespace moe {
namespace int8 {
namespace {

using few_rows::launch_flow;
using few_rows::launch_split;

struct Int8 {
  using Args = int8::Args;
  using Sum = int;
  using Acc = v4i;
  struct Row {
    float s;
  };
  struct Col {
    float s;
  };
  static constexpr bool kClearB = false;  // (whole numbers: one zero operand is enough)
  static __device__ __forceinline__ int64_t row_bytes(const Args& a) { return a.K; }
  static __device__ __forceinline__ const uint8_t* A(const Args& a) { return reinterpret_cast<const uint8_t*>(a.A); }
  static __device__ __forceinline__ const uint8_t* B(const Args& a) { return reinterpret_cast<const uint8_t*>(a.B); }
  static __device__ __forceinline__ uint16_t* out(const Args& a) { return a.C; }
  static __device__ __forceinline__ Acc mfma(const v4i& x, const v4i& y, const Acc& c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8(x, y, c, 0, 0, 0);
  }
  static __device__ __forceinline__ Row row(const Args& a, int64_t src) { return {a.sa[src]}; }
  static __device__ __forceinline__ Col col(const Args& a, int64_t b_row) { return {a.sb[b_row]}; }
  static __device__ __forceinline__ float value(int s, Row r, Col c) { return (float)s * (r.s * c.s); }
  static __device__ __forceinline__ float glu(const Args&, int64_t, int64_t, float g, float u) { return silu_mul(g, u); }
};

template <bool SWIGLU>
void dispatch(const Args& a, Plan p, hipStream_t st) {
  const Shape s{SWIGLU, a.index != nullptr, a.A_rows, a.G, a.M_total, a.N, a.K};
  constexpr int N1 = SWIGLU ? 2 : 1;
  switch (p) {
    case kFlow: return launch_flow<Int8, 1, 3, SWIGLU>(a, st);
    case kSplit16x64: return launch_split<Int8, 4, 1, 3, SWIGLU>(a, m16(s) * n64(s), st);
    case kSplit16x16: return launch_split<Int8, N1, 1, 3, SWIGLU>(a, m16(s) * n16(s), st);
    case kSplit64x64: return launch_split<Int8, 4, 4, 2, SWIGLU>(a, m64(s) * n64(s), st);
    case kSplit64x32: return launch_split<Int8, 2, 4, 3, SWIGLU>(a, m64(s) * n32(s), st);
    default: return launch_split<Int8, N1, 4, 3, SWIGLU>(a, m64(s) * n16(s), st);
  }
}

}  // namespace

void launch_stream(const Args& a, Plan p, bool swiglu, hipStream_t st) {
  if (swiglu) dispatch<true>(a, p, st);
  else dispatch<false>(a, p, st);
}

}  // namespace int8
}  // namespace moe
