// Grouped bf16 product for groups of few rows, or too few tiles for the other
// kernels (few_rows.h: the weights read once, straight into registers), with
// v_mfma_f32_16x16x32_bf16; plain or with the gated activation.
#include "bf16_common.h"
#include "few_rows.h"

namespace moe {
namespace bf16 {
namespace {

using few_rows::launch_split;

struct Bf16 {
  using Args = bf16::Args;
  using Sum = float;
  typedef float Acc __attribute__((ext_vector_type(4)));
  struct Row {};
  struct Col {};
  static constexpr bool kClearB = true;  // (zero times an infinity is none)
  static __device__ __forceinline__ int64_t row_bytes(const Args& a) { return 2 * a.K; }
  static __device__ __forceinline__ const uint8_t* A(const Args& a) { return reinterpret_cast<const uint8_t*>(a.P); }
  static __device__ __forceinline__ const uint8_t* B(const Args& a) { return reinterpret_cast<const uint8_t*>(a.Q); }
  static __device__ __forceinline__ uint16_t* out(const Args& a) { return static_cast<uint16_t*>(a.out); }
  static __device__ __forceinline__ Acc mfma(const v4i& x, const v4i& y, const Acc& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, x), __builtin_bit_cast(v8bf, y), c, 0, 0,
                                                   0);
  }
  static __device__ __forceinline__ Row row(const Args&, int64_t) { return {}; }
  static __device__ __forceinline__ Col col(const Args&, int64_t) { return {}; }
  static __device__ __forceinline__ float value(float s, Row, Col) { return s; }
  static __device__ __forceinline__ float glu(const Args& a, int64_t row, int64_t c, float g, float u) {
    if (a.keep) {
      a.keep[row * 2 * a.N + c] = (uint16_t)f32_to_bf16_rne(g);
      a.keep[row * 2 * a.N + a.N + c] = (uint16_t)f32_to_bf16_rne(u);
    }
    return bf16::glu(g, u, a.act);
  }
};

template <bool GLU>
void dispatch(const Args& a, Plan p, hipStream_t st) {
  const Shape s{GLU ? kGlu : kPlain, a.index != nullptr, a.A_rows, a.G, a.M_total, a.N, a.K};
  switch (p) {
    case kSplit16x64: return launch_split<Bf16, 4, 1, 3, GLU>(a, m16(s) * n64(s), st);
    case kSplit16x16: return launch_split<Bf16, 1, 1, 3, GLU>(a, m16(s) * n16(s), st);
    case kSplit64x64: return launch_split<Bf16, 4, 4, 2, GLU>(a, m64(s) * n64(s), st);
    case kSplit64x32: return launch_split<Bf16, 2, 4, 3, GLU>(a, m64(s) * n32(s), st);
    default: return launch_split<Bf16, 1, 4, 3, GLU>(a, m64(s) * n16(s), st);
  }
}

}  // namespace

void launch_stream(const Args& a, Mode m, Plan p, hipStream_t st) {
  if (m == kGlu) dispatch<true>(a, p, st);
  else dispatch<false>(a, p, st);
}

}  // namespace bf16
}  // namespace moe
