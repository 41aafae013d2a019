// The norms before and after a block: RMS norm of the residual stream with the
// residual add before it and the experts' operand codes after it, and the
// combine's gate-weighted sum with its norm and the scaled residual sum after
// it; and both backward.
//
// HBM bound: a workgroup holds a whole row (or a token's k + 1 rows) in
// registers, 8 columns a thread and chunk, between the row's sums and what
// they scale, so that nothing is read twice (but by the combine's gradient of
// more than 8192 columns, whose rows do not fit: they are read twice).  Sums are
// formed in fp32, over a thread's columns, the wave (DPP) and the waves (LDS) in a
// fixed order.  The backward passes run a fixed number of workgroups over the
// tokens, each with its part of the weight's gradient in registers; a second
// launch adds up the parts, in a fixed order.
//
// 16384 x 7168 (HBM reads 6.05, copies 4.7 TB/s): norm of fp32 with the add and
// E4M3 codes 266 us (5.8 TB/s), its gradient in bf16 183 us (5.1); combine of 8
// rows and the shared one with norm 475 us (5.4), its gradient with codes 1290
// us (4.3).  128 rows: 4.9 us, a launch and one row's chain of steps; the weight
// loaded ahead of the sums gains nothing there and costs 4 % at 16384.
#include "gemm_common.h"

namespace moe {
namespace {

constexpr int MAXW = 16;  // waves of a workgroup

__device__ __forceinline__ void unpack8(const uint4& v, float* f) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_to_f32(w[i] & 0xFFFFu);
    f[2 * i + 1] = bf16_to_f32(w[i] >> 16);
  }
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(f32x2_to_bf16x2(f[0], f[1]), f32x2_to_bf16x2(f[2], f[3]), f32x2_to_bf16x2(f[4], f[5]),
                    f32x2_to_bf16x2(f[6], f[7]));
}

// 8 columns of a tensor of the residual stream's type, as loaded
template <int TYPE>
struct Raw {
  uint4 w[TYPE == MOE_TYPE_F32 ? 2 : 1];
};
template <int TYPE>
__device__ __forceinline__ Raw<TYPE> load8(const void* p, int64_t i) {
  Raw<TYPE> r;
  const uint4* q = TYPE == MOE_TYPE_F32 ? reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i)
                                        : reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
  r.w[0] = q[0];
  if constexpr (TYPE == MOE_TYPE_F32) r.w[1] = q[1];
  return r;
}
template <int TYPE>
__device__ __forceinline__ void values8(const Raw<TYPE>& r, float* f) {
  if constexpr (TYPE == MOE_TYPE_F32) {
    const uint32_t w[8] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w, r.w[1].x, r.w[1].y, r.w[1].z, r.w[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
  } else {
    unpack8(r.w[0], f);
  }
}
// Stores 8 columns; f becomes the values as stored.
template <int TYPE>
__device__ __forceinline__ void store8(void* p, int64_t i, float* f) {
  if constexpr (TYPE == MOE_TYPE_F32) {
    float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    q[0] = make_float4(f[0], f[1], f[2], f[3]);
    q[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    const uint4 w = pack8(f);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = w;
    unpack8(w, f);
  }
}
__device__ __forceinline__ void load_f32x8(const float* p, float* f) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

__device__ __forceinline__ float wave_sum(float v) {
  v += row_other<1>(v);
  v += row_other<2>(v);
  v += row_other<4>(v);
  v += row_other<8>(v);
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

// Sums over the workgroup of N values a thread, for every thread.  `s` is used
// by one call in two, so that one barrier a call is enough.
template <int N>
struct Sums {
  float s[2][MAXW][N];
};
template <int N>
__device__ __forceinline__ void block_sums(float* v, Sums<N>& sh, int slot, int waves) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) sh.s[slot][wv][i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float t = 0.0f;
    for (int w = 0; w < waves; ++w) t += sh.s[slot][w][i];
    v[i] = t;
  }
}

__device__ __forceinline__ float rstd_of(float squares, int64_t H, float eps) {
  return 1.0f / sqrtf(squares / (float)H + eps);
}

// ---- the norm before the block -----------------------------------------------
struct NormArgs {
  const void* x;
  const uint16_t* add;
  const float* weight;
  int64_t T, H;
  float eps;
  void* sum;
  uint16_t* n;
  float* rstd;
  uint8_t* codes;
  float* scales;
};

// (of rows_grid; past the last row there is none)
__device__ __forceinline__ int64_t row_index() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

template <int NC, int TYPE, int QUANT>
__global__ __launch_bounds__(1024) void norm_kernel(NormArgs a) {
  __shared__ Sums<1> s_sum, s_max;
  const int tid = threadIdx.x, waves = blockDim.x >> 6;
  const int64_t t = row_index(), H = a.H, row = t * H;
  if (t >= a.T) return;
  float v[NC][8];
  float acc[1] = {0.0f};
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int64_t col = ((int64_t)c * blockDim.x + tid) * 8;
    if (col < H) {
      const Raw<TYPE> r = load8<TYPE>(a.x, row + col);
      values8<TYPE>(r, v[c]);
      if (a.add) {
        float d[8];
        unpack8(*reinterpret_cast<const uint4*>(a.add + row + col), d);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] += d[i];
        store8<TYPE>(a.sum, row + col, v[c]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[0] = fmaf(v[c][i], v[c][i], acc[0]);
  }
  block_sums<1>(acc, s_sum, 0, waves);
  const float r = rstd_of(acc[0], H, a.eps);
  if (tid == 0 && a.rstd) a.rstd[t] = r;
  float top = 0.0f;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int64_t col = ((int64_t)c * blockDim.x + tid) * 8;
    if (col < H) {
      float w[8];
      if (a.weight) load_f32x8(a.weight + col, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[c][i] *= r;
        if (a.weight) v[c][i] *= w[i];
        top = fmaxf(top, fabsf(v[c][i]));
      }
      *reinterpret_cast<uint4*>(a.n + row + col) = pack8(v[c]);
      if (QUANT == MOE_QUANT_E4M3) {  // (H is whole tiles: 16 lanes hold one)
        float s;
        *reinterpret_cast<uint2*>(a.codes + row + col) = quant_tile_1x128(v[c], &s);
        if ((tid & 15) == 0) a.scales[(row + col) >> 7] = s;
      }
    }
  }
  if (QUANT == MOE_QUANT_INT8) {
    top = wave_max_xor(top, 64);
    if ((tid & 63) == 0) s_max.s[0][tid >> 6][0] = top;
    __syncthreads();
    for (int w = 0; w < waves; ++w) top = fmaxf(top, s_max.s[0][w][0]);
    float s = top * (1.0f / 127.0f);
    s = s > 0.0f ? s : 1.0f;
    if (tid == 0) a.scales[t] = s;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int64_t col = ((int64_t)c * blockDim.x + tid) * 8;
      if (col >= H) continue;
      uint32_t b[2] = {0u, 0u};
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int code = (int)rintf(__builtin_amdgcn_fmed3f(v[c][i] / s, -127.0f, 127.0f));
        b[i >> 2] |= (uint32_t)(code & 0xFF) << (8 * (i & 3));
      }
      *reinterpret_cast<uint2*>(a.codes + row + col) = make_uint2(b[0], b[1]);
    }
  }
}

// ---- its backward --------------------------------------------------------------
struct NormBwdArgs {
  const uint16_t* dn;
  const void* x;
  const float* weight;
  const float* rstd;
  const void* res;
  float res_scale;
  int64_t T, H;
  void* dx;
  float* part;  // [workgroups, H], or null
};

template <int NC, int TYPE>
__global__ __launch_bounds__(1024) void norm_backward_kernel(NormBwdArgs a) {
  __shared__ Sums<1> s_sum;
  const int tid = threadIdx.x, waves = blockDim.x >> 6;
  const int64_t H = a.H;
  float w[NC][8], dw[NC][8];
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int64_t col = ((int64_t)c * blockDim.x + tid) * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[c][i] = 0.0f, w[c][i] = 1.0f;
    if (a.weight && col < H) load_f32x8(a.weight + col, w[c]);
  }
  uint4 dn[NC];
  Raw<TYPE> x[NC], res[NC];
  float r = 0.0f;
  auto load = [&](int64_t t) {
    r = a.rstd[t];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int64_t col = ((int64_t)c * blockDim.x + tid) * 8;
      if (col >= H) continue;
      dn[c] = *reinterpret_cast<const uint4*>(a.dn + t * H + col);
      x[c] = load8<TYPE>(a.x, t * H + col);
      if (a.res) res[c] = load8<TYPE>(a.res, t * H + col);
    }
  };
  int slot = 0;
  if (blockIdx.x < a.T) load(blockIdx.x);
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    float hat[NC][8], g[NC][8], old[NC][8];
    float sum[1] = {0.0f};
    const float rt = r;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      if (((int64_t)c * blockDim.x + tid) * 8 >= H) continue;
      unpack8(dn[c], g[c]);
      values8<TYPE>(x[c], hat[c]);
      if (a.res) values8<TYPE>(res[c], old[c]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        hat[c][i] *= rt;
        dw[c][i] = fmaf(g[c][i], hat[c][i], dw[c][i]);
        g[c][i] *= w[c][i];
        sum[0] = fmaf(g[c][i], hat[c][i], sum[0]);
      }
    }
    if (t + gridDim.x < a.T) load(t + gridDim.x);
    block_sums<1>(sum, s_sum, slot, waves);
    slot ^= 1;
    const float mean = sum[0] / (float)H;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      const int64_t col = ((int64_t)c * blockDim.x + tid) * 8;
      if (col >= H) continue;
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        o[i] = rt * fmaf(-mean, hat[c][i], g[c][i]);
        if (a.res) o[i] = fmaf(a.res_scale, old[c][i], o[i]);
      }
      store8<TYPE>(a.dx, t * H + col, o);
    }
  }
  if (!a.part) return;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int64_t col = ((int64_t)c * blockDim.x + tid) * 8;
    if (col >= H) continue;
    float* p = a.part + (int64_t)blockIdx.x * H + col;
    *reinterpret_cast<float4*>(p) = make_float4(dw[c][0], dw[c][1], dw[c][2], dw[c][3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(dw[c][4], dw[c][5], dw[c][6], dw[c][7]);
  }
}

// out[h] = sum over the parts, in a fixed order: RG groups of threads take every
// RG-th part of 64 columns, their sums meet in LDS.  (P = 0: zero.)
constexpr int RG = 64, RD = 16 * RG;
__global__ __launch_bounds__(RD) void add_parts_kernel(const float* part, int P, int64_t H, float* out) {
  __shared__ float4 s[RG][16];
  const int g = threadIdx.x >> 4, l = threadIdx.x & 15;
  const int64_t col = (int64_t)blockIdx.x * 64 + 4 * l;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  if (col < H)
#pragma unroll 8
    for (int p = g; p < P; p += RG) {
      const float4 w = *reinterpret_cast<const float4*>(part + (int64_t)p * H + col);
      v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
    }
  s[g][l] = v;
  __syncthreads();
  if (g || col >= H) return;
  for (int i = 1; i < RG; ++i) {
    const float4 w = s[i][l];
    v.x += w.x, v.y += w.y, v.z += w.z, v.w += w.w;
  }
  *reinterpret_cast<float4*>(out + col) = v;
}

// ---- the combine with the norm after the block ---------------------------------
constexpr int KR = 9;  // rows of a token: up to 8 experts and the shared one

struct CombineArgs {
  const uint16_t* D;
  const int32_t* inv_perm;
  const float* topk_w;
  const uint16_t* S;      // shared rows, or null
  const float* shared_w;  // [T], or null: 1
  const void* residual;
  float residual_scale, scale;
  int norm;
  const float* weight;
  float eps;
  int64_t T, H;
  int k;
  void* y;
  float* rstd;
  // backward
  const void* dy;
  uint16_t* dD;
  float* d_topk_w;
  float* d_shared_w;
  uint8_t* codes;
  float* scales;
  float* part;
};

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ uint4 stream16(const uint16_t* p) {
  const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// (read only here, and the same for every lane: through the scalar cache)
template <class V>
__device__ __forceinline__ V scalar(const V* p, int64_t i) {
  return ((const __attribute__((address_space(4))) V*)p)[i];
}
// Rows and weights of a token (uniform): its experts' in the slots below k, the
// shared row's in the last.  An entry of the permutation outside [0, T k) is
// kept as it is: it reads the last routed row, and its gradient is not written.
struct Token {
  uint32_t row[KR];
  float w[KR];
};
__device__ __forceinline__ bool has(const CombineArgs& a, int j) { return j < KR - 1 ? j < a.k : a.S != nullptr; }
__device__ __forceinline__ Token token_of(const CombineArgs& a, int64_t t) {
  Token o;
  // (slots past k repeat the last one: all loads at once, none behind a branch)
#pragma unroll
  for (int j = 0; j < KR - 1; ++j) {
    o.row[j] = (uint32_t)scalar(a.inv_perm, t * a.k + min(j, a.k - 1));
    o.w[j] = scalar(a.topk_w, t * a.k + min(j, a.k - 1));
  }
  o.row[KR - 1] = (uint32_t)t;
  const float w = scalar(a.shared_w ? a.shared_w + t : a.topk_w, 0);
  o.w[KR - 1] = a.shared_w ? w : 1.0f;
  return o;
}
__device__ __forceinline__ const uint16_t* row_of(const CombineArgs& a, const Token& tk, int j) {
  if (j == KR - 1) return a.S + (int64_t)tk.row[j] * a.H;
  return a.D + (int64_t)min(tk.row[j], (uint32_t)(a.T * a.k - 1)) * a.H;
}

// z: the rows' sum in slot order
__device__ __forceinline__ void gather8(const CombineArgs& a, const Token& tk, const uint4* rows, float* z) {
#pragma unroll
  for (int i = 0; i < 8; ++i) z[i] = 0.0f;
#pragma unroll
  for (int j = 0; j < KR; ++j)
    if (has(a, j)) {
      float d[8];
      unpack8(rows[j], d);
#pragma unroll
      for (int i = 0; i < 8; ++i) z[i] = fmaf(tk.w[j], d[i], z[i]);
    }
}

template <int NC, int TYPE>
__global__ __launch_bounds__(1024) void combine_norm_kernel(CombineArgs a) {
  __shared__ Sums<1> s_sum;
  const int tid = threadIdx.x, waves = blockDim.x >> 6;
  const int64_t t = row_index(), H = a.H;
  if (t >= a.T) return;
  const Token tk = token_of(a, t);
  float z[NC][8];
  Raw<TYPE> res[NC];
  float acc[1] = {0.0f};
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int64_t col = ((int64_t)c * blockDim.x + tid) * 8;
    if (col < H) {
      uint4 rows[KR];
#pragma unroll
      for (int j = 0; j < KR; ++j)
        if (has(a, j)) rows[j] = stream16(row_of(a, tk, j) + col);
      res[c] = load8<TYPE>(a.residual, t * H + col);
      gather8(a, tk, rows, z[c]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) z[c][i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[0] = fmaf(z[c][i], z[c][i], acc[0]);
  }
  float r = 1.0f;
  if (a.norm) {
    block_sums<1>(acc, s_sum, 0, waves);
    r = rstd_of(acc[0], H, a.eps);
    if (tid == 0 && a.rstd) a.rstd[t] = r;
  }
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    const int64_t col = ((int64_t)c * blockDim.x + tid) * 8;
    if (col >= H) continue;
    float o[8], w[8];
    values8<TYPE>(res[c], o);
    if (a.weight) load_f32x8(a.weight + col, w);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float b = z[c][i] * r;
      if (a.weight) b *= w[i];
      o[i] = fmaf(a.scale, b, a.residual_scale * o[i]);
    }
    store8<TYPE>(a.y, t * H + col, o);
  }
}

// A token's rows are held in registers between the sums and the gradients
// (HOLD); as soon as a row's gradient is formed, the next token's row is loaded
// in its place.  Without HOLD (H > 8192) they are read twice.  One barrier a
// token: the dots' parts are added up behind the next one.
template <int NC, int TYPE, bool HOLD>
__global__ __launch_bounds__(1024) void combine_norm_backward_kernel(CombineArgs a) {
  __shared__ Sums<2> s_sum;
  __shared__ float s_dot[2][MAXW][KR];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, waves = blockDim.x >> 6;
  const int64_t H = a.H, TK = a.T * a.k;
  float dw[NC][8];
#pragma unroll
  for (int c = 0; c < NC; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[c][i] = 0.0f;
  const uint32_t H32 = (uint32_t)H;
  auto col_of = [&](int c) -> uint32_t { return ((uint32_t)c * blockDim.x + (uint32_t)tid) * 8; };
  auto at_row = [&](const void* p, int64_t t) -> const void* {  // (uniform)
    return static_cast<const uint8_t*>(p) + t * H * (TYPE == MOE_TYPE_F32 ? 4 : 2);
  };
  uint4 rows[KR];
  Raw<TYPE> dy;
  auto load = [&](const Token& tk, int64_t t, uint32_t col) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < KR; ++j)
      if (has(a, j)) rows[j] = stream16(row_of(a, tk, j) + col);
    dy = load8<TYPE>(at_row(a.dy, t), col);
  };
  // (through an empty asm, so that the rows stay packed and are not kept as the
  // 72 values that the passes before unpacked)
  auto keep_packed = [&]() __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < KR; ++j)
      if (has(a, j)) asm volatile("" : "+v"(rows[j].x), "+v"(rows[j].y), "+v"(rows[j].z), "+v"(rows[j].w));
  };
  auto weights = [&](uint32_t col, float* w) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.0f;
    if (a.weight) load_f32x8(a.weight + col, w);
  };
  // d_topk_w and d_shared_w of a token whose waves' dots lie in `slot`
  auto dots = [&](int64_t t, int slot) __attribute__((always_inline)) {
    if (tid < a.k || (tid == KR - 1 && a.d_shared_w)) {
      float v = 0.0f;
      for (int i = 0; i < waves; ++i) v += s_dot[slot][i][tid];
      if (tid < a.k) a.d_topk_w[t * a.k + tid] = v;
      else a.d_shared_w[t] = v;
    }
  };
  const int64_t stride = gridDim.x;
  int slot = 0;
  Token next = token_of(a, blockIdx.x);
  if (HOLD && col_of(0) < H32) load(next, blockIdx.x, col_of(0));
  for (int64_t t = blockIdx.x; t < a.T; t += stride, slot ^= 1) {
    const Token tk = next;
    const bool more = t + stride < a.T;
    if (more) next = token_of(a, t + stride);
    float sum[2] = {0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      uint32_t col = col_of(c);
      asm volatile("" : "+v"(col));  // (so that no address is kept over the loop)
      if (col >= H32) continue;
      if (!HOLD) load(tk, t, col);
      float z[8], g[8], w[8];
      gather8(a, tk, rows, z);
      values8<TYPE>(dy, g);
      weights(col, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sum[0] = fmaf(z[i], z[i], sum[0]);
        sum[1] = fmaf(a.scale * g[i] * w[i], z[i], sum[1]);
      }
    }
    if (HOLD) keep_packed();
    block_sums<2>(sum, s_sum, slot, waves);
    if (t > blockIdx.x) dots(t - stride, slot ^ 1);
    const float r = a.norm ? rstd_of(sum[0], H, a.eps) : 1.0f;
    const float mean = a.norm ? r * sum[1] / (float)H : 0.0f;  // of the normed row and its gradient
    float dot[KR];
#pragma unroll
    for (int j = 0; j < KR; ++j) dot[j] = 0.0f;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
      uint32_t col = col_of(c);
      asm volatile("" : "+v"(col));  // (so that no address is kept over the loop)
      if (col >= H32) continue;
      if (!HOLD) load(tk, t, col);
      float dz[8];
      {
        float z[8], g[8], w[8];
        gather8(a, tk, rows, z);
        values8<TYPE>(dy, g);
        weights(col, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float hat = z[i] * r;
          g[i] *= a.scale;
          dw[c][i] = fmaf(g[i], hat, dw[c][i]);
          dz[i] = r * fmaf(-mean, hat, g[i] * w[i]);
        }
      }
      if (HOLD && more) dy = load8<TYPE>(at_row(a.dy, t + stride), col);
      keep_packed();
#pragma unroll
      for (int j = 0; j < KR; ++j)
        if (has(a, j)) {
          float d[8], o[8];
          unpack8(rows[j], d);
          if (HOLD && more) rows[j] = stream16(row_of(a, next, j) + col);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            dot[j] = fmaf(dz[i], d[i], dot[j]);
            o[i] = tk.w[j] * dz[i];
          }
          if (j < KR - 1 && tk.row[j] >= TK) continue;
          const int64_t to = (j < KR - 1 ? (int64_t)tk.row[j] : TK + t) * H;
          *reinterpret_cast<uint4*>(a.dD + to + col) = pack8(o);
          if (a.codes) {
            float s;
            *reinterpret_cast<uint2*>(a.codes + to + col) = quant_tile_1x128(o, &s);
            if ((tid & 15) == 0) a.scales[(to >> 7) + (col >> 7)] = s;
          }
        }
    }
#pragma unroll
    for (int j = 0; j < KR; ++j) dot[j] = wave_sum(dot[j]);
    if (lane == 0)
#pragma unroll
      for (int j = 0; j < KR; ++j) s_dot[slot][wv][j] = dot[j];
  }
  __syncthreads();
  dots(blockIdx.x + (a.T - 1 - blockIdx.x) / stride * stride, slot ^ 1);
  if (!a.part) return;
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    if (col_of(c) >= H32) continue;
    float* p = a.part + (int64_t)blockIdx.x * H + col_of(c);
    *reinterpret_cast<float4*>(p) = make_float4(dw[c][0], dw[c][1], dw[c][2], dw[c][3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(dw[c][4], dw[c][5], dw[c][6], dw[c][7]);
  }
}

constexpr int64_t kMaxH = 16384;
// A workgroup a row: a dimension of a grid holds less than 2^32 threads, 2^21 rows of
// up to 1024 are one of 2^31, and further rows go along y.
inline dim3 rows_grid(int64_t T) {
  const int64_t x = std::min<int64_t>(T, (int64_t)1 << 21);
  return dim3((unsigned)x, (unsigned)ceil_div(T, x));
}
inline unsigned threads_of(int64_t H, int nc) { return (unsigned)(ceil_div(ceil_div(H, 8 * nc), 64) * 64); }
// Workgroups of a backward pass, each with its part of d_weight: two a CU of 256
// where a row takes 16 waves, more of shorter rows.
inline int64_t parts_of(int64_t T, int64_t H) {
  const int64_t waves = ceil_div(ceil_div(H, 8 * (H <= 8192 ? 1 : 2)), 64);
  return std::min<int64_t>(T, 512 * std::max<int64_t>(1, std::min<int64_t>(4, 16 / waves)));
}
// A single workgroup (one row) writes d_weight itself, and the parts' launch is
// saved (H = 7168: norm 8.5 -> 5.5 us, combine 15.3 -> 11.6).  Not so two rows in
// one workgroup: a combine's take 20.6 us one after the other, 15.4 side by side.
inline float* part_of(float* d_weight, int64_t parts, void* workspace) {
  return d_weight && parts > 1 ? static_cast<float*>(workspace) : d_weight;
}

bool aligned(const void* p, int n) { return ((uintptr_t)p & (uintptr_t)(n - 1)) == 0; }

int check_rows(const char* who, int64_t T, int64_t H, int32_t type) {
  MOE_INVALID(T >= 0 && T < (1ll << 28), "%s: T=%lld out of [0, 2^28)", who, (long long)T);
  MOE_INVALID(H > 0 && H % 8 == 0, "%s: H=%lld must be a positive multiple of 8", who, (long long)H);
  MOE_UNSUPPORTED(H <= kMaxH, "%s: H=%lld > %lld is not supported", who, (long long)H, (long long)kMaxH);
  MOE_INVALID(type == MOE_TYPE_F32 || type == MOE_TYPE_BF16, "%s: x_type=%d must be MOE_TYPE_F32 or MOE_TYPE_BF16",
              who, (int)type);
  return MOE_OK;
}

// d_weight of a backward pass: the parts' sum, or zero where there are none
void add_parts(const float* part, int64_t P, int64_t H, float* out, hipStream_t st) {
  add_parts_kernel<<<dim3((unsigned)ceil_div(H, 64)), dim3(RD), 0, st>>>(part, (int)P, H, out);
}

template <int NC, int TYPE>
void launch_norm(const NormArgs& a, int quant, hipStream_t st) {
  const dim3 grid = rows_grid(a.T), block(threads_of(a.H, NC));
  if (quant == MOE_QUANT_E4M3) norm_kernel<NC, TYPE, MOE_QUANT_E4M3><<<grid, block, 0, st>>>(a);
  else if (quant == MOE_QUANT_INT8) norm_kernel<NC, TYPE, MOE_QUANT_INT8><<<grid, block, 0, st>>>(a);
  else norm_kernel<NC, TYPE, MOE_QUANT_NONE><<<grid, block, 0, st>>>(a);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_norm(const void* x, int32_t x_type, const void* add_bf16, const float* weight, int64_t T,
                        int64_t H, float eps, void* sum_out, void* n_bf16, float* rstd, int32_t quant,
                        void* codes, float* scales, void* stream) {
  clear_error();
  if (const int rc = check_rows("moe_norm", T, H, x_type)) return rc;
  MOE_INVALID(eps >= 0.0f && eps <= 1.0f, "moe_norm: eps=%g must be in [0, 1]", (double)eps);
  MOE_INVALID(quant >= MOE_QUANT_NONE && quant <= MOE_QUANT_INT8, "moe_norm: quant=%d is none of MOE_QUANT_*",
              (int)quant);
  MOE_INVALID(quant != MOE_QUANT_E4M3 || H % 128 == 0, "moe_norm: E4M3 codes need H %% 128 == 0, got %lld",
              (long long)H);
  MOE_INVALID((add_bf16 == nullptr) == (sum_out == nullptr),
              "moe_norm: add and sum_out are given together or not at all");
  if (T == 0) return MOE_OK;
  MOE_INVALID(x && n_bf16 && (quant == MOE_QUANT_NONE || (codes && scales)), "moe_norm: null pointer");
  MOE_INVALID(aligned(x, 16) && aligned(add_bf16, 16) && aligned(weight, 16) && aligned(sum_out, 16) &&
                  aligned(n_bf16, 16) && aligned(rstd, 4) && aligned(codes, 8) && aligned(scales, 4),
              "moe_norm: tensors must be 16-byte, codes 8-byte, rstd and scales 4-byte aligned");
  MOE_INVALID(n_bf16 != x && n_bf16 != add_bf16 && n_bf16 != sum_out, "moe_norm: n must not alias x, add or sum_out");
  const NormArgs a{x, static_cast<const uint16_t*>(add_bf16), weight, T, H, eps, sum_out,
                   static_cast<uint16_t*>(n_bf16), rstd, static_cast<uint8_t*>(codes), scales};
  hipStream_t st = as_stream(stream);
  if (x_type == MOE_TYPE_F32) {
    if (H <= 8192) launch_norm<1, MOE_TYPE_F32>(a, quant, st);
    else launch_norm<2, MOE_TYPE_F32>(a, quant, st);
  } else {
    if (H <= 8192) launch_norm<1, MOE_TYPE_BF16>(a, quant, st);
    else launch_norm<2, MOE_TYPE_BF16>(a, quant, st);
  }
  return check_launch("moe_norm");
}

extern "C" size_t moe_norm_backward_workspace_bytes(int64_t T, int64_t H) {
  return T > 0 && H > 0 ? (size_t)(parts_of(T, H) * H) * sizeof(float) : 0;
}

extern "C" int moe_norm_backward(const void* dn_bf16, const void* x, int32_t x_type, const float* weight,
                                 const float* rstd, const void* d_res, float res_scale, int64_t T, int64_t H,
                                 void* dx, float* d_weight, void* workspace, size_t workspace_bytes,
                                 void* stream) {
  clear_error();
  if (const int rc = check_rows("moe_norm_backward", T, H, x_type)) return rc;
  hipStream_t st = as_stream(stream);
  MOE_INVALID(aligned(d_weight, 16), "moe_norm_backward: d_weight must be 16-byte aligned");
  if (T == 0) {
    if (d_weight) add_parts(nullptr, 0, H, d_weight, st);
    return d_weight ? check_launch("moe_norm_backward") : MOE_OK;
  }
  MOE_INVALID(dn_bf16 && x && rstd && dx, "moe_norm_backward: null pointer");
  MOE_INVALID(aligned(dn_bf16, 16) && aligned(x, 16) && aligned(weight, 16) && aligned(rstd, 4) &&
                  aligned(d_res, 16) && aligned(dx, 16) && aligned(workspace, 16),
              "moe_norm_backward: tensors and workspace must be 16-byte, rstd 4-byte aligned");
  MOE_INVALID(dx != dn_bf16 && dx != x, "moe_norm_backward: dx must not alias dn or x");
  const int64_t P = parts_of(T, H);
  MOE_REQUIRE(!d_weight || (workspace && workspace_bytes >= moe_norm_backward_workspace_bytes(T, H)),
              MOE_ERR_WORKSPACE, "moe_norm_backward: workspace of %zu bytes, %zu needed", workspace_bytes,
              moe_norm_backward_workspace_bytes(T, H));
  const NormBwdArgs a{static_cast<const uint16_t*>(dn_bf16), x, weight, rstd, d_res, res_scale, T, H, dx,
                      part_of(d_weight, P, workspace)};
  const dim3 grid((unsigned)P);
  if (x_type == MOE_TYPE_F32) {
    if (H <= 8192) norm_backward_kernel<1, MOE_TYPE_F32><<<grid, dim3(threads_of(H, 1)), 0, st>>>(a);
    else norm_backward_kernel<2, MOE_TYPE_F32><<<grid, dim3(threads_of(H, 2)), 0, st>>>(a);
  } else {
    if (H <= 8192) norm_backward_kernel<1, MOE_TYPE_BF16><<<grid, dim3(threads_of(H, 1)), 0, st>>>(a);
    else norm_backward_kernel<2, MOE_TYPE_BF16><<<grid, dim3(threads_of(H, 2)), 0, st>>>(a);
  }
  if (d_weight && P > 1) add_parts(a.part, P, H, d_weight, st);
  return check_launch("moe_norm_backward");
}

static int check_combine(const char* who, int64_t T, int32_t k, int64_t H, int32_t type, int32_t norm, float eps) {
  if (const int rc = check_rows(who, T, H, type)) return rc;
  MOE_INVALID(k >= 1 && k <= 8, "%s: k=%d must be in [1, 8]", who, (int)k);
  MOE_INVALID(norm == 0 || norm == 1, "%s: norm=%d must be 0 or 1", who, (int)norm);
  MOE_INVALID(eps >= 0.0f && eps <= 1.0f, "%s: eps=%g must be in [0, 1]", who, (double)eps);
  return MOE_OK;
}

extern "C" int moe_combine_norm(const void* expert_out_bf16, const int32_t* inv_perm, const float* topk_w,
                                const void* shared_out_bf16, const float* shared_w, const void* residual,
                                int32_t x_type, float residual_scale, int32_t norm, const float* weight,
                                float eps, float scale, int64_t T, int32_t k, int64_t H, void* y, float* rstd,
                                void* stream) {
  clear_error();
  if (const int rc = check_combine("moe_combine_norm", T, k, H, x_type, norm, eps)) return rc;
  MOE_INVALID(!shared_w || shared_out_bf16, "moe_combine_norm: shared_w without shared rows");
  if (T == 0) return MOE_OK;
  MOE_INVALID(expert_out_bf16 && inv_perm && topk_w && residual && y, "moe_combine_norm: null pointer");
  MOE_INVALID(aligned(expert_out_bf16, 16) && aligned(shared_out_bf16, 16) && aligned(residual, 16) &&
                  aligned(weight, 16) && aligned(y, 16) && aligned(inv_perm, 4) && aligned(topk_w, 4) &&
                  aligned(shared_w, 4) && aligned(rstd, 4),
              "moe_combine_norm: tensors must be 16-byte, indices, gate weights and rstd 4-byte aligned");
  MOE_INVALID(y != expert_out_bf16 && y != shared_out_bf16, "moe_combine_norm: y must not alias the experts' rows");
  CombineArgs a{};
  a.D = static_cast<const uint16_t*>(expert_out_bf16);
  a.inv_perm = inv_perm, a.topk_w = topk_w;
  a.S = static_cast<const uint16_t*>(shared_out_bf16), a.shared_w = shared_w;
  a.residual = residual, a.residual_scale = residual_scale, a.scale = scale;
  a.norm = norm, a.weight = weight, a.eps = eps;
  a.T = T, a.H = H, a.k = k, a.y = y, a.rstd = norm ? rstd : nullptr;
  hipStream_t st = as_stream(stream);
  const dim3 grid = rows_grid(T);
  if (x_type == MOE_TYPE_F32) {
    if (H <= 8192) combine_norm_kernel<1, MOE_TYPE_F32><<<grid, dim3(threads_of(H, 1)), 0, st>>>(a);
    else combine_norm_kernel<2, MOE_TYPE_F32><<<grid, dim3(threads_of(H, 2)), 0, st>>>(a);
  } else {
    if (H <= 8192) combine_norm_kernel<1, MOE_TYPE_BF16><<<grid, dim3(threads_of(H, 1)), 0, st>>>(a);
    else combine_norm_kernel<2, MOE_TYPE_BF16><<<grid, dim3(threads_of(H, 2)), 0, st>>>(a);
  }
  return check_launch("moe_combine_norm");
}

extern "C" size_t moe_combine_norm_backward_workspace_bytes(int64_t T, int64_t H) {
  return moe_norm_backward_workspace_bytes(T, H);
}

extern "C" int moe_combine_norm_backward(const void* dy, int32_t x_type, const int32_t* inv_perm,
                                         const float* topk_w, const void* expert_out_bf16, int32_t n_shared,
                                         const float* shared_w, int32_t norm, const float* weight, float eps,
                                         float scale, int64_t T, int32_t k, int64_t H, void* d_expert_out_bf16,
                                         float* d_topk_w, float* d_shared_w, uint8_t* d_expert_out_e4m3,
                                         float* d_expert_out_scale, float* d_weight, void* workspace,
                                         size_t workspace_bytes, void* stream) {
  clear_error();
  const char* who = "moe_combine_norm_backward";
  if (const int rc = check_combine(who, T, k, H, x_type, norm, eps)) return rc;
  MOE_INVALID(n_shared == 0 || n_shared == 1, "%s: n_shared=%d must be 0 or 1", who, (int)n_shared);
  MOE_INVALID(n_shared == 1 || (!shared_w && !d_shared_w), "%s: shared_w or d_shared_w without shared rows", who);
  MOE_INVALID((d_expert_out_e4m3 == nullptr) == (d_expert_out_scale == nullptr),
              "%s: dD codes and scales are given together or not at all", who);
  MOE_INVALID(!d_expert_out_e4m3 || H % 128 == 0, "%s: quantised dD needs H %% 128 == 0, got %lld", who,
              (long long)H);
  MOE_INVALID(aligned(d_weight, 16), "%s: d_weight must be 16-byte aligned", who);
  hipStream_t st = as_stream(stream);
  if (T == 0) {
    if (d_weight) add_parts(nullptr, 0, H, d_weight, st);
    return d_weight ? check_launch(who) : MOE_OK;
  }
  MOE_INVALID(dy && inv_perm && topk_w && expert_out_bf16 && d_expert_out_bf16 && d_topk_w, "%s: null pointer", who);
  MOE_INVALID(aligned(dy, 16) && aligned(expert_out_bf16, 16) && aligned(d_expert_out_bf16, 16) &&
                  aligned(weight, 16) && aligned(workspace, 16) && aligned(inv_perm, 4) && aligned(topk_w, 4) &&
                  aligned(shared_w, 4) && aligned(d_topk_w, 4) && aligned(d_shared_w, 4) &&
                  aligned(d_expert_out_e4m3, 8) && aligned(d_expert_out_scale, 4),
              "%s: tensors and workspace must be 16-byte, codes 8-byte, the rest 4-byte aligned", who);
  MOE_INVALID(d_expert_out_bf16 != expert_out_bf16 && d_expert_out_bf16 != dy, "%s: dD must not alias D or dy", who);
  const int64_t P = parts_of(T, H);
  MOE_REQUIRE(!d_weight || (workspace && workspace_bytes >= moe_norm_backward_workspace_bytes(T, H)),
              MOE_ERR_WORKSPACE, "%s: workspace of %zu bytes, %zu needed", who, workspace_bytes,
              moe_norm_backward_workspace_bytes(T, H));
  CombineArgs a{};
  a.D = static_cast<const uint16_t*>(expert_out_bf16);
  a.inv_perm = inv_perm, a.topk_w = topk_w;
  a.S = n_shared ? a.D + T * k * H : nullptr, a.shared_w = shared_w;
  a.scale = scale, a.norm = norm, a.weight = weight, a.eps = eps;
  a.T = T, a.H = H, a.k = k, a.dy = dy;
  a.dD = static_cast<uint16_t*>(d_expert_out_bf16);
  a.d_topk_w = d_topk_w, a.d_shared_w = d_shared_w;
  a.codes = d_expert_out_e4m3, a.scales = d_expert_out_scale;
  a.part = part_of(d_weight, P, workspace);
  const dim3 grid((unsigned)P);
  if (x_type == MOE_TYPE_F32) {
    if (H <= 8192) combine_norm_backward_kernel<1, MOE_TYPE_F32, true><<<grid, dim3(threads_of(H, 1)), 0, st>>>(a);
    else combine_norm_backward_kernel<2, MOE_TYPE_F32, false><<<grid, dim3(threads_of(H, 2)), 0, st>>>(a);
  } else {
    if (H <= 8192) combine_norm_backward_kernel<1, MOE_TYPE_BF16, true><<<grid, dim3(threads_of(H, 1)), 0, st>>>(a);
    else combine_norm_backward_kernel<2, MOE_TYPE_BF16, false><<<grid, dim3(threads_of(H, 2)), 0, st>>>(a);
  }
  if (d_weight && P > 1) add_parts(a.part, P, H, d_weight, st);
  return check_launch(who);
}
