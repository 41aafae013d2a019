// The gate on given router logits: softmax or sigmoid scores, an optional
// bias that only moves the choice, group-limited top-k, weights that are
// renormalised or not, the experts' counts; and its gradient.
//
// Per token with logits l and chosen experts e_j:
//   s = softmax(l) or 1 / (1 + exp(-l));  v = s + bias (l itself without one)
//   w_j = scale * s_{e_j}, divided by S = sum_j s_{e_j} when renormalised
// and backwards, for the gradients dw of w and ds of s:
//   ds[e_j] += scale * dw_j                              (as they are)
//   ds[e_j] += scale * (dw_j - sum_i dw_i s_i / S) / S   (renormalised)
//   dl = s (ds - sum_e ds_e s_e)  (softmax),  ds s (1 - s)  (sigmoid)
//
// The order of the experts is that of the exact values: v is formed in 64
// bits from the fp32 logits, so that two experts whose fp32 scores round to
// the same number, or the wrong way round, are still told apart.
#include "common.h"

namespace moe {
namespace {

constexpr int GT = 256;       // threads of a workgroup: four waves
constexpr int GMAXE = 1024;   // experts (16 to a lane)
constexpr int GMAXG = 32;     // groups
constexpr int GMAXK = 8;

struct GateArgs {
  const void* logits;
  const float* bias;
  int64_t T;
  int E, n_group, topk_group, group_top, k;
  bool softmax, renorm;
  float scale;
  int32_t* topk_idx;
  float* topk_w;
  int32_t* counts;
  float* scores;
};

template <typename D>
__device__ __forceinline__ float load_logit(const D* p);
template <>
__device__ __forceinline__ float load_logit<float>(const float* p) { return *p; }
template <>
__device__ __forceinline__ float load_logit<uint16_t>(const uint16_t* p) { return bf16_to_f32(*p); }

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
  return v;
}
template <typename F>
__device__ __forceinline__ F wave_sum(F v) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) v += __shfl_xor(v, o, 64);
  return v;
}

// One token by one wave; expert i * 64 + lane sits in slot i of a lane.
// s_v: the wave's [E] doubles, s_g: its [GMAXG] doubles.
template <typename D, int VPL>
__device__ __forceinline__ void gate_token(const GateArgs& a, int64_t t, double* s_v, double* s_g,
                                           int* hist) {
  const int lane = threadIdx.x & 63;
  const D* row = static_cast<const D*>(a.logits) + t * a.E;
  const int E = a.E, size = E / a.n_group;
  float l[VPL], s[VPL];
  double v[VPL];
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = i * 64 + lane;
    l[i] = e < E ? load_logit(row + e) : -INFINITY;
    m = fmaxf(m, l[i]);
  }
  m = wave_max(m);
  if (a.softmax) {
    double z = 0.0;
    float zf = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      // a row of -inf has no score at all
      const bool there = l[i] != -INFINITY;
      v[i] = there ? exp((double)l[i] - (double)m) : 0.0;
      s[i] = there ? expf(l[i] - m) : 0.f;
      z += v[i];
      zf += s[i];
    }
    z = wave_sum(z);
    zf = wave_sum(zf);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      v[i] = z > 0.0 ? v[i] / z : 0.0;
      s[i] = zf > 0.f ? s[i] / zf : 0.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      v[i] = 1.0 / (1.0 + exp(-(double)l[i]));
      s[i] = 1.0f / (1.0f + expf(-l[i]));
    }
  }
  if (a.scores) {
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (i * 64 + lane < E) a.scores[t * E + i * 64 + lane] = s[i];
  }
  // values of the order; excluded experts (-inf or NaN) below every other,
  // slots that are no candidates at -inf
  const double kExcluded = -1.7e308;
  auto order = [&](double x, float li) { return (li > -INFINITY && x > kExcluded) ? x : kExcluded; };
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = i * 64 + lane;
    if (e >= E) {
      v[i] = -INFINITY;
      continue;
    }
    if (a.bias) v[i] += (double)a.bias[e];
    const double x = (a.bias || a.group_top == 2) ? v[i] : (double)l[i];
    if (a.n_group > 1) s_v[e] = order(x, l[i]);
    v[i] = order(a.bias ? v[i] : (double)l[i], l[i]);
  }
  if (a.n_group > 1) {
    __builtin_amdgcn_wave_barrier();
    if (lane < a.n_group) {
      double t1 = -INFINITY, t2 = -INFINITY;
      for (int i = 0; i < size; ++i) {
        const double x = s_v[lane * size + i];
        if (x > kExcluded) {
          t2 = fmax(t2, fmin(t1, x));
          t1 = fmax(t1, x);
        }
      }
      s_g[lane] = (a.group_top == 2 && t2 > -INFINITY) ? t1 + t2 : t1;
    }
    __builtin_amdgcn_wave_barrier();
    const double mine = s_g[lane < a.n_group ? lane : 0];
    int rank = 0;
    for (int j = 0; j < a.n_group; ++j) {
      const double x = s_g[j];
      rank += (x > mine || (x == mine && j < lane)) ? 1 : 0;
    }
    const uint64_t kept = __ballot(lane < a.n_group && rank < a.topk_group);
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (i * 64 + lane < E && !((kept >> ((i * 64 + lane) / size)) & 1)) v[i] = -INFINITY;
  }
  // k times the largest that is left, the lowest id among equals
  uint32_t taken = 0;
  for (int j = 0; j < a.k; ++j) {
    double best = -INFINITY;
    int at = 0x7FFFFFFF;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (!((taken >> i) & 1) && (v[i] > best)) {
        best = v[i];
        at = i * 64 + lane;
      }
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const double b = __shfl_xor(best, o, 64);
      const int w = __shfl_xor(at, o, 64);
      if (b > best || (b == best && w < at)) {
        best = b;
        at = w;
      }
    }
    if ((at & 63) == lane) taken |= 1u << (at >> 6);
  }
  // ids ascending: slots in order, lanes in order within a slot
  const uint64_t below = (1ull << lane) - 1ull;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) sum += ((taken >> i) & 1) ? s[i] : 0.f;
  sum = wave_sum(sum);
  int base = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const bool mine = (taken >> i) & 1;
    const uint64_t msk = __ballot(mine);
    if (mine) {
      const int64_t o = t * a.k + base + __popcll(msk & below);
      a.topk_idx[o] = i * 64 + lane;
      const float w = a.renorm ? (sum > 0.f ? s[i] / sum : 0.f) : s[i];
      a.topk_w[o] = w * a.scale;
      atomicAdd(&hist[i * 64 + lane], 1);
    }
    base += __popcll(msk);
  }
}

template <typename D, int VPL>
__global__ __launch_bounds__(GT) void gate_kernel(GateArgs a) {
  __shared__ int hist[64 * VPL];
  __shared__ double s_v[GT / 64][64 * VPL];
  __shared__ double s_g[GT / 64][GMAXG];
  for (int i = threadIdx.x; i < 64 * VPL; i += GT) hist[i] = 0;
  __syncthreads();
  const int wv = threadIdx.x >> 6;
  for (int64_t t = (int64_t)blockIdx.x * (GT / 64) + wv; t < a.T; t += (int64_t)gridDim.x * (GT / 64))
    gate_token<D, VPL>(a, t, s_v[wv], s_g[wv], hist);
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += GT) {
    const int c = hist[e];
    if (c) atomicAdd(&a.counts[e], c);
  }
}

__global__ __launch_bounds__(GT) void gate_zero_kernel(int32_t* p, int n) {
  for (int i = threadIdx.x; i < n; i += GT) p[i] = 0;
}

struct GateBwdArgs {
  const void* logits;
  const int32_t* idx;
  const float* dw;
  const float* ds;
  void* dl;
  int64_t T;
  int E, k;
  bool softmax, renorm;
  float scale;
};

template <typename D>
__device__ __forceinline__ void store_grad(D* p, float v);
template <>
__device__ __forceinline__ void store_grad<float>(float* p, float v) { *p = v; }
template <>
__device__ __forceinline__ void store_grad<uint16_t>(uint16_t* p, float v) { *p = (uint16_t)f32_to_bf16_rne(v); }

// One wave per token, expert i * 64 + lane in slot i.
template <typename D, int VPL>
__global__ __launch_bounds__(GT) void gate_backward_kernel(GateBwdArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * (GT / 64) + (threadIdx.x >> 6);
  if (t >= a.T) return;
  const int E = a.E;
  const D* row = static_cast<const D*>(a.logits) + t * E;
  float s[VPL], g[VPL];
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = i * 64 + lane;
    s[i] = e < E ? load_logit(row + e) : -INFINITY;
    g[i] = a.ds && e < E ? a.ds[t * E + e] : 0.f;
    m = fmaxf(m, s[i]);
  }
  if (a.softmax) {
    m = wave_max(m);
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      s[i] = s[i] == -INFINITY ? 0.f : expf(s[i] - m);
      z += s[i];
    }
    z = wave_sum(z);
#pragma unroll
    for (int i = 0; i < VPL; ++i) s[i] = z > 0.f ? s[i] / z : 0.f;
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) s[i] = 1.0f / (1.0f + expf(-s[i]));
  }
  int id[GMAXK];
  float dw[GMAXK], sj[GMAXK];
  float S = 0.f, dot = 0.f;
#pragma unroll
  for (int j = 0; j < GMAXK; ++j) {
    id[j] = -1;
    dw[j] = sj[j] = 0.f;
    if (j < a.k) {
      const int e = a.idx[t * a.k + j];
      if ((uint32_t)e < (uint32_t)E) {
        id[j] = e;
        dw[j] = a.scale * a.dw[t * a.k + j];
      }
      float mine = 0.f;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (id[j] == i * 64 + lane) mine = s[i];
      sj[j] = wave_sum(mine);
      S += sj[j];
    }
  }
  if (a.renorm) {
#pragma unroll
    for (int j = 0; j < GMAXK; ++j) dot = fmaf(dw[j], S > 0.f ? sj[j] / S : 0.f, dot);
#pragma unroll
    for (int j = 0; j < GMAXK; ++j) dw[j] = S > 0.f ? (dw[j] - dot) / S : 0.f;
  }
#pragma unroll
  for (int j = 0; j < GMAXK; ++j)
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (id[j] == i * 64 + lane) g[i] += dw[j];
  float p = 0.f;
  if (a.softmax) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) p = fmaf(g[i], s[i], p);
    p = wave_sum(p);
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = i * 64 + lane;
    if (e < E)
      store_grad(static_cast<D*>(a.dl) + t * E + e,
                 a.softmax ? s[i] * (g[i] - p) : g[i] * s[i] * (1.0f - s[i]));
  }
}

template <typename D>
void launch_gate(const GateArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)std::min<int64_t>(ceil_div(a.T, GT / 64), 2048)), block(GT);
  if (a.E <= 64) gate_kernel<D, 1><<<grid, block, 0, st>>>(a);
  else if (a.E <= 128) gate_kernel<D, 2><<<grid, block, 0, st>>>(a);
  else if (a.E <= 256) gate_kernel<D, 4><<<grid, block, 0, st>>>(a);
  else if (a.E <= 512) gate_kernel<D, 8><<<grid, block, 0, st>>>(a);
  else gate_kernel<D, 16><<<grid, block, 0, st>>>(a);
}

template <typename D>
void launch_gate_backward(const GateBwdArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)ceil_div(a.T, GT / 64)), block(GT);
  if (a.E <= 64) gate_backward_kernel<D, 1><<<grid, block, 0, st>>>(a);
  else if (a.E <= 128) gate_backward_kernel<D, 2><<<grid, block, 0, st>>>(a);
  else if (a.E <= 256) gate_backward_kernel<D, 4><<<grid, block, 0, st>>>(a);
  else if (a.E <= 512) gate_backward_kernel<D, 8><<<grid, block, 0, st>>>(a);
  else gate_backward_kernel<D, 16><<<grid, block, 0, st>>>(a);
}

int gate_shape(const char* who, int64_t T, int32_t E, int32_t type, int32_t score, int32_t k,
               float scale) {
  MOE_INVALID(T >= 0, "%s: T=%lld < 0", who, (long long)T);
  MOE_INVALID(E >= 1, "%s: E=%d < 1", who, (int)E);
  MOE_INVALID(type == MOE_TYPE_F32 || type == MOE_TYPE_BF16, "%s: logits_type=%d must be 0 or 1", who,
              (int)type);
  MOE_INVALID(score == MOE_SCORE_SOFTMAX || score == MOE_SCORE_SIGMOID,
              "%s: score=%d must be 0 or 1", who, (int)score);
  MOE_INVALID(k >= 1 && k <= E, "%s: k=%d must be in [1, E=%d]", who, (int)k, (int)E);
  MOE_INVALID(scale - scale == 0.f, "%s: scale must be finite", who);
  MOE_UNSUPPORTED(E <= GMAXE, "%s: E=%d > %d experts is not supported", who, (int)E, GMAXE);
  MOE_UNSUPPORTED(k <= GMAXK, "%s: k=%d > %d is not supported", who, (int)k, GMAXK);
  MOE_UNSUPPORTED(T < (1ll << 31), "%s: T=%lld is not supported", who, (long long)T);
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" int moe_gate(const void* logits, int32_t logits_type, int64_t T, int32_t E,
                        const float* bias, int32_t score, int32_t n_group, int32_t topk_group,
                        int32_t group_top, int32_t k, int32_t renormalize, float scale,
                        int32_t* topk_idx, float* topk_w, int32_t* expert_counts, float* scores,
                        void* stream) {
  clear_error();
  const int rc = gate_shape("moe_gate", T, E, logits_type, score, k, scale);
  if (rc != MOE_OK) return rc;
  MOE_INVALID(n_group >= 1 && E % n_group == 0, "moe_gate: E=%d not divisible by n_group=%d", (int)E,
              (int)n_group);
  MOE_INVALID(topk_group >= 1 && topk_group <= n_group,
              "moe_gate: topk_group=%d must be in [1, n_group=%d]", (int)topk_group, (int)n_group);
  MOE_INVALID(group_top == 1 || group_top == 2, "moe_gate: group_top=%d must be 1 or 2",
              (int)group_top);
  MOE_INVALID(renormalize == 0 || renormalize == 1, "moe_gate: renormalize=%d must be 0 or 1",
              (int)renormalize);
  MOE_INVALID(k <= topk_group * (E / n_group), "moe_gate: k=%d must be in [1, %d]", (int)k,
              (int)(topk_group * (E / n_group)));
  MOE_UNSUPPORTED(n_group <= GMAXG, "moe_gate: n_group=%d > %d is not supported", (int)n_group, GMAXG);
  MOE_INVALID(expert_counts && ((uintptr_t)expert_counts & 3) == 0,
              "moe_gate: expert_counts must be non-null and 4-byte aligned");
  hipStream_t st = as_stream(stream);
  if (T > 0) {
    MOE_INVALID(logits && topk_idx && topk_w, "moe_gate: null pointer");
    MOE_INVALID(((uintptr_t)logits & (logits_type == MOE_TYPE_F32 ? 3 : 1)) == 0 &&
                    ((uintptr_t)bias & 3) == 0 && ((uintptr_t)topk_idx & 3) == 0 &&
                    ((uintptr_t)topk_w & 3) == 0 && ((uintptr_t)scores & 3) == 0,
                "moe_gate: tensors must be aligned to their elements");
  }
  gate_zero_kernel<<<1, GT, 0, st>>>(expert_counts, E);
  if (T > 0) {
    const GateArgs a{logits, bias, T, E, n_group, topk_group, group_top, k,
                     score == MOE_SCORE_SOFTMAX, renormalize != 0, scale,
                     topk_idx, topk_w, expert_counts, scores};
    if (logits_type == MOE_TYPE_F32) launch_gate<float>(a, st);
    else launch_gate<uint16_t>(a, st);
  }
  return check_launch("moe_gate");
}

extern "C" int moe_gate_backward(const void* logits, int32_t logits_type, int64_t T, int32_t E,
                                 int32_t score, int32_t k, int32_t renormalize, float scale,
                                 const int32_t* topk_idx, const float* d_topk_w,
                                 const float* d_scores, void* d_logits, void* stream) {
  clear_error();
  const int rc = gate_shape("moe_gate_backward", T, E, logits_type, score, k, scale);
  if (rc != MOE_OK) return rc;
  MOE_INVALID(renormalize == 0 || renormalize == 1, "moe_gate_backward: renormalize=%d must be 0 or 1",
              (int)renormalize);
  if (T == 0) return MOE_OK;
  MOE_INVALID(logits && topk_idx && d_topk_w && d_logits, "moe_gate_backward: null pointer");
  const uintptr_t lm = logits_type == MOE_TYPE_F32 ? 3 : 1;
  MOE_INVALID(((uintptr_t)logits & lm) == 0 && ((uintptr_t)d_logits & lm) == 0 &&
                  ((uintptr_t)topk_idx & 3) == 0 && ((uintptr_t)d_topk_w & 3) == 0 &&
                  ((uintptr_t)d_scores & 3) == 0,
              "moe_gate_backward: tensors must be aligned to their elements");
  MOE_INVALID(logits != d_logits, "moe_gate_backward: logits and d_logits alias");
  const GateBwdArgs a{logits, topk_idx, d_topk_w, d_scores, d_logits, T, E, k,
                      score == MOE_SCORE_SOFTMAX, renormalize != 0, scale};
  if (logits_type == MOE_TYPE_F32) launch_gate_backward<float>(a, as_stream(stream));
  else launch_gate_backward<uint16_t>(a, as_stream(stream));
  return check_launch("moe_gate_backward");
}
