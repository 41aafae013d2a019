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
// (renormalised: with p_j = s_j / S, dl[e_j] += scale p_j (dw_j - sum_i dw_i p_i),
// times 1 - s_j for a sigmoid).
//
// The order of the experts is that of the values in 64 bits: where the fp32
// values at the border between chosen and not chosen (of experts or of groups)
// are nearer to each other than their error, a token is done again with v in 64
// bits from the logits.  Without a bias the logits themselves are ordered, equal
// ones in place.
//
// The floor is one read of the logits (16.8 MB of fp32 at 16384 x 256: 2.8 us);
// the selection is what costs, so it is spread over four tokens a wave: 16
// lanes hold a token (all 64 above 256 experts), a lane 4 C of its logits
// (chunk c: experts 4 (16 c + lane) .. +3).  Each lane sorts its 8 largest,
// then lists of 8 are merged across the lanes (DPP moves); the k-th entry is
// the threshold that every lane compares its values with.
//
// Measured, with the counts' launch, 256 experts of fp32, softmax without a bias:
// 16384 tokens 9.6 us, 11.9 with the scores stored (34.6 MB), one token 3.9 (one
// launch).  A biased sigmoid in 8 groups: 16384 tokens 21.3 us, of which 7 are the
// second look of the few that need one; 128 tokens 8.4; one token 6.6, 13.0 with
// a second look.  With bf16 logits and equal biases 8 % of 16384 tokens tie at the
// border, up to four of a wave one after the other: 30 to 36 us.
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
  int size;        // of a group
  int share;       // log2 of the lanes that look at one
  uint32_t magic;  // e / size = e * magic >> 20 for e < 1024
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

__device__ __forceinline__ void load4(const float* p, float* v) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}
__device__ __forceinline__ void load4(const uint16_t* p, float* v) {
  const uint2 a = *reinterpret_cast<const uint2*>(p);
  v[0] = bf16_to_f32(a.x & 0xFFFFu); v[1] = bf16_to_f32(a.x >> 16);
  v[2] = bf16_to_f32(a.y & 0xFFFFu); v[3] = bf16_to_f32(a.y >> 16);
}

// The value of a lane's partner in the merge rounds 0, 1, 2, 3 (of 16 lanes:
// quad_perm [1,0,3,2] and [2,3,0,1], then the mirror lane of a half row and of
// a row) and 4, 5 (xor 16 and 32): after round r a lane has combined 2^(r+1)
// lanes, each once.
template <int R>
__device__ __forceinline__ int partner(int x) {
  if (R == 0) return __builtin_amdgcn_mov_dpp(x, 0xB1, 0xF, 0xF, true);
  if (R == 1) return __builtin_amdgcn_mov_dpp(x, 0x4E, 0xF, 0xF, true);
  if (R == 2) return __builtin_amdgcn_mov_dpp(x, 0x141, 0xF, 0xF, true);
  if (R == 3) return __builtin_amdgcn_mov_dpp(x, 0x140, 0xF, 0xF, true);
  // rows (halves) exchanged between two registers: [0] has the even rows (the
  // lower half) twice, [1] the odd ones (the upper half)
  const int lane = threadIdx.x & 63;
  if (R == 4) {
    const auto r = __builtin_amdgcn_permlane16_swap((uint32_t)x, (uint32_t)x, false, false);
    return (int)(lane & 16 ? r[0] : r[1]);
  }
  const auto r = __builtin_amdgcn_permlane32_swap((uint32_t)x, (uint32_t)x, false, false);
  return (int)(lane & 32 ? r[0] : r[1]);
}
template <int R>
__device__ __forceinline__ float partner(float v) { return __int_as_float(partner<R>(__float_as_int(v))); }
template <int R>
__device__ __forceinline__ double partner(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)partner<R>((int)(uint32_t)b), hi = (uint32_t)partner<R>((int)(b >> 32));
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
template <int LPT, typename F, typename V>
__device__ __forceinline__ V over_row(F f, V v) {
  v = f(v, partner<0>(v));
  v = f(v, partner<1>(v));
  v = f(v, partner<2>(v));
  v = f(v, partner<3>(v));
  if (LPT == 64) {
    v = f(v, partner<4>(v));
    v = f(v, partner<5>(v));
  }
  return v;
}
template <int LPT, typename V>
__device__ __forceinline__ V row_max(V v) { return over_row<LPT>([](V a, V b) { return max(a, b); }, v); }
template <int LPT, typename V>
__device__ __forceinline__ V row_sum(V v) { return over_row<LPT>([](V a, V b) { return a + b; }, v); }
template <typename V>
__device__ __forceinline__ V wave_sum(V v) { return row_sum<64>(v); }
__device__ __forceinline__ float wave_max(float v) {
  return over_row<64>([](float a, float b) { return fmaxf(a, b); }, v);
}

// whole numbers in the order of the floats (and back): their maxima need no
// care for NaN, which would cost an instruction each
__device__ __forceinline__ int order_key(float x) {
  const int b = __float_as_int(x);
  return b ^ ((b >> 31) & 0x7FFFFFFF);
}
__device__ __forceinline__ float from_key(int b) { return __int_as_float(b ^ ((b >> 31) & 0x7FFFFFFF)); }

// 1 / (1 + exp(-l)) with a relative error of 6 roundings at any l
__device__ __forceinline__ float sigmoid_f32(float l) {
  const float z = expf(-fabsf(l)), d = 1.0f + z;  // d in [1, 2]
  float y = __builtin_amdgcn_rcpf(d);
  y = fmaf(fmaf(-d, y, 1.0f), y, y);
  return l >= 0.f ? y : z * y;
}
// its slope, s (1 - s) = z / (1 + z)^2 with z = exp(-|l|): 1 - s of a rounded s
// has no bits left where s is near 1.  Relative error 9 roundings at any l.
__device__ __forceinline__ float sigmoid_slope(float l) {
  const float z = expf(-fabsf(l)), d = 1.0f + z;
  float y = __builtin_amdgcn_rcpf(d);
  y = fmaf(fmaf(-d, y, 1.0f), y, y);
  return z * y * y;
}
// exp(l - m), relative error (2.2 |l - m| + 2) roundings
__device__ __forceinline__ float exp_from(float l, float m) {
  return __builtin_amdgcn_exp2f((l - m) * 1.4426950408889634f);
}

// Under such a sum S of chosen scores those under 2^-126 (0 in a softmax, or
// subnormal) would be more than 2^-62 of it.  The scores are exp(l) times one
// factor there (1 + exp(l) is 1), so that s_j / S can be formed of exp(l_j - c),
// c the largest logit chosen.
constexpr float kLow = 0x1p-64f;

// s_j / S over the choices of a token, of which lane j of the row of 16 has the
// logit lj (-inf: none); m, inv: the softmax's largest logit and 1 / sum.  0
// where all scores are 0 in fp32.
__device__ __forceinline__ float share(bool softmax, float lj, float m, float inv) {
  float s = softmax ? exp_from(lj, m) * inv : sigmoid_f32(lj);
  float sum = row_sum<16>(s);
  if (sum > 0.f && sum < kLow) {
    s = exp_from(lj, row_max<16>(lj));
    sum = row_sum<16>(s);
  }
  return sum > 0.f ? s / sum : 0.f;
}

// One token by one wave, its order in 64 bits; expert i * 64 + lane sits in
// slot i of a lane.  s_v: the wave's [64 VPL] doubles, s_g: its [GMAXG].  The
// code is small (one exp in a rolled loop): it is read cold.
template <typename D, int VPL, bool ONE>
__device__ __forceinline__ void gate_token(const GateArgs& a, int64_t t, double* s_v, double* s_g,
                                           int* s_hist) {
  const int lane = threadIdx.x & 63;
  const D* row = static_cast<const D*>(a.logits) + t * a.E;
  const int E = a.E, size = a.size;
  float l[VPL], s[VPL], bias[VPL];
  double v[VPL];
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = i * 64 + lane;
    l[i] = e < E ? load_logit(row + e) : -INFINITY;
    bias[i] = a.bias && e < E ? a.bias[e] : 0.f;
    m = fmaxf(m, l[i]);
  }
  m = a.softmax ? wave_max(m) : 0.f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) s_v[i * 64 + lane] = a.softmax ? (double)l[i] - (double)m : -fabs((double)l[i]);
  double z = 0.0;
#pragma unroll 1
  for (int i = 0; i < VPL; ++i) {
    const double x = s_v[i * 64 + lane];
    const double y = x > -INFINITY ? exp(x) : 0.0;  // (a row of -inf has no score at all)
    s_v[i * 64 + lane] = y;
    z += y;
  }
  z = a.softmax ? wave_sum(z) : 0.0;
  const double inv = z > 0.0 ? 1.0 / z : 0.0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const double y = s_v[i * 64 + lane];
    v[i] = a.softmax ? y * inv : (l[i] >= 0.f ? 1.0 : y) / (1.0 + y);
    // (0 where the first look has 0)
    s[i] = a.softmax && !(exp_from(l[i], m) > 0.f) ? 0.f : (float)v[i];
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
    v[i] += (double)bias[i];
    const double x = (a.bias || a.group_top == 2) ? v[i] : (double)l[i];
    if (a.n_group > 1) s_v[e] = order(x, l[i]);
    v[i] = order(a.bias ? v[i] : (double)l[i], l[i]);
  }
  if (a.n_group > 1) {
    __builtin_amdgcn_wave_barrier();
    // 2^sh lanes a group, every 2^sh-th expert each
    int sh = 0;
    while (sh < 3 && a.n_group << (sh + 1) <= 64) ++sh;
    const int g = lane >> sh, part = lane & ((1 << sh) - 1);
    double t1 = -INFINITY, t2 = -INFINITY;
    auto take = [&](double x) {
      t2 = fmax(t2, fmin(t1, x));
      t1 = fmax(t1, x);
    };
    if (g < a.n_group) {
#pragma unroll 4
      for (int i = part; i < size; i += 1 << sh) {
        const double x = s_v[g * size + i];
        if (x > kExcluded) take(x);
      }
    }
    auto meet2 = [&](double y1, double y2) {
      take(y1);
      t2 = fmax(t2, y2);
    };
    if (sh > 0) meet2(partner<0>(t1), partner<0>(t2));
    if (sh > 1) meet2(partner<1>(t1), partner<1>(t2));
    if (sh > 2) meet2(partner<2>(t1), partner<2>(t2));
    if (g < a.n_group && part == 0) s_g[g] = (a.group_top == 2 && t2 > -INFINITY) ? t1 + t2 : t1;
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
      if (i * 64 + lane < E && !((kept >> (((i * 64 + lane) * a.magic) >> 20)) & 1)) v[i] = -INFINITY;
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
    auto meet = [&](double b, int w) {
      if (b > best || (b == best && w < at)) {
        best = b;
        at = w;
      }
    };
    meet(partner<0>(best), partner<0>(at));
    meet(partner<1>(best), partner<1>(at));
    meet(partner<2>(best), partner<2>(at));
    meet(partner<3>(best), partner<3>(at));
    meet(partner<4>(best), partner<4>(at));
    meet(partner<5>(best), partner<5>(at));
    if ((at & 63) == lane) taken |= 1u << (at >> 6);
  }
  // ids ascending: slots in order, lanes in order within a slot
  const uint64_t below = (1ull << lane) - 1ull;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < VPL; ++i) sum += ((taken >> i) & 1) ? s[i] : 0.f;
  sum = wave_sum(sum);
  if (a.renorm && sum > 0.f && sum < kLow) {  // (as in share)
    float c = -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) c = ((taken >> i) & 1) ? fmaxf(c, l[i]) : c;
    c = wave_max(c);
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      s[i] = exp_from(l[i], c);
      sum += ((taken >> i) & 1) ? s[i] : 0.f;
    }
    sum = wave_sum(sum);
  }
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
      if (ONE) atomicAdd(&s_hist[i * 64 + lane], 1);
    }
    base += __popcll(msk);
  }
}

__device__ __forceinline__ void order2(int& hi, int& lo) {
  const int a = max(hi, lo), b = min(hi, lo);
  hi = a;
  lo = b;
}
// descending sort of 8 (19 exchanges), and of 8 that rise and then fall or
// fall and then rise (12)
__device__ __forceinline__ void sort8(int* v) {
  order2(v[0], v[1]); order2(v[2], v[3]); order2(v[4], v[5]); order2(v[6], v[7]);
  order2(v[0], v[2]); order2(v[1], v[3]); order2(v[4], v[6]); order2(v[5], v[7]);
  order2(v[1], v[2]); order2(v[5], v[6]); order2(v[0], v[4]); order2(v[3], v[7]);
  order2(v[1], v[5]); order2(v[2], v[6]);
  order2(v[1], v[4]); order2(v[3], v[6]);
  order2(v[2], v[4]); order2(v[3], v[5]);
  order2(v[3], v[4]);
}
__device__ __forceinline__ void merge8(int* v) {
#pragma unroll
  for (int d = 4; d > 0; d >>= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!(i & d)) order2(v[i], v[i + d]);
}
// a: the 8 largest of a and of b (both descending)
__device__ __forceinline__ void join8(int* a, const int* b) {
#pragma unroll
  for (int i = 0; i < 8; ++i) a[i] = max(a[i], b[7 - i]);
  merge8(a);
}
template <int R>
__device__ __forceinline__ void round8(int* a) {
  int b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = partner<R>(a[i]);
  join8(a, b);
}

// sum over the lanes up to this one (l: its place in the row)
template <int LPT>
__device__ __forceinline__ int row_scan(int v, int l) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);  // row_shr 1, 2, 4, 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
  if (LPT == 64) {
    const int r0 = __builtin_amdgcn_readlane(v, 15), r1 = __builtin_amdgcn_readlane(v, 31),
              r2 = __builtin_amdgcn_readlane(v, 47);
    v += (l >= 16 ? r0 : 0) + (l >= 32 ? r1 : 0) + (l >= 48 ? r2 : 0);
  }
  return v;
}

// LPT lanes hold a token, each 4 C of its logits: expert 4 (LPT c + lane) + j
// in slot 4 c + j.  ONE: a single workgroup, which counts the choices itself.
template <typename D, int LPT, int C, bool ONE>
__global__ __launch_bounds__(GT) void gate_kernel(GateArgs a) {
  constexpr int TPW = 64 / LPT, V = 4 * C, EMAX = LPT * V, W = GT / 64;
  constexpr int PITCH = EMAX + 8;  // floats of a token's row in LDS: rows in different banks
  constexpr int BYTES = TPW * PITCH * 4 > EMAX * 8 ? TPW * PITCH * 4 : EMAX * 8;
  __shared__ __attribute__((aligned(16))) uint8_t s_mem[W][BYTES];
  __shared__ __attribute__((aligned(16))) double s_g[W][GMAXG];
  __shared__ __attribute__((aligned(16))) int s_ids[W][TPW][GMAXK];
  __shared__ int s_hist[ONE ? EMAX : 1];
  if (ONE) {
    for (int e = threadIdx.x; e < a.E; e += GT) s_hist[e] = 0;
    __syncthreads();
  } else if (blockIdx.x == 0) {  // for the counting kernel
    for (int e = threadIdx.x; e < a.E; e += GT) a.counts[e] = 0;
  }
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int sub = lane / LPT;
  const int E = a.E, k = a.k;
  const bool vec = (E & 3) == 0 && ((uintptr_t)a.logits & (4 * sizeof(D) - 1)) == 0;
  const bool vec_out = (E & 3) == 0 && ((uintptr_t)a.scores & 15) == 0;
  const int64_t step = (int64_t)gridDim.x * W * TPW, first = ((int64_t)blockIdx.x * W + wv) * TPW;
  const int size = a.size;
  // the bias waits in LDS, read while the first tokens' logits are on their way
  __shared__ __attribute__((aligned(16))) float s_bias[EMAX];
  if (a.bias) {
    const float warm = load_logit(static_cast<const D*>(a.logits) + min(first + sub, a.T - 1) * E +
                                  min((lane & (LPT - 1)) * V, E - 1));
    for (int e = threadIdx.x; e < EMAX; e += GT) s_bias[e] = a.bias[min(e, E - 1)];
    __syncthreads();
    asm volatile("" ::"v"(warm));
  }
  uint64_t any = 0;  // whether a token of this wave is left for the second look
  for (int64_t t0 = first; t0 < a.T; t0 += step) {
    const int64_t t = min(t0 + sub, a.T - 1);
    const bool here = t0 + sub < a.T;
    // (through an empty asm: what follows from the lane's place is formed in
    // every round, not kept in registers for the next)
    int l = lane & (LPT - 1);
    asm volatile("" : "+v"(l));
    const D* row = static_cast<const D*>(a.logits) + t * E;
    float x[V], s[V];  // logits, then the values ordered; scores
    if (vec && E == EMAX) {
#pragma unroll
      for (int c = 0; c < C; ++c) load4(row + 4 * (LPT * c + l), x + 4 * c);
    } else if (vec) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int e = 4 * (LPT * c + l);
        load4(row + min(e, E - 4), x + 4 * c);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[4 * c + j] = e < E ? x[4 * c + j] : -INFINITY;
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = 4 * (LPT * (i >> 2) + l) + (i & 3);
        const float y = load_logit(row + min(e, E - 1));
        x[i] = e < E ? y : -INFINITY;
      }
    }
    float m = 0.f, inv = 0.f, smax = 1.f;
    if (a.softmax) {
      int mk = order_key(x[0]);
#pragma unroll
      for (int i = 1; i < V; ++i) mk = max(mk, order_key(x[i]));
      m = from_key(row_max<LPT>(mk));
      m = m == -INFINITY ? 0.f : m;  // (no logit there: every score is 0)
      float z = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        s[i] = exp_from(x[i], m);
        z += s[i];
      }
      z = row_sum<LPT>(z);
      smax = inv = z > 0.f ? 1.0f / z : 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] *= inv;
    } else if (a.scores || a.bias || a.n_group > 1) {
#pragma unroll
      for (int i = 0; i < V; ++i) s[i] = sigmoid_f32(x[i]);
    }
    if (a.scores && here) {
      float* o = a.scores + t * E + 4 * l;
      if (vec_out) {
#pragma unroll
        for (int c = 0; c < C; ++c)
          if (4 * (LPT * c + l) < E)
            *reinterpret_cast<float4*>(o + 4 * LPT * c) = make_float4(s[4 * c], s[4 * c + 1], s[4 * c + 2], s[4 * c + 3]);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (4 * (LPT * (i >> 2) + l) + (i & 3) < E) o[4 * LPT * (i >> 2) + (i & 3)] = s[i];
      }
    }
    // fp32 scores are off by less than 2^-19 of the row's largest (softmax: 29
    // roundings of 2^-24 - the exponent's 2.2 |x| e^x < 1, exp, 22 additions,
    // the quotient) or 6 * 2^-24 (sigmoid); two that differ by more than 2^-17
    // of it, or 2^-20, and the roundings of their sums with the bias are in
    // their exact order
    const float err = a.softmax ? 0x1p-17f * smax : 0x1p-20f;
    bool redo = false;
    // v, except that without a bias a choice of logits needs no rounding
    const bool by_score = a.bias || a.group_top == 2;  // of the groups' values
    if (a.bias) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float b[4];
        load4(s_bias + 4 * (LPT * c + l), b);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          x[4 * c + j] = x[4 * c + j] == -INFINITY ? -INFINITY : s[4 * c + j] + b[j];
      }
    }
    if (a.n_group > 1) {
      float* v = reinterpret_cast<float*>(s_mem[wv]) + sub * PITCH;
      const bool of_scores = !a.bias && by_score;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        float y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          y[j] = of_scores && x[4 * c + j] != -INFINITY ? s[4 * c + j] : x[4 * c + j];
        *reinterpret_cast<float4*>(v + 4 * (LPT * c + l)) = make_float4(y[0], y[1], y[2], y[3]);
      }
      __builtin_amdgcn_wave_barrier();
      // the two largest of each group: 2^sh lanes a group, every 2^sh-th of
      // its experts (in fours) each
      const int sh = a.share, g = l >> sh, part = l & ((1 << sh) - 1);
      const float* mine_v = v + (g < a.n_group ? g : 0) * size;
      float t1 = -INFINITY, t2 = -INFINITY;
      auto take = [&](float y) {
        t2 = __builtin_amdgcn_fmed3f(t1, t2, y);  // t2 <= t1: the second largest of the three
        t1 = y > t1 ? y : t1;
      };
      if ((size & 3) == 0) {
        const int n = ((size >> 2) - part + (1 << sh) - 1) >> sh;
        int at = g < n ? g : 0;  // each group begins at a place of its own: other banks
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
          const float4 y = *reinterpret_cast<const float4*>(mine_v + 4 * ((at << sh) + part));
          take(y.x); take(y.y); take(y.z); take(y.w);
          at = at + 1 == n ? 0 : at + 1;
        }
      } else {
#pragma unroll 4
        for (int i = part; i < size; i += 1 << sh) take(mine_v[i]);
      }
      auto meet2 = [&](float y1, float y2) {
        take(y1);
        t2 = y2 > t2 ? y2 : t2;
      };
      if (sh > 0) meet2(partner<0>(t1), partner<0>(t2));
      if (sh > 1) meet2(partner<1>(t1), partner<1>(t2));
      if (sh > 2) meet2(partner<2>(t1), partner<2>(t2));
      constexpr int GL = LPT == 64 ? GMAXG : 16;
      float* gs = reinterpret_cast<float*>(s_g[wv]) + 16 * sub;
      if (part == 0 && g < GL)
        gs[g] = g >= a.n_group ? -INFINITY : a.group_top == 2 && t2 > -INFINITY ? t1 + t2 : t1;
      if (sh > 0 && l < GL && l >= LPT >> sh) gs[l] = -INFINITY;
      __builtin_amdgcn_wave_barrier();
      const float worth = gs[l < GL ? l : 0];
      // the sums' roundings go by their parts, which may cancel: those of the
      // two groups compared are under 2^-22 of the token's largest |t1| + |t2|
      const bool two = a.group_top == 2 && t2 > -INFINITY;
      const float parts = (t1 > -INFINITY ? fabsf(t1) : 0.f) + (two ? fabsf(t2) : 0.f);
      const float near =
          by_score ? 2.f * err + 0x1p-21f * __int_as_float(row_max<LPT>(__float_as_int(parts))) : 0.f;
      int rank = 0, close = 0;
#pragma unroll
      for (int j = 0; j < GL; j += 4) {
        const float4 y4 = *reinterpret_cast<const float4*>(gs + j);
        const float y[4] = {y4.x, y4.y, y4.z, y4.w};
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          rank += (y[h] > worth || (y[h] == worth && j + h < l)) ? 1 : 0;
          close += y[h] < worth - near ? 0 : 1;  // (infinite values: close)
        }
      }
      const bool mine = l < a.n_group && rank < a.topk_group;
      // (without scores equal groups are in their order already)
      redo = by_score && mine && close > a.topk_group;
      const uint32_t kept = (uint32_t)(__ballot(mine) >> (LPT == 64 ? 0 : 16 * sub));
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const uint32_t e = 4 * (LPT * c + l);
        if ((size & 3) == 0) {
          const bool in = (kept >> ((e * a.magic) >> 20)) & 1;
#pragma unroll
          for (int j = 0; j < 4; ++j) x[4 * c + j] = in ? x[4 * c + j] : -INFINITY;
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            x[4 * c + j] = (kept >> (((e + j) * a.magic) >> 20)) & 1 ? x[4 * c + j] : -INFINITY;
        }
      }
    }
    // the k-th largest
    int top[8];
    if (C == 1) {
#pragma unroll
      for (int i = 0; i < 8; ++i) top[i] = i < 4 ? order_key(x[i]) : (int)0x80000000;
      order2(top[0], top[1]); order2(top[2], top[3]); order2(top[0], top[2]);
      order2(top[1], top[3]); order2(top[1], top[2]);
    } else {
#pragma unroll
      for (int h = 0; h < V / 8; ++h) {
        int w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = order_key(x[(8 * h + i) % V]);
        sort8(w);
        if (h == 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) top[i] = w[i];
        } else {
          join8(top, w);
        }
      }
    }
    round8<0>(top);
    round8<1>(top);
    round8<2>(top);
    round8<3>(top);
    if (LPT == 64) {
      round8<4>(top);
      round8<5>(top);
    }
    int kth = top[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) kth = i < k ? top[i] : kth;
    const float thr = from_key(kth);
    const float least = a.bias ? thr - (err + 0x1p-21f * fabsf(thr)) : thr;
    uint32_t mask = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) mask |= x[i] >= least ? 1u << i : 0u;
    int over = row_sum<LPT>((int)__popc(mask)) - k;
    if (!a.bias && __ballot(over > 0)) {
      // equal logits at the border: of them, in the order of the experts
      // (chunk, lane, place), the last `over` go
      uint32_t equal = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) equal |= x[i] == thr ? 1u << i : 0u;
      int room = row_sum<LPT>((int)__popc(equal)) - over;  // that stay
      const bool ties = over > 0 && room > 0 && thr > -INFINITY;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const uint32_t of = (equal >> (4 * c)) & 15u;
        const int n = __popc(of), upto = row_scan<LPT>(n, l);
        int left = room - (upto - n);  // for this lane and those after it
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if ((of >> j) & 1) {
            if (ties && left <= 0) mask &= ~(1u << (4 * c + j));
            --left;
          }
        room -= row_sum<LPT>(n);
      }
      over = row_sum<LPT>((int)__popc(mask)) - k;
    }
    const int mine = __popc(mask);
    redo = redo || over != 0;
    const uint64_t again = __ballot(redo && here);
    const bool clean = here && !((again >> (lane & ~(LPT - 1))) & (LPT == 64 ? ~0ull : 0xFFFFull));
    any |= again;
    // places of this lane's in the token's list: after those of the lanes before
    const int upto = row_scan<LPT>(mine, l);
    if (clean) {
      int pos = upto - mine;
      while (mask) {
        const int i = __ffs(mask) - 1;
        mask &= mask - 1;
        s_ids[wv][sub][pos++] = 4 * (LPT * (i >> 2) + l) + (i & 3);
      }
    }
    __builtin_amdgcn_wave_barrier();
    bool low = false;  // the scores' sum: for the second look
    if (clean && l < 16) {
      float sj = 0.f;
      int id = 0, place = 0;
      if (l < k) {
        id = s_ids[wv][sub][l];
        for (int j = 0; j < k; ++j) place += s_ids[wv][sub][j] < id ? 1 : 0;
        const float lj = load_logit(row + id);
        sj = a.softmax ? exp_from(lj, m) * inv : sigmoid_f32(lj);
      }
      const float sum = row_sum<16>(sj);
      low = a.renorm && sum > 0.f && sum < kLow;
      if (l < k) {
        a.topk_idx[t * k + place] = low && place == 0 ? -1 : id;
        a.topk_w[t * k + place] = a.scale * (a.renorm ? (sum > 0.f ? sj / sum : 0.f) : sj);
        if (ONE && !low) atomicAdd(&s_hist[id], 1);
      }
    } else if (here && l == 0) {
      a.topk_idx[t * k] = -1;  // for the second look
    }
    any |= __ballot(low);
    __builtin_amdgcn_wave_barrier();
  }
  if (any) {
    for (int64_t t0 = first; t0 < a.T; t0 += step) {
      const bool in = lane < TPW && t0 + lane < a.T;
      uint64_t todo = __ballot(in && ((volatile int32_t*)a.topk_idx)[(in ? t0 + lane : 0) * k] == -1);
      for (; todo; todo &= todo - 1)
        gate_token<D, EMAX / 64, ONE>(a, t0 + __ffsll((unsigned long long)todo) - 1,
                                      reinterpret_cast<double*>(s_mem[wv]), s_g[wv], s_hist);
    }
  }
  if (ONE) {
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += GT) a.counts[e] = s_hist[e];
  }
}

// counts[e] = how often e is named in ids (counts are 0 before, unless one
// workgroup does it all).  A launch of its own costs 1 us less than adding up
// in gate_kernel's loop, whose registers and adds take longer (16384 tokens).
// Few workgroups, so that few add to one number; U ids a thread in flight
// (16384 x 8 ids: 2.8 us; one at a time 3.1).
template <int U>
__global__ __launch_bounds__(1024) void gate_count_kernel(const int32_t* __restrict__ ids, int64_t n,
                                                          int E, int32_t* __restrict__ counts) {
  __shared__ int hist[GMAXE];
  for (int e = threadIdx.x; e < E; e += 1024) hist[e] = 0;
  __syncthreads();
  for (int64_t i = (int64_t)blockIdx.x * (1024 * U) + threadIdx.x; i < n; i += (int64_t)gridDim.x * (1024 * U)) {
    int id[U];
#pragma unroll
    for (int u = 0; u < U; ++u) id[u] = i + 1024 * u < n ? ids[i + 1024 * u] : -1;
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (id[u] >= 0) atomicAdd(&hist[id[u]], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += 1024) {
    const int c = hist[e];
    if (gridDim.x == 1) counts[e] = c;
    else if (c) atomicAdd(&counts[e], c);
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
__device__ __forceinline__ void store4(float* p, const float* v) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(uint16_t* p, const float* v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]));
}

// Lanes and slots as in gate_kernel.  Bound by its reads and writes of [T, E]
// (16384 x 256 of fp32 with a dense gradient, 51 MB: 10.2 us, 5.0 TB/s);
// lane j < k of a token has its j-th choice (score from the logit again),
// whose gradient goes into the row of ds (renormalised: of dl) in LDS, each place
// written once: of an id named twice the first lane adds both.
template <typename D, int LPT, int C>
__global__ __launch_bounds__(GT) void gate_backward_kernel(GateBwdArgs a) {
  constexpr int TPW = 64 / LPT, V = 4 * C, EMAX = LPT * V, W = GT / 64;
  __shared__ __attribute__((aligned(16))) float s_row[W][TPW][EMAX + 8];
  __shared__ int s_id[W][TPW][GMAXK];
  __shared__ float s_val[W][TPW][GMAXK];
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  const int l = lane & (LPT - 1), sub = lane / LPT;
  const int E = a.E, k = a.k;
  const int64_t t0 = ((int64_t)blockIdx.x * W + wv) * TPW;
  if (t0 >= a.T) return;
  const bool here = t0 + sub < a.T;
  const int64_t t = here ? t0 + sub : a.T - 1;
  const D* row = static_cast<const D*>(a.logits) + t * E;
  D* out = static_cast<D*>(a.dl) + t * E;
  const bool vec = (E & 3) == 0 && (((uintptr_t)a.logits | (uintptr_t)a.dl) & (4 * sizeof(D) - 1)) == 0 &&
                   ((uintptr_t)a.ds & 15) == 0;
  float s[V], g[V];  // logits, then softmax scores or the sigmoids' slopes; ds, then dl
#pragma unroll
  for (int i = 0; i < V; ++i) g[i] = 0.f;
  if (vec) {
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int e = 4 * (LPT * c + l);
      load4(row + min(e, E - 4), s + 4 * c);
      if (a.ds) load4(a.ds + t * E + min(e, E - 4), g + 4 * c);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[4 * c + j] = e < E ? s[4 * c + j] : -INFINITY;
        g[4 * c + j] = e < E ? g[4 * c + j] : 0.f;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = 4 * (LPT * (i >> 2) + l) + (i & 3);
      const float y = load_logit(row + min(e, E - 1));
      s[i] = e < E ? y : -INFINITY;
      if (a.ds) {
        const float d = a.ds[t * E + min(e, E - 1)];
        g[i] = e < E ? d : 0.f;
      }
    }
  }
  int id = -1;
  float lj = 0.f, dwj = 0.f;
  if (l < k) {
    const int e = a.idx[t * k + l];
    if ((uint32_t)e < (uint32_t)E) {
      id = e;
      lj = load_logit(row + e);
      dwj = a.scale * a.dw[t * k + l];
    }
  }
  float m = 0.f, inv = 0.f;
  if (a.softmax) {
    int mk = order_key(s[0]);
#pragma unroll
    for (int i = 1; i < V; ++i) mk = max(mk, order_key(s[i]));
    m = from_key(row_max<LPT>(mk));
    m = m == -INFINITY ? 0.f : m;
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      s[i] = exp_from(s[i], m);
      z += s[i];
    }
    z = row_sum<LPT>(z);
    inv = z > 0.f ? 1.0f / z : 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] *= inv;
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = sigmoid_slope(s[i]);
  }
  // the choices' gradients (lanes 0..15 of a token; k <= 8).  Renormalised ones,
  // p_j (dw_j - sum_i dw_i p_i) of the shares p, sum to 0 over a token, so they
  // join behind the sum over the row; s_j (..) / S would overflow in 1 / S.
  float val = dwj;
  if (a.renorm) {
    const float pj = share(a.softmax, id < 0 ? -INFINITY : lj, m, inv);
    val = pj * (dwj - row_sum<16>(dwj * pj));
    if (!a.softmax) val *= sigmoid_f32(-lj);
  }
  float* buf = s_row[wv][sub];
  auto add_choices = [&]() __attribute__((always_inline)) {  // to g
#pragma unroll
    for (int c = 0; c < C; ++c)
      *reinterpret_cast<float4*>(buf + 4 * (LPT * c + l)) =
          make_float4(g[4 * c], g[4 * c + 1], g[4 * c + 2], g[4 * c + 3]);
    if (l < k) {
      s_id[wv][sub][l] = id;
      s_val[wv][sub][l] = val;
    }
    __builtin_amdgcn_wave_barrier();
    if (id >= 0) {
      float sum = 0.f;
      bool first = true;
      for (int j = 0; j < k; ++j)
        if (s_id[wv][sub][j] == id) {
          first = first && j >= l;
          sum += s_val[wv][sub][j];
        }
      if (first) buf[id] += sum;
    }
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int c = 0; c < C; ++c) load4(buf + 4 * (LPT * c + l), g + 4 * c);
  };
  if (!a.renorm) add_choices();
  float p = 0.f;
  if (a.softmax) {
#pragma unroll
    for (int i = 0; i < V; ++i) p = fmaf(g[i], s[i], p);
    p = row_sum<LPT>(p);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) g[i] = a.softmax ? s[i] * (g[i] - p) : g[i] * s[i];
  if (a.renorm) add_choices();
  if (!here) return;
  if (vec) {
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (4 * (LPT * c + l) < E) store4(out + 4 * (LPT * c + l), g + 4 * c);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int e = 4 * (LPT * (i >> 2) + l) + (i & 3);
      if (e < E) store_grad(out + e, g[i]);
    }
  }
}

template <typename D, int LPT, int C>
void launch_gate_as(const GateArgs& a, hipStream_t st) {
  const int64_t blocks = std::min<int64_t>(ceil_div(a.T, GT / LPT), 4096);
  if (blocks == 1) {
    gate_kernel<D, LPT, C, true><<<dim3(1), dim3(GT), 0, st>>>(a);
    return;
  }
  gate_kernel<D, LPT, C, false><<<dim3((unsigned)blocks), dim3(GT), 0, st>>>(a);
  const int64_t n = a.T * a.k, parts = ceil_div(n, 1024);
  if (parts <= 32)
    gate_count_kernel<1><<<dim3((unsigned)parts), dim3(1024), 0, st>>>(a.topk_idx, n, a.E, a.counts);
  else
    gate_count_kernel<4><<<dim3(32), dim3(1024), 0, st>>>(a.topk_idx, n, a.E, a.counts);
}

template <typename D>
void launch_gate(const GateArgs& a, hipStream_t st) {
  if (a.E > 512) launch_gate_as<D, 64, 4>(a, st);
  else if (a.E > 256 || a.n_group > 16) launch_gate_as<D, 64, 2>(a, st);
  else if (a.E > 128) launch_gate_as<D, 16, 4>(a, st);
  else if (a.E > 64) launch_gate_as<D, 16, 2>(a, st);
  else launch_gate_as<D, 16, 1>(a, st);
}

template <typename D, int LPT, int C>
void launch_backward_as(const GateBwdArgs& a, hipStream_t st) {
  // a launch holds less than 2^32 threads: runs of 2^25 tokens (offsets that
  // keep every tensor's alignment)
  constexpr int64_t RUN = 1ll << 25;
  for (int64_t t = 0; t < a.T; t += RUN) {
    GateBwdArgs r = a;
    r.T = std::min(RUN, a.T - t);
    r.logits = static_cast<const D*>(a.logits) + t * a.E;
    r.idx += t * a.k;
    r.dw += t * a.k;
    if (a.ds) r.ds += t * a.E;
    r.dl = static_cast<D*>(a.dl) + t * a.E;
    gate_backward_kernel<D, LPT, C><<<dim3((unsigned)ceil_div(r.T, GT / LPT)), dim3(GT), 0, st>>>(r);
  }
}

template <typename D>
void launch_gate_backward(const GateBwdArgs& a, hipStream_t st) {
  if (a.E > 512) launch_backward_as<D, 64, 4>(a, st);
  else if (a.E > 256) launch_backward_as<D, 64, 2>(a, st);
  else if (a.E > 128) launch_backward_as<D, 16, 4>(a, st);
  else if (a.E > 64) launch_backward_as<D, 16, 2>(a, st);
  else launch_backward_as<D, 16, 1>(a, st);
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
    MOE_INVALID(logits != scores, "moe_gate: logits and scores alias");
  }
  if (T == 0) {
    gate_zero_kernel<<<1, GT, 0, st>>>(expert_counts, E);
  } else {
    const int size = E / n_group, lanes = E > 256 || n_group > 16 ? 64 : 16;
    int share = 0;
    while (share < 3 && n_group << (share + 1) <= lanes) ++share;
    const GateArgs a{logits, bias, T, E, n_group, topk_group, group_top, k, size, share,
                     ((1u << 20) + (uint32_t)size - 1) / (uint32_t)size, score == MOE_SCORE_SOFTMAX, renormalize != 0, scale,
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
