/*
 * moe_fp8.h - C ABI of libmoe_fp8.so, the DeepSeekMoE layer forward on
 * MI355X (gfx950).
 *
 * The layer follows the DeepSeek-V3 pages:
 *   - sigmoid gating with a per-expert bias used only to choose experts
 *     (aliyun study note developer.aliyun.com/article/1776647, section 2.2;
 *     news.qq.com/rain/a/20241229A05OQF00, section 无额外损耗的负载均衡);
 *   - 1 shared + 256 routed experts, 8 routed per token, at most 4 nodes per
 *     token (news.qq.com article, sections DeepSeekMoE 架构 and 节点限制路由);
 *   - FP8 GEMMs with 1x128 activation tiles, 128x128 weight blocks and
 *     high-precision accumulation (news.qq.com article, section FP8 低精度训练,
 *     items 细粒度量化 and 提高累加精度).
 *
 * Conventions shared by every call:
 *   - All tensor pointers are DEVICE pointers owned by the caller.  The
 *     library never allocates, frees or keeps a pointer after the call.
 *   - Layouts are row-major and dense unless a leading dimension is given.
 *     "bf16" buffers hold raw bfloat16 bit patterns (uint16).  "e4m3" buffers
 *     hold OCP E4M3FN bytes.  Scales are fp32.
 *   - `stream` is a hipStream_t passed as void* (NULL = the default stream).
 *     Work is enqueued asynchronously on it; the caller keeps every buffer
 *     alive until the stream has finished.  No call synchronises the host.
 *   - Arguments are validated on the host before anything is launched.  On
 *     error nothing is launched, the return value is negative and
 *     moe_last_error() describes it.  Faults inside kernels surface at the
 *     caller's next synchronisation, as for any HIP kernel.
 *   - Outputs are fully overwritten, never accumulated into.  Inputs and
 *     outputs must not alias (except where a call says "in place").
 *   - A zero-sized problem (T == 0, M_total == 0) is a successful no-op that
 *     still writes the outputs that do not depend on it (counts, offsets).
 *   - Calls with group_offsets take at most M_total = 2^31 - 256 rows.
 *   - NaN or Inf inputs give unspecified results.
 */
#ifndef MOE_FP8_H
#define MOE_FP8_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Return codes. */
#define MOE_OK               0
#define MOE_ERR_INVALID     -1  /* null pointer, bad shape or parameter      */
#define MOE_ERR_UNSUPPORTED -2  /* valid but outside what the kernels handle */
#define MOE_ERR_HIP         -3  /* a HIP launch or API call failed            */
#define MOE_ERR_WORKSPACE   -4  /* workspace too small                        */

/* Element types and score functions of the gate (moe_gate). */
#define MOE_TYPE_F32         0
#define MOE_TYPE_BF16        1
#define MOE_SCORE_SOFTMAX    0
#define MOE_SCORE_SIGMOID    1

/* Activations of the gated feed-forward products (grouped_bf16_gemm_glu):
 * act(g) = g / (1 + exp(-z)), z = g (SiLU) or 2 sqrt(2/pi) (g + 0.044715 g^3)
 * (the tanh form of GELU). */
#define MOE_ACT_SILU         0
#define MOE_ACT_GELU         1

/* Codes that moe_norm writes beside the normed rows. */
#define MOE_QUANT_NONE       0
#define MOE_QUANT_E4M3       1   /* 1x128 tiles, as fp8_quant_1x128 */
#define MOE_QUANT_INT8       2   /* one scale a row, as int8_quant_rows */

/* Message of the last failed call on this thread ("" if none). */
const char* moe_last_error(void);

/* Library version string. */
const char* moe_version(void);

/*
 * moe_route - router: sigmoid scores, selection bias, group-limited top-k.
 *
 * Follows the aliyun study note, section 2.2 (sigmoid gate per expert, a bias
 * per expert that shifts only the choice), and the news.qq.com article,
 * sections DeepSeekMoE 架构 (top-8 of 256) and 节点限制路由 (at most 4 nodes;
 * here: groups).  Gating stays in high precision (same article,
 * 选择性高精度): logits are computed with fp32 accumulation of exact
 * products (bf16 x times a three-piece bf16 split of the fp32 centroids).
 *
 * For each token t:
 *   l[e]  = sum_h x[t,h] * centroids[e,h]
 *   s[e]  = 1 / (1 + exp(-l[e]))               (fp32)
 *   s'[e] = s[e] + bias[e]                     (fp32, used to choose only)
 *   experts form n_group contiguous groups of E/n_group; a group's score is
 *   the sum of its two largest s'; the topk_group best groups are kept; the
 *   k largest s' among the kept experts are chosen; ties go to the lower
 *   index; ids are written in ascending order;
 *   w[j]  = s[e_j] / sum_j' s[e_j']            (unbiased scores, fp32)
 *   expert_counts[e] = number of tokens that chose e (overwritten).
 *
 * x_bf16          [T, H] bf16
 * centroids       [E, H] fp32
 * bias            [E] fp32
 * topk_idx  (out) [T, k] int32, ascending per row
 * topk_w    (out) [T, k] fp32, each row sums to 1
 * expert_counts (out) [E] int32
 * workspace       device scratch of at least moe_route_workspace_bytes(T, H, E)
 *                 bytes (partial logits); contents on entry are ignored.
 * topk_s    (out, optional: NULL skips it) [T, k] fp32, 4-byte aligned: the
 *                 unbiased scores s[e_j] of the chosen experts (w[j] times
 *                 their sum), which moe_router_backward can take instead of
 *                 computing the logits again.
 * Requirements: H % 128 == 0; 2 <= E <= 256; E % n_group == 0; the group
 * size E/n_group is 4 times a power of two (4 .. 256); 1 <= topk_group <=
 * n_group; 1 <= k <= 8; k <= topk_group * E / n_group.
 */
size_t moe_route_workspace_bytes(int64_t T, int64_t H, int32_t E);
int moe_route(const void* x_bf16, int64_t T, int64_t H,
              const float* centroids, const float* bias,
              int32_t E, int32_t n_group, int32_t topk_group, int32_t k,
              int32_t* topk_idx, float* topk_w, int32_t* expert_counts,
              void* workspace, size_t workspace_bytes, float* topk_s, void* stream);

/*
 * moe_route_scores - moe_route that also writes what the sequence-wise
 * balance statistic reads: scores [T, E] fp32, the unbiased sigmoid score of
 * every routed expert for every token (16-byte aligned), and score_sums [T]
 * fp32, their sum per token.  Same arguments, requirements, workspace and
 * results as moe_route otherwise.
 */
int moe_route_scores(const void* x_bf16, int64_t T, int64_t H,
                     const float* centroids, const float* bias,
                     int32_t E, int32_t n_group, int32_t topk_group, int32_t k,
                     int32_t* topk_idx, float* topk_w, int32_t* expert_counts,
                     void* workspace, size_t workspace_bytes, float* scores,
                     float* score_sums, float* topk_s, void* stream);

/*
 * moe_seq_balance - sequence-wise balance statistic (news.qq.com article,
 * section 无额外损耗的负载均衡: factor alpha = 0.0001; the V3 summary at
 * m.jxzklqfsx.com/aigc/3586.html, section （二）無輔助損失負載均衡策略革新: a
 * sequence-level term against imbalance inside one sequence).  The pages
 * give no formula; computed here, for each sequence b of L_b consecutive
 * tokens (runs of seq_len, the last may be shorter):
 *   P[b, e] = (1/L_b) sum_t scores[t, e] / score_sums[t]
 *   f[b, e] = E * (tokens of b that chose e) / (k * L_b)
 *   loss[b] = alpha * sum_e f[b, e] * P[b, e]
 * in fp32 with fixed summation order (f is exact up to one rounding).
 * scores, score_sums: moe_route_scores' outputs; topk_idx [T, k];
 * f_out, p_out (out) [B, E]; loss_out (out) [B], B = ceil(T / seq_len).
 * workspace: moe_seq_balance_workspace_bytes(T, E, seq_len) bytes.
 * Requirements: 1 <= E <= 256, 1 <= k <= E, 1 <= seq_len <= 65536.
 */
size_t moe_seq_balance_workspace_bytes(int64_t T, int32_t E, int64_t seq_len);
int moe_seq_balance(const float* scores, const float* score_sums, const int32_t* topk_idx,
                    int64_t T, int32_t E, int32_t k, int64_t seq_len, float alpha,
                    float* f_out, float* p_out, float* loss_out, void* workspace,
                    size_t workspace_bytes, void* stream);

/*
 * moe_bias_update - aux-loss-free balancing step, in place.
 *
 * aliyun study note section 2.2 (overloaded experts' bias goes down,
 * underloaded goes up, no loss term) and news.qq.com article section
 * 无额外损耗的负载均衡 (update speed gamma = 0.001).  With total = sum_e
 * counts[e]: bias[e] -= gamma if counts[e]*E > total; bias[e] += gamma if
 * counts[e]*E < total; unchanged otherwise.  fp32 arithmetic; integer test.
 *
 * expert_counts [E] int32 (e.g. the output of moe_route for this batch)
 * bias          [E] fp32, updated in place
 * Requirements: 1 <= E <= 1024.
 */
int moe_bias_update(const int32_t* expert_counts, float* bias, int32_t E,
                    float gamma, void* stream);

/*
 * moe_permute - dispatch: expert-contiguous order of the token-expert
 * assignments (the all-to-all dispatch of the news.qq.com article, section
 * DualPipe 流水线并行, done inside one GPU).
 *
 * Rows of expert e are the assignments (t, j) with topk_idx[t,j] == e in
 * ascending (t, j) order; the n_shared shared expert(s) follow, one block of
 * T rows each in token order.  R = T*k + n_shared*T.
 *
 * topk_idx       [T, k] int32, values in [0, E)
 * expert_counts  [E] int32, the histogram of topk_idx (as moe_route writes)
 * offsets  (out) [E + n_shared + 1] int32: exclusive prefix sum of group sizes
 * perm_src (out) [R] int32: token of each row
 * inv_perm (out) [T*k] int32: row of assignment (t, j) at t*k + j
 * xq, xs         optional [T, H] e4m3 and [T, H/128] fp32; when a_out is not
 *                NULL, a_out[r] = xq[perm_src[r]] and a_scale_out[r] =
 *                xs[perm_src[r]] ([R, H] e4m3, [R, H/128] fp32).
 * workspace      at least moe_permute_workspace_bytes(T, k, E) bytes.
 * Requirements: 1 <= k <= 8; 1 <= E <= 4096; n_shared in {0, 1};
 * H % 128 == 0 when gathering.  topk_idx and expert_counts must be consistent.
 */
size_t moe_permute_workspace_bytes(int64_t T, int32_t k, int32_t E);
int moe_permute(const int32_t* topk_idx, const int32_t* expert_counts,
                int64_t T, int32_t k, int32_t E, int32_t n_shared,
                int32_t* offsets, int32_t* perm_src, int32_t* inv_perm,
                const uint8_t* xq, const float* xs, int64_t H,
                uint8_t* a_out, float* a_scale_out,
                void* workspace, size_t workspace_bytes, void* stream);

/*
 * moe_permute_noalloc - moe_permute for callers that cannot allocate device
 * memory: code under HIP graph capture, tight serving loops, harnesses that
 * forbid hipMalloc.  Same arguments, outputs and errors as moe_permute minus
 * the workspace: the per-chunk histograms live in a static device array of
 * MOE_PERMUTE_SCRATCH_BYTES bytes that the library keeps on every GPU it
 * runs on until the process ends (its address is looked up once per device,
 * on the first call with that device current).  The call allocates nothing.
 * Its scratch need is moe_permute_workspace_bytes(T, k, E); a larger need
 * (ceil(T/64) * E > 262144, e.g. T > 65536 at E = 256) returns
 * MOE_ERR_WORKSPACE without launching.  Every call on one GPU shares that
 * GPU's array: calls that overlap on one GPU (different streams, or host
 * threads without ordering) race; calls ordered on one stream do not.
 */
#define MOE_PERMUTE_SCRATCH_BYTES ((size_t)1 << 20)
int moe_permute_noalloc(const int32_t* topk_idx, const int32_t* expert_counts,
                        int64_t T, int32_t k, int32_t E, int32_t n_shared,
                        int32_t* offsets, int32_t* perm_src, int32_t* inv_perm,
                        const uint8_t* xq, const float* xs, int64_t H,
                        uint8_t* a_out, float* a_scale_out, void* stream);

/*
 * fp8_quant_1x128 - fine-grained activation quantisation (news.qq.com
 * article, section FP8 低精度训练 › 细粒度量化: 1x128 tiles for activations).
 *
 * For each row m and 128-column tile j of the output:
 *   v     = mode 0: in[m, j*128 + c]
 *           mode 1: silu(g) * u with g = in[m, j*128 + c], u = in[m, K + j*128 + c]
 *                   evaluated in fp32 as a = g / (1 + exp(-g)); v = a * u
 *   amax  = max_c |v|;  s = amax / 448 (fp32), or 1 if amax == 0
 *   out   = E4M3FN(v / s): correctly rounded fp32 division, round to nearest
 *           even, saturate to +-448, sign of zero kept
 *   scales[m, j] = s
 *
 * in_bf16  [M, ld_in] bf16; mode 0 needs ld_in >= K, mode 1 needs ld_in >= 2K
 * out_e4m3 [M, K] e4m3;  scales [M, K/128] fp32
 * Requirements: K % 128 == 0, ld_in % 8 == 0, mode in {0, 1}.
 */
int fp8_quant_1x128(const void* in_bf16, int64_t M, int64_t K, int64_t ld_in,
                    int32_t mode, uint8_t* out_e4m3, float* scales, void* stream);

/*
 * fp8_quant_128x128 - weight quantisation in 128x128 blocks (aliyun study
 * note section 4.1; news.qq.com article section 细粒度量化).  Same scale and
 * rounding rule as fp8_quant_1x128, with amax taken over each block.
 *
 * w_f32    [G, N, K] fp32;  out_e4m3 [G, N, K];  scales [G, N/128, K/128]
 * Requirements: N % 128 == 0, K % 128 == 0.
 */
int fp8_quant_128x128(const float* w_f32, int64_t G, int64_t N, int64_t K,
                      uint8_t* out_e4m3, float* scales, void* stream);

/*
 * fp8_transpose_128x128 - weights in 128x128 blocks, transposed block by block
 * (news.qq.com article, section FP8 低精度训练 › 细粒度量化: 128x128 weight
 * blocks; section 工程 › DualPipe 流水线并行: the pipeline's backward-for-input
 * chunks).  The expert GEMM C = A W^T has the input gradient dA = dY W, a
 * contraction over n: grouped_fp8_gemm computes it with dY quantised by
 * fp8_quant_1x128 and B = W^T from this call (N' = K, K' = N).
 *
 *   wt[g, k, n] = w[g, n, k];   wt_scale[g, kb, nb] = w_scale[g, nb, kb]
 *
 * Codes and scales move unchanged, so the output is exactly the 128x128
 * quantisation of W^T.
 * w_e4m3   [G, N, K] e4m3 (16-byte aligned);  w_scale [G, N/128, K/128] fp32
 * wt_e4m3  (out) [G, K, N] e4m3;  wt_scale (out) [G, K/128, N/128] fp32
 * Requirements: N % 128 == 0, K % 128 == 0, 0 <= G <= 65535, outputs not
 * aliasing inputs.  G == 0 is a no-op.
 */
int fp8_transpose_128x128(const uint8_t* w_e4m3, const float* w_scale, int64_t G,
                          int64_t N, int64_t K, uint8_t* wt_e4m3, float* wt_scale,
                          void* stream);

/*
 * fp8_quant_128x1_grouped - the weight-gradient operands: per-group FP8
 * quantisation in 128x1 tiles along the token axis (news.qq.com article,
 * section FP8 低精度训练 › 细粒度量化 gives 1x128 activation tiles; the
 * weight gradient contracts over tokens, so the tile is taken along them - a
 * reading, the pages give no backward orientation; section 工程 › DualPipe
 * 流水线并行 names the backward-for-weights chunks).
 *
 * Group g (rows group_offsets[g] .. group_offsets[g+1]) is cut into 128-row
 * chunks from its first row, the last one padded with zeros; chunk c of the
 * layout is the c-th in group order (group g's chunks start at the sum over
 * g' < g of ceil(rows_g' / 128)).  Stored chunk-major: for column j and
 * chunk c,
 *   s = amax over the chunk's rows of |in[r, j]| / 448 (1 if 0)
 *   out_c[c, j, i]  = E4M3(in[row i of chunk c, j] / s)  (0 for padding)
 *   scales_c[c, j]  = s
 * with the rounding of fp8_quant_1x128.  (out_c[c] transposed is the 128
 * tokens of chunk c as rows: a tile's chunk is one contiguous block.)
 *
 * in_bf16   [in_rows, ld_in] bf16 (C columns used; 16-byte aligned, ld_in % 8 == 0)
 * row_index [M_total] int32 or NULL: layout row r reads input row row_index[r]
 *           (an entry outside [0, in_rows) reads row in_rows - 1), else row r
 * in_rows   rows of in_bf16: >= M_total without a row index, >= 1 with one
 * group_offsets [G+1] int32 on the device, as in grouped_fp8_gemm
 * out_c     (out) [chunks_cap, C, 128] e4m3 (16-byte aligned)
 * scales_c  (out) [chunks_cap, C] fp32
 * chunks_cap >= ceil(M_total / 128) + G (chunks past the last are not written)
 * Requirements: 1 <= G <= 1024, C % 128 == 0, ld_in >= C.
 */
int fp8_quant_128x1_grouped(const void* in_bf16, int64_t ld_in, const int32_t* row_index,
                            int64_t in_rows, const int32_t* group_offsets, int32_t G,
                            int64_t M_total, int64_t C, uint8_t* out_c, float* scales_c,
                            int64_t chunks_cap, void* stream);

/*
 * grouped_fp8_wgrad - weight gradient of the expert GEMMs (news.qq.com article,
 * section 工程 › DualPipe 流水线并行: backward-for-weights chunks; section FP8
 * 低精度训练: FP8 products accumulated in FP32 at a fixed K interval).
 *
 * For the forward C_g = A_g W_g^T (W_g [N, K]) and the output gradient dY,
 *   dW[g, n, k] = sum_{c in group g's chunks}  dy_scale_c[c, n] * a_scale_c[c, k]
 *                 * sum_{i<128} dy_c[c, n, i] * a_c[c, k, i]
 * with dy_c / a_c from fp8_quant_128x1_grouped of dY [M_total, N] and
 * A [M_total, K] on the same group_offsets.  Each chunk's 128-term FP8
 * partial is an FP32 MFMA sum added to one FP32 accumulator kept in units of
 * the current chunk's scale product (rescaled by the ratio of consecutive
 * chunks' scales, multiplied by the last one at the end).  A group without
 * rows gets dW[g] = 0.
 *
 * dy_c [chunks_cap, N, 128], dy_scale_c [chunks_cap, N];
 * a_c  [chunks_cap, K, 128], a_scale_c  [chunks_cap, K]
 * dW   (out) [G, N, K] fp32 (overwritten)
 * Requirements: N % 128 == 0, K % 128 == 0, 1 <= G <= 65535,
 * chunks_cap >= ceil(M_total / 128) + G; operands and dW 16-byte, scales
 * 4-byte aligned.
 */
int grouped_fp8_wgrad(const uint8_t* dy_c, const float* dy_scale_c, const uint8_t* a_c,
                      const float* a_scale_c, int64_t chunks_cap, const int32_t* group_offsets,
                      int32_t G, int64_t M_total, int64_t N, int64_t K, float* dW,
                      void* stream);

/*
 * moe_combine_backward - backward of moe_combine (news.qq.com article, section
 * DeepSeekMoE 架构: gate-weighted routed experts plus the always-on shared
 * one; section 工程 › DualPipe 流水线并行: the backward-for-input chunks).
 *
 * For the forward y[t] = sum_j w[t,j] D[inv_perm[t*k+j]] + D[T*k + t]:
 *   dD[inv_perm[t*k+j], :] = bf16( w[t,j] * dy[t, :] )   (fp32 product)
 *   dD[T*k + t, :]         = dy[t, :]                      (n_shared == 1)
 *   dw[t*k + j]            = sum_h dy[t, h] * D[inv_perm[t*k+j], h]  (fp32,
 *                            summed in a fixed order)
 * dy_bf16 [T, H]; inv_perm [T*k] (a permutation of [0, T*k)); topk_w [T*k];
 * expert_out_bf16 D [T*k + n_shared*T, H]; d_expert_out_bf16 (out) like D;
 * d_topk_w (out) [T*k] fp32.
 * d_expert_out_e4m3, d_expert_out_scale (out, both or neither; NULL: not
 * written) [T*k + n_shared*T, H] e4m3 and [.., H/128] fp32: the 1x128
 * quantisation of dD as stored (bit for bit what fp8_quant_1x128 mode 0
 * writes for d_expert_out_bf16), formed in the same pass so the input-
 * gradient GEMM's operand needs no second read of dD (section FP8 低精度训练
 * › 细粒度量化); requires H % 128 == 0, codes 8-byte and scales 4-byte aligned.
 * Requirements: 1 <= k <= 8, H % 8 == 0, n_shared in {0, 1}; dy, D, dD
 * 16-byte aligned, dD not aliasing D.
 */
int moe_combine_backward(const void* dy_bf16, const int32_t* inv_perm, const float* topk_w,
                         const void* expert_out_bf16, int64_t T, int32_t k, int64_t H,
                         int32_t n_shared, void* d_expert_out_bf16, float* d_topk_w,
                         uint8_t* d_expert_out_e4m3, float* d_expert_out_scale, void* stream);

/*
 * swiglu_backward - backward of h = silu(g) * u (the experts' SwiGLU, see
 * grouped_fp8_gemm_swiglu) from the bf16 gate/up outputs, in fp32:
 *   s = 1 / (1 + exp(-g));  dg = dh * u * s * (1 + g * (1 - s));  du = dh * g * s;
 *   h = g * s * u
 * gu_bf16 [M, 2I] = [g | u]; dh_bf16 [M, I]; dgu_bf16 (out) [M, 2I] = [dg | du];
 * h_bf16 (out) [M, I] (the down projection's weight-gradient operand); all
 * stored as bf16 (round to nearest even), 16-byte aligned.  I % 8 == 0.
 * dgu_e4m3, dgu_scale (out, both or neither; NULL: not written) [M, 2I] e4m3
 * and [M, 2I/128] fp32: the 1x128 quantisation of dGU as stored (bit for
 * bit what fp8_quant_1x128 mode 0 writes for dgu_bf16), in the same pass;
 * requires I % 128 == 0, codes 8-byte and scales 4-byte aligned.
 */
int swiglu_backward(const void* gu_bf16, const void* dh_bf16, int64_t M, int64_t I,
                    void* dgu_bf16, void* h_bf16, uint8_t* dgu_e4m3, float* dgu_scale,
                    void* stream);

/*
 * swiglu_backward_grouped - swiglu_backward over the rows of G groups (the
 * experts' permuted rows) that also writes the FP8 operands the backward's
 * GEMMs read, from the stored bf16 values, in the same pass (news.qq.com
 * article, section FP8 低精度训练 › 细粒度量化; section 工程 › DualPipe
 * 流水线并行: backward-for-input and backward-for-weights chunks):
 *   dgu_bf16, h_bf16 (out, optional: both NULL to skip them): as
 *     swiglu_backward, bit for bit (the codes below do not depend on them);
 *   dgu_e4m3 [M_total, 2I], dgu_scale [M_total, 2I/128] (out): what
 *     fp8_quant_1x128 mode 0 writes for dgu_bf16;
 *   dgu_c, dgu_scale_c (out, C = 2I) and h_c, h_scale_c (out, C = I): what
 *     fp8_quant_128x1_grouped writes for dgu_bf16 and h_bf16 with the same
 *     group_offsets and chunks_cap (chunk-major, zero-padded chunks).
 * gu_bf16 [M_total, 2I] = [g | u]; dh_bf16 [M_total, I]; group_offsets [G+1]
 * int32 on the device (non-decreasing, [0] == 0, [G] == M_total).
 * Requirements: I % 128 == 0, 1 <= G <= 1024, chunks_cap >= ceil(M_total/128)
 * + G; tensors and codes 16-byte aligned, scales 4-byte aligned.  M_total ==
 * 0 is a no-op.
 */
int swiglu_backward_grouped(const void* gu_bf16, const void* dh_bf16,
                            const int32_t* group_offsets, int32_t G, int64_t M_total, int64_t I,
                            void* dgu_bf16, void* h_bf16, uint8_t* dgu_e4m3, float* dgu_scale,
                            int64_t chunks_cap, uint8_t* dgu_c, float* dgu_scale_c, uint8_t* h_c,
                            float* h_scale_c, void* stream);

/*
 * moe_router_backward - backward of the gate weights to the router's input and
 * the per-expert logits (news.qq.com article: section 无额外损耗的负载均衡 - the
 * bias only selects, so neither it nor the choice of experts has a gradient;
 * section FP8 低精度训练 - the gating stays in FP32).
 *
 * For token t with selected experts e_j = topk_idx[t, j] and the unbiased
 * scores s_j = sigmoid(x[t] . C[e_j]) - the forward's (topk_s as moe_route
 * wrote it), or recomputed here in fp32 when topk_s is NULL - (S = sum_j
 * s_j in slot order, w_j = s_j / S, the forward's gate weights):
 *   dlogit_j = (dw_j - sum_i dw_i w_i) / S * s_j * (1 - s_j)
 *   dx_out[t, :] = bf16( dx_in[t, :] + sum_j dlogit_j * C[e_j, :] )   (fp32 sums)
 *   dlogit_rows[inv_perm[t*k + j]] = dlogit_j   (expert-row order, for the
 *                                                centroid gradient)
 * x_bf16 [T, H]; centroids [E, H] fp32; topk_idx, d_topk_w, inv_perm [T*k];
 * dx_in_bf16 [T, H] or NULL (then 0); dx_out_bf16 (out) [T, H] (may equal
 * dx_in); dlogit_rows (out) [T*k] fp32.  Requirements: 1 <= k <= 8, k <= E,
 * H % 8 == 0; x, centroids, dx_in, dx_out 16-byte aligned.  Expert ids
 * outside [0, E) read centroid E - 1 and inv_perm rows outside [0, T*k) are
 * not written (neither occurs for moe_route / moe_permute outputs).
 */
int moe_router_backward(const void* x_bf16, const float* centroids, const int32_t* topk_idx,
                        const float* d_topk_w, const int32_t* inv_perm, const void* dx_in_bf16,
                        int64_t T, int64_t H, int32_t E, int32_t k, void* dx_out_bf16,
                        float* dlogit_rows, const float* topk_s, void* stream);

/*
 * moe_router_dcentroids - gradient of the router centroids (same sections):
 *   dC[e, :] = sum over rows r in [group_offsets[e], group_offsets[e+1]) of
 *              dlogit_rows[r] * x[perm_src[r], :]
 * summed in fp32 in row order (the rows of expert e are its tokens in
 * ascending order, as moe_permute lays them out).
 * x_bf16 [T, H]; perm_src, dlogit_rows: moe_permute's / moe_router_backward's;
 * group_offsets [E+1] (the routed part of moe_permute's offsets, on the device);
 * d_centroids (out) [E, H] fp32.  Requirements: H % 8 == 0, 1 <= E <= 65535;
 * x and d_centroids 16-byte aligned.  T = 0 writes d_centroids = 0 (the other
 * pointers may then be NULL).  perm_src entries outside [0, T) read token
 * T - 1; group_offsets must be moe_permute's.
 */
int moe_router_dcentroids(const void* x_bf16, const int32_t* perm_src,
                          const int32_t* group_offsets, const float* dlogit_rows, int64_t T,
                          int64_t H, int32_t E, float* d_centroids, void* stream);

/*
 * moe_router_backward_dense - the router's backward when the loss also holds
 * the sequence-wise balance term alpha * sum_b L_bal,b of moe_seq_balance
 * (news.qq.com article, section 无额外损耗的负载均衡: the bias only selects,
 * alpha = 0.0001; section FP8 低精度训练: gating in FP32; the V3 summary at
 * m.jxzklqfsx.com/aigc/3586.html, section （二）無輔助損失負載均衡策略革新).
 * With the selection (and so f) held fixed, for token t of sequence b
 * (L_b tokens), s = scores[t, :], S = score_sums[t]:
 *   dlogit[t, e] = alpha / L_b * (f[b, e] - sum_i f[b, i] s_i / S) / S
 *                  * s_e (1 - s_e)
 *                + on each chosen expert e_j: (dw_j - sum_i dw_i w_i) / S_sel
 *                  * s_j (1 - s_j), S_sel = sum_j s_{e_j}, w_j = s_{e_j} / S_sel
 *   dx_out[t, :]  = bf16(dx_in[t, :] + sum_e dlogit[t, e] C[e, :])  (fp32 sums)
 *   d_centroids[e, :] = sum_t dlogit[t, e] x[t, :]  (fp32, tokens in slices of
 *                       ~1024 summed in order, then the slices in order)
 * x_bf16 [T, H]; centroids [E, H] fp32; topk_idx, d_topk_w [T, k]; scores,
 * score_sums: moe_route_scores' outputs of the forward; seq_f [B, E]:
 * moe_seq_balance's f for the same seq_len; dx_in_bf16 [T, H] or NULL (0),
 * must not alias dx_out; dx_out_bf16 (out) [T, H]; d_centroids (out) [E, H];
 * dlogit (out) [T, E] fp32.  workspace:
 * moe_router_backward_dense_workspace_bytes(T, H, E) bytes (0: none needed).
 * Requirements: E % 16 == 0, 16 <= E <= 256, 1 <= k <= 8, H % 128 == 0,
 * 1 <= seq_len <= 65536; x, centroids, scores, seq_f, dx_in, dx_out,
 * d_centroids, dlogit 16-byte aligned.  T = 0 writes d_centroids = 0.
 * Expert ids outside [0, E) count as expert E - 1.
 */
size_t moe_router_backward_dense_workspace_bytes(int64_t T, int64_t H, int32_t E);
int moe_router_backward_dense(const void* x_bf16, const float* centroids,
                              const int32_t* topk_idx, const float* d_topk_w,
                              const float* scores, const float* score_sums, const float* seq_f,
                              int64_t T, int64_t H, int32_t E, int32_t k, int64_t seq_len,
                              float alpha, const void* dx_in_bf16, void* dx_out_bf16,
                              float* d_centroids, float* dlogit, void* workspace,
                              size_t workspace_bytes, void* stream);

/*
 * grouped_fp8_gemm - block-scaled FP8 grouped GEMM with FP32 accumulation
 * (news.qq.com article, section FP8 低精度训练, items 细粒度量化 and
 * 提高累加精度).
 *
 * For group g, rows r in [group_offsets[g], group_offsets[g+1]):
 *   C[r, n] = bf16( sum_kb  sa[r, kb] * B_scale[g, n/128, kb]
 *                           * sum_{k in block kb} a[r, k] * B[g, n, k] )
 * where a[r, :] = A[src(r), :], sa[r, :] = A_scale[src(r), :], and
 * src(r) = a_row_index[r] if a_row_index is not NULL, else r.  Each 128-wide
 * K block is one FP8 MFMA partial in FP32 that is scaled and added to an FP32
 * total; the total is rounded to bf16 (nearest even) once.
 *
 * A        [A_rows, K] e4m3
 * A_scale  [A_rows, K/128] fp32
 * a_row_index  [M_total] int32 or NULL; entries should lie in [0, A_rows):
 *          an entry outside it reads row A_rows - 1 (never memory past A)
 * A_rows   rows of A and A_scale: >= M_total when a_row_index is NULL, >= 1
 *          otherwise
 * B        [G, N, K] e4m3 (each group's matrix stored N x K, K contiguous)
 * B_scale  [G, N/128, K/128] fp32
 * group_offsets [G+1] int32 on the device, non-decreasing, [0] == 0,
 *          [G] == M_total (read by the kernels, never by the host)
 * C  (out) [M_total, N] bf16
 * Requirements: N % 128 == 0, K % 128 == 0, G >= 1 (more than 1024 groups returns
 * MOE_ERR_UNSUPPORTED).
 */
int grouped_fp8_gemm(const uint8_t* A, const float* A_scale, const int32_t* a_row_index,
                     int64_t A_rows, const uint8_t* B, const float* B_scale,
                     const int32_t* group_offsets, int32_t G, int64_t M_total,
                     int64_t N, int64_t K, void* C_bf16, void* stream);

/*
 * grouped_fp8_gemm_dgrad - the input gradient of grouped_fp8_gemm, read
 * from the weights in their forward layout (news.qq.com article, section
 * FP8 低精度训练 › 细粒度量化: 1x128 activation tiles, 128x128 weight blocks;
 * section 工程 › DualPipe 流水线并行: the backward-for-input chunks).  For
 * the forward C = A W^T of group g (W [N, K]), the gradient is dA = dC W, a
 * contraction over n:
 *   dA[r, k] = bf16( sum_nb  sdc[r, nb] * W_scale[g, nb, k/128]
 *                            * sum_{n in block nb} dC[r, n] * W[g, n, k] )
 * with dC quantised by fp8_quant_1x128 along n.  Each 128-wide n block is one
 * FP8 MFMA partial in FP32, as in grouped_fp8_gemm, whose result this equals
 * bit for bit when given B = the fp8_transpose_128x128 of W; no transposed
 * copy is made (the kernel forms its operand with LDS transpose reads).
 *
 * dC       [M_total, N] e4m3;  dC_scale [M_total, N/128] fp32
 * W        [G, N, K] e4m3, W_scale [G, N/128, K/128] fp32: the forward B
 * group_offsets [G+1] int32 on the device, as in grouped_fp8_gemm
 * dA (out) [M_total, K] bf16
 * Requirements: N % 128 == 0, K % 128 == 0, G >= 1 (more than 1024 groups
 * returns MOE_ERR_UNSUPPORTED).
 */
int grouped_fp8_gemm_dgrad(const uint8_t* dC, const float* dC_scale, const uint8_t* W,
                           const float* W_scale, const int32_t* group_offsets, int32_t G,
                           int64_t M_total, int64_t N, int64_t K, void* dA_bf16, void* stream);

/*
 * grouped_fp8_gemm_swiglu - the gate+up GEMM of the experts with SwiGLU and
 * 1x128 requantisation fused into its epilogue (news.qq.com article, section
 * FP8 低精度训练: FP8 GEMM with fine-grained scales and FP32 accumulation,
 * activations kept in FP8; the SwiGLU form is this layer's expert FFN).
 *
 * B holds each group's fused weight [2I, K]: rows [0, I) gate, [I, 2I) up.
 * For row r of group g and column c < I, with the FP32 totals
 *   gt = sum_kb sa[r,kb] * B_scale[g, c/128, kb]     * sum_k a[r,k] B[g, c, k]
 *   ut = sum_kb sa[r,kb] * B_scale[g, (I+c)/128, kb] * sum_k a[r,k] B[g, I+c, k]
 * (accumulated as in grouped_fp8_gemm but never rounded to bf16 or stored):
 *   h = (gt / (1 + exp(-gt))) * ut  in fp32, then per 128 columns of h
 *   s = amax/448 (1 if 0), H_e4m3[r, c] = E4M3(h / s), H_scale[r, c/128] = s.
 *
 * A, A_scale, a_row_index, A_rows, B_scale, group_offsets: as grouped_fp8_gemm with
 * N = 2I.  H_e4m3 (out) [M_total, I] e4m3; H_scale (out) [M_total, I/128].
 * Requirements: I % 128 == 0, K % 128 == 0, 1 <= G <= 1024.
 */
int grouped_fp8_gemm_swiglu(const uint8_t* A, const float* A_scale,
                            const int32_t* a_row_index, int64_t A_rows, const uint8_t* B,
                            const float* B_scale, const int32_t* group_offsets,
                            int32_t G, int64_t M_total, int64_t I, int64_t K,
                            uint8_t* H_e4m3, float* H_scale, void* stream);

/*
 * grouped_fp8_gemm_swiglu_keep - grouped_fp8_gemm_swiglu that also writes
 * the gate/up totals as bf16 (round to nearest even): GU_bf16 [M_total, 2I]
 * = [gt | ut], the bits grouped_fp8_gemm would write for the same operands.
 * For training: the backward's SwiGLU step reads them instead of running the
 * gate+up GEMM again (the pages' FP8 training keeps the FP8 GEMMs; keeping
 * rather than recomputing these outputs is this library's choice, with the
 * HBM to hold them).  Same arguments, requirements and H outputs as
 * grouped_fp8_gemm_swiglu; GU_bf16 16-byte aligned.  Groups below the fused
 * 256-row kernel's size run the fused kernel and grouped_fp8_gemm in turn.
 */
int grouped_fp8_gemm_swiglu_keep(const uint8_t* A, const float* A_scale,
                                 const int32_t* a_row_index, int64_t A_rows, const uint8_t* B,
                                 const float* B_scale, const int32_t* group_offsets,
                                 int32_t G, int64_t M_total, int64_t I, int64_t K,
                                 uint8_t* H_e4m3, float* H_scale, void* GU_bf16, void* stream);

/*
 * moe_combine - weighted combine plus shared expert (news.qq.com article,
 * section DeepSeekMoE 架构: shared experts are always on, routed experts are
 * weighted by their gates).
 *
 *   y[t, :] = bf16( sum_{j<k} w[t, j] * D[inv_perm[t*k + j], :] + S[t, :] )
 * accumulated in fp32 in slot order j = 0..k-1, then S added.
 *
 * expert_out_bf16 D [R, H] bf16 (R >= T*k)
 * inv_perm        [T*k] int32
 * topk_w          [T, k] fp32
 * shared_out_bf16 S [T, H] bf16, or NULL for no shared expert
 * y_bf16    (out) [T, H] bf16
 * Requirements: 1 <= k <= 8, H % 8 == 0.
 */
int moe_combine(const void* expert_out_bf16, const int32_t* inv_perm,
                const float* topk_w, const void* shared_out_bf16,
                int64_t T, int32_t k, int64_t H, void* y_bf16, void* stream);

/*
 * moe_router_logits - the router's logits on their own: logits[t, e] = sum_h
 * x[t, h] * centroids[e, h], the exact products summed in fp32 as moe_route
 * sums them (its kernels), for a gate other than moe_route's (moe_gate).
 * x_bf16 [T, H]; centroids [E, H] fp32; logits (out) [T, E] fp32; workspace:
 * moe_route_workspace_bytes(T, H, E) bytes, 16-byte aligned.
 * Requirements: H % 128 == 0, 1 <= E <= 1024; x and centroids 16-byte aligned.
 * T == 0 is a no-op.
 */
int moe_router_logits(const void* x_bf16, int64_t T, int64_t H, const float* centroids, int32_t E,
                      float* logits, void* workspace, size_t workspace_bytes, void* stream);

/*
 * moe_router_logits_backward - the gradient of moe_router_logits, with the
 * kernels of moe_router_backward_dense:
 *   dx_out[t, :]      = bf16(dx_in[t, :] + sum_e d_logits[t, e] centroids[e, :])
 *   d_centroids[e, :] = sum_t d_logits[t, e] x[t, :]    (fp32, fixed order)
 * d_logits [T, E] fp32; dx_in_bf16 [T, H] or NULL (0), not aliasing dx_out;
 * workspace: moe_router_backward_dense_workspace_bytes(T, H, E) bytes.
 * Requirements: E % 16 == 0, 16 <= E <= 1024, H % 128 == 0, T <= 8388480;
 * tensors 16-byte aligned.  T == 0 writes d_centroids = 0.
 */
int moe_router_logits_backward(const void* x_bf16, const float* centroids, const float* d_logits,
                               int64_t T, int64_t H, int32_t E, const void* dx_in_bf16,
                               void* dx_out_bf16, float* d_centroids, void* workspace,
                               size_t workspace_bytes, void* stream);

/*
 * moe_gate - routing from given logits, in the forms moe_route does not have.
 * For each token, with its logits l (fp32 or bf16; scores and weights in fp32):
 *   s[e] = softmax(l)[e] over all E experts, or 1 / (1 + exp(-l[e]))
 *   v[e] = s[e] + bias[e], or l[e] without a bias (the same order as s)
 *   experts form n_group contiguous groups of E / n_group; a group's score is
 *   its largest v (group_top 1) or the sum of its two largest s + bias
 *   (group_top 2; of its only one, if it has one); the topk_group best groups
 *   are kept (n_group 1: every expert is); the k largest v among the kept
 *   experts are chosen; ties go to the lower index; ids are written in
 *   ascending order;
 *   w[j] = scale * s[e_j] / sum_j' s[e_j']  (renormalize 1; 0 if every s[e_j] is
 *                                           0 in fp32)
 *          scale * s[e_j]                   (renormalize 0)
 *   expert_counts[e] = number of tokens that chose e (overwritten).
 * The choice is that of s and v of the given logits and bias in 64-bit floating
 * point (values that are the same there tie: sigmoids of logits above 37, for
 * one): where fp32 values are too close to be told apart those are formed.
 * A logit of -inf excludes its expert: its score is 0 and it is chosen only
 * where fewer than k others are kept, a row of nothing but -inf has weights 0;
 * so does a bias of -inf, which leaves the score as it is.  Logits of +inf or
 * NaN give unspecified scores and weights, and k different ids in [0, E).
 * A softmax score under 2^-126, a sigmoid's under 2^-149, may be 0 in fp32.
 *
 * logits          [T, E] fp32 (logits_type MOE_TYPE_F32) or bf16 (MOE_TYPE_BF16)
 * bias            [E] fp32, or NULL
 * score           MOE_SCORE_SOFTMAX or MOE_SCORE_SIGMOID
 * topk_idx  (out) [T, k] int32, ascending per row;  topk_w (out) [T, k] fp32
 * expert_counts (out) [E] int32
 * scores    (out, optional: NULL skips it) [T, E] fp32: s; not aliasing logits
 * Requirements: 1 <= E <= 1024; n_group <= 32 divides E; 1 <= topk_group <=
 * n_group; group_top in {1, 2}; 1 <= k <= 8; k <= topk_group * E / n_group;
 * scale finite; tensors aligned to their elements.
 */
int moe_gate(const void* logits, int32_t logits_type, int64_t T, int32_t E, const float* bias,
             int32_t score, int32_t n_group, int32_t topk_group, int32_t group_top, int32_t k,
             int32_t renormalize, float scale, int32_t* topk_idx, float* topk_w,
             int32_t* expert_counts, float* scores, void* stream);

/*
 * moe_gate_backward - gradient of moe_gate's weights, and of its scores, to the
 * logits (the choice and the bias have none), in fp32:
 *   ds[e]  = d_scores[t, e] (0 if NULL), and for every chosen e_j
 *     renormalize 0:  ds[e_j] += scale * dw_j
 *     renormalize 1:  ds[e_j] += scale * (dw_j - sum_i dw_i s_i / S) / S,
 *                     S = sum_i s[e_i]  (nothing if every s[e_i] is 0 in fp32)
 *   d_logits[t, e] = s[e] * (ds[e] - sum_i ds[i] s[i])   (softmax)
 *                    ds[e] * s[e] * (1 - s[e])            (sigmoid)
 * logits, score, renormalize, scale as in moe_gate; topk_idx [T, k] its choice
 * (an id outside [0, E) is passed over, its dw with it; an id named twice
 * counts twice); d_topk_w [T, k]; d_scores [T, E] fp32 or NULL; d_logits (out)
 * [T, E] in the logits' type, not aliasing them.  Requirements: 1 <= E <= 1024,
 * 1 <= k <= 8, k <= E.
 */
int moe_gate_backward(const void* logits, int32_t logits_type, int64_t T, int32_t E, int32_t score,
                      int32_t k, int32_t renormalize, float scale, const int32_t* topk_idx,
                      const float* d_topk_w, const float* d_scores, void* d_logits, void* stream);

/*
 * int8_quant_rows - activations to 8-bit integers, one scale a token:
 *   scales[m] = max_k |in[m, k]| * (1 / 127)  (both fp32, the product rounded
 *               once: within 2^-23 of the quotient; 1 if it is 0)
 *   out[m, k] = in[m, k] / scales[m], the exact quotient rounded to the nearest
 *               whole number, ties to even: -127 .. 127
 * in_bf16 [M, ld_in], K columns used (16-byte aligned); out_int8 (out) [M, K]
 * (8-byte aligned); scales (out) [M] fp32.
 * Requirements: K % 8 == 0, K <= 2^24, ld_in % 8 == 0, ld_in >= K.
 */
int int8_quant_rows(const void* in_bf16, int64_t M, int64_t K, int64_t ld_in, int8_t* out_int8,
                    float* scales, void* stream);

/*
 * int8_quant_channels - weights to 8-bit integers, one scale an output channel:
 * the rule of int8_quant_rows on each row of w_f32 [G, N, K] fp32 (16-byte
 * aligned); out_int8 (out) [G, N, K] (8-byte aligned); scales (out) [G, N].
 * Requirements: K % 8 == 0, K <= 2^24, N > 0, G * N < 2^31.  G == 0 is a no-op.
 */
int int8_quant_channels(const float* w_f32, int64_t G, int64_t N, int64_t K, int8_t* out_int8,
                        float* scales, void* stream);

/*
 * grouped_int8_gemm - grouped product of 8-bit integers with a scale for each
 * token and each output channel (G = 1: a linear layer).  For group g, rows r
 * in [group_offsets[g], group_offsets[g+1]):
 *   C[r, n] = bf16( sum_k A[src, k] * B[g, n, k] * (A_scale[src] * B_scale[g, n]) )
 * src = a_row_index[r] if that is not NULL, else r.  The sum is exact (32-bit
 * integers), converted to fp32 once and scaled in fp32.
 *
 * A        [A_rows, K] int8;  A_scale [A_rows] fp32
 * a_row_index [M_total] int32 or NULL, A_rows: as in grouped_fp8_gemm
 * B        [G, N, K] int8 (K contiguous);  B_scale [G, N] fp32
 * group_offsets [G+1] int32 on the device, non-decreasing, [0] == 0, [G] <=
 *          M_total; rows from [G] on are left as they were
 * C  (out) [M_total, N] bf16
 * Requirements: N % 8 == 0, N <= 2^21, K % 16 == 0, K < 2^17, 1 <= G <= 1024;
 * A, B, C 16-byte aligned.
 */
int grouped_int8_gemm(const int8_t* A, const float* A_scale, const int32_t* a_row_index,
                      int64_t A_rows, const int8_t* B, const float* B_scale,
                      const int32_t* group_offsets, int32_t G, int64_t M_total, int64_t N, int64_t K,
                      void* C_bf16, void* stream);

/*
 * grouped_int8_gemm_swiglu - the gate+up product with SwiGLU in its epilogue.
 * B holds each group's fused weight [2I, K]: rows [0, I) gate, [I, 2I) up.
 * With gt and ut the fp32 values that grouped_int8_gemm (N = 2I) rounds to C:
 *   H[r, c] = bf16( gt / (1 + exp(-gt)) * ut )   (fp32)
 * H_bf16 (out) [M_total, I]; B_scale [G, 2I]; the rest and the requirements as
 * grouped_int8_gemm's, for I in place of N.
 */
int grouped_int8_gemm_swiglu(const int8_t* A, const float* A_scale, const int32_t* a_row_index,
                             int64_t A_rows, const int8_t* B, const float* B_scale,
                             const int32_t* group_offsets, int32_t G, int64_t M_total, int64_t I,
                             int64_t K, void* H_bf16, void* stream);

/*
 * grouped_bf16_gemm - grouped product of bf16 matrices: experts that are not
 * quantised (G = 1: a linear layer).  For group g, rows r in
 * [group_offsets[g], group_offsets[g+1]):
 *   C[r, n] = bf16( sum_k A[src, k] * B[g, n, k] )       (fp32 sums)
 * src = a_row_index[r] if that is not NULL, else r.
 *
 * A        [A_rows, K] bf16
 * a_row_index [M_total] int32 or NULL, A_rows: as in grouped_fp8_gemm
 * B        [G, N, K] bf16 (K contiguous)
 * group_offsets [G+1] int32 on the device, non-decreasing, [0] == 0, [G] <=
 *          M_total; rows from [G] on are left as they were
 * C  (out) [M_total, N] bf16
 * An infinity or NaN reaches the results that it takes part in and no others.
 * Requirements of all grouped bf16 products: N, K (I) multiples of 8, at most
 * 2^21; 1 <= G <= 1024; tensors 16-byte aligned.  M_total == 0 is a no-op
 * (grouped_bf16_wgrad writes dW = 0).
 */
int grouped_bf16_gemm(const void* A_bf16, const int32_t* a_row_index, int64_t A_rows,
                      const void* B_bf16, const int32_t* group_offsets, int32_t G, int64_t M_total,
                      int64_t N, int64_t K, void* C_bf16, void* stream);

/*
 * grouped_bf16_gemm_glu - both projections of the gated feed-forward block, the
 * activation and the product in one kernel.  B holds each group's fused
 * weight [2I, K]: rows [0, I) gate, [I, 2I) up.  With the fp32 sums gt and ut
 * that grouped_bf16_gemm (N = 2I) rounds to C:
 *   H[r, c] = bf16( act(gt) * ut )   (fp32);  act MOE_ACT_SILU or MOE_ACT_GELU
 * H_bf16 (out) [M_total, I]; GU_bf16 (out, optional: NULL skips it) [M_total,
 * 2I] = bf16 [gt | ut], what grouped_bf16_gemm_dgrad_glu reads.
 */
int grouped_bf16_gemm_glu(const void* A_bf16, const int32_t* a_row_index, int64_t A_rows,
                          const void* B_bf16, const int32_t* group_offsets, int32_t G,
                          int64_t M_total, int64_t I, int64_t K, int32_t act, void* H_bf16,
                          void* GU_bf16, void* stream);

/*
 * grouped_bf16_gemm_dgrad - the input gradient of grouped_bf16_gemm, from the
 * weights as stored (no transposed copy):
 *   dA[r, k] = bf16( sum_n dC[r, n] * W[g, n, k] )       (fp32 sums)
 * dC [M_total, N] bf16; W [G, N, K] bf16; dA (out) [M_total, K] bf16.  With a
 * row gather in the forward, dA's rows are the gathered ones (moe_combine with
 * unit weights adds them up for each token).
 */
int grouped_bf16_gemm_dgrad(const void* dC_bf16, const void* W_bf16, const int32_t* group_offsets,
                            int32_t G, int64_t M_total, int64_t N, int64_t K, void* dA_bf16,
                            void* stream);

/*
 * grouped_bf16_gemm_dgrad_glu - grouped_bf16_gemm_dgrad of the down projection
 * W [G, N, I] with the gated activation's backward in its epilogue: with dh the
 * fp32 sum that grouped_bf16_gemm_dgrad (K = I) rounds, g and u from GU_bf16
 * [M_total, 2I] = [g | u] (grouped_bf16_gemm_glu's),
 *   dGU[r, c]     = bf16( dh * u * act'(g) )
 *   dGU[r, I + c] = bf16( dh * act(g) )                  (fp32)
 * dGU_bf16 (out) [M_total, 2I], not aliasing GU_bf16.
 */
int grouped_bf16_gemm_dgrad_glu(const void* dC_bf16, const void* W_bf16, const void* GU_bf16,
                                const int32_t* group_offsets, int32_t G, int64_t M_total, int64_t N,
                                int64_t I, int32_t act, void* dGU_bf16, void* stream);

/*
 * grouped_bf16_wgrad - each group's weight gradient:
 *   dW[g, n, k] = sum_{r of group g} dY[r, n] * A[src(r), k]     (fp32)
 * summed in ascending order of rows, in steps of the matrix instruction.
 * dY [M_total, N] bf16; A [A_rows, K] bf16 with a_row_index as in
 * grouped_bf16_gemm; dW (out) [G, N, K] fp32, 0 for a group without rows.
 */
int grouped_bf16_wgrad(const void* dY_bf16, const void* A_bf16, const int32_t* a_row_index,
                       int64_t A_rows, const int32_t* group_offsets, int32_t G, int64_t M_total,
                       int64_t N, int64_t K, float* dW, void* stream);

/*
 * moe_norm - the norm before a block: the residual add, the RMS norm and the
 * codes that the block's first product reads, in one pass.  For each row t:
 *   v       = x[t, :] + add[t, :]     stored to sum_out in x's type (rounded to
 *                                     nearest even; what is stored is normed);
 *             x[t, :] without an add
 *   rstd[t] = 1 / sqrt( (1/H) sum_h v[h]^2 + eps )
 *   n[t, h] = bf16( v[h] * rstd[t] * weight[h] )
 * and from the fp32 products v * rstd * weight, before their rounding to bf16:
 *   MOE_QUANT_E4M3  codes [T, H] e4m3, scales [T, H/128]: fp8_quant_1x128's rule
 *   MOE_QUANT_INT8  codes [T, H] int8, scales [T]: int8_quant_rows' rule, the
 *                   quotient rounded to fp32 before it is to a whole number
 * in fp32: a row's squares have to stay under the largest fp32 number, and with
 * an eps under 2^-126 their mean above that (a row of zeros gives NaN with eps 0).
 * x        [T, H] fp32 or bf16 (x_type MOE_TYPE_*)
 * add_bf16 [T, H] bf16 or NULL;  sum_out (out) [T, H] of x_type, given if and
 *          only if add is; may equal x
 * weight   [H] fp32, or NULL (1)
 * n_bf16   (out) [T, H];  rstd (out, optional: NULL skips it) [T] fp32
 * Requirements: H % 8 == 0 (% 128 with E4M3 codes), H <= 16384, T < 2^28, 0 <=
 * eps <= 1; tensors 16-byte, codes 8-byte aligned.  T == 0 is a no-op.
 */
int moe_norm(const void* x, int32_t x_type, const void* add_bf16, const float* weight, int64_t T,
             int64_t H, float eps, void* sum_out, void* n_bf16, float* rstd, int32_t quant, void* codes,
             float* scales, void* stream);

/*
 * moe_norm_backward - the gradient of moe_norm's n to its normed rows v (and so
 * to x and add alike), with what comes down the residual path beside it:
 *   hat = v[t, :] * rstd[t];  g = dn[t, :] * weight
 *   dx[t, :]    = res_scale * d_res[t, :] + rstd[t] * (g - hat * (1/H) sum_h g hat)
 *   d_weight[h] = sum_t dn[t, h] * hat[t, h]        (fp32, in a fixed order)
 * dn_bf16 [T, H]; x [T, H] of x_type: v as stored (sum_out, or x without an
 * add); rstd [T]: moe_norm's; d_res [T, H] of x_type or NULL (0); dx (out)
 * [T, H] of x_type, may equal d_res; d_weight (out) [H] fp32, or NULL to skip
 * it; weight [H] or NULL (1).
 * workspace: moe_norm_backward_workspace_bytes(T, H) bytes, 16-byte aligned
 * (NULL without d_weight); calls that overlap need one each.
 * Requirements: as moe_norm's.  T == 0 writes d_weight = 0.
 */
size_t moe_norm_backward_workspace_bytes(int64_t T, int64_t H);
int moe_norm_backward(const void* dn_bf16, const void* x, int32_t x_type, const float* weight,
                      const float* rstd, const void* d_res, float res_scale, int64_t T, int64_t H,
                      void* dx, float* d_weight, void* workspace, size_t workspace_bytes, void* stream);

/*
 * moe_combine_norm - the end of a block: moe_combine's gate-weighted sum, a norm
 * after it and the scaled residual sum, in one pass.  For each token:
 *   z = sum_{j<k} topk_w[t, j] * D[inv_perm[t*k + j], :] + shared_w[t] * S[t, :]
 *   b = z * rstd[t] * weight,  rstd[t] = 1 / sqrt( (1/H) sum_h z[h]^2 + eps )
 *       (norm 0: rstd = 1, weight a scale for each channel)
 *   y[t, :] = residual_scale * residual[t, :] + scale * b
 * in fp32, z in slot order and never rounded; y rounded once to x_type.
 * D [R, H] bf16 (R >= T*k), inv_perm [T*k] (an entry outside [0, T*k) reads row
 * T*k - 1), topk_w [T, k], S [T, H] bf16 or NULL: as in moe_combine
 * shared_w  [T] fp32 or NULL (1): the shared expert's own gate
 * residual  [T, H] of x_type (MOE_TYPE_*);  weight [H] fp32 or NULL (1)
 * y (out)   [T, H] of x_type, may equal residual;  rstd (out, optional) [T]
 *           fp32, written with norm 1
 * Requirements: 1 <= k <= 8; H % 8 == 0, H <= 16384; T < 2^28; 0 <= eps <= 1;
 * tensors 16-byte aligned.  T == 0 is a no-op.
 */
int moe_combine_norm(const void* expert_out_bf16, const int32_t* inv_perm, const float* topk_w,
                     const void* shared_out_bf16, const float* shared_w, const void* residual,
                     int32_t x_type, float residual_scale, int32_t norm, const float* weight, float eps,
                     float scale, int64_t T, int32_t k, int64_t H, void* y, float* rstd, void* stream);

/*
 * moe_combine_norm_backward - backward of moe_combine_norm but for the residual's
 * part (residual_scale * dy, which moe_norm_backward adds as d_res).  z and
 * rstd are formed again from D, bit for bit; with hat = z * rstd, g = scale *
 * dy[t, :]:
 *   d_weight[h] = sum_t g * hat                      (fp32, in a fixed order)
 *   dz          = rstd * (g * weight - hat * (1/H) sum_h g * weight * hat)
 *                 (norm 0: g * weight)
 *   dD[inv_perm[t*k + j], :] = bf16( topk_w[t, j] * dz ),  d_topk_w[t, j] = <dz, D[..]>
 *   dD[T*k + t, :] = bf16( shared_w[t] * dz ),  d_shared_w[t] = <dz, D[T*k + t, :]>
 * dy [T, H] of x_type; D, dD (out) [T*k + n_shared*T, H] bf16; d_topk_w (out)
 * [T, k], d_shared_w (out, optional) [T] fp32; d_weight (out, optional) [H].
 * inv_perm entries outside [0, T*k) read row T*k - 1 and are not written.
 * d_expert_out_e4m3, d_expert_out_scale (out, both or neither): the 1x128
 * quantisation of dD, as in moe_combine_backward but of the fp32 products
 * before their rounding to bf16; needs H % 128 == 0.
 * workspace: moe_combine_norm_backward_workspace_bytes(T, H) bytes, as
 * moe_norm_backward's.  Requirements: as moe_combine_norm's, n_shared in {0,
 * 1}.  T == 0 writes d_weight = 0.
 */
size_t moe_combine_norm_backward_workspace_bytes(int64_t T, int64_t H);
int moe_combine_norm_backward(const void* dy, int32_t x_type, const int32_t* inv_perm,
                              const float* topk_w, const void* expert_out_bf16, int32_t n_shared,
                              const float* shared_w, int32_t norm, const float* weight, float eps,
                              float scale, int64_t T, int32_t k, int64_t H, void* d_expert_out_bf16,
                              float* d_topk_w, float* d_shared_w, uint8_t* d_expert_out_e4m3,
                              float* d_expert_out_scale, float* d_weight, void* workspace,
                              size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}  /* extern "C" */
#endif

#endif /* MOE_FP8_H */
