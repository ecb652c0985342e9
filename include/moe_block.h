/*
 * moe_block.h -- C ABI of what stands around and inside one GPU's MoE share
 * (moe_ep.h) in a transformer block, in libmoe_block.so:
 *
 *   moe_add_rms_norm -> (router logits) -> moe_router_group_topk
 *     -> moe_dispatch_layout -> moe_permute_fp8 -> moe_grouped_gemv_w4 (twice)
 *     -> moe_combine
 *
 * and the gradients of the norm and of the routing.
 *
 * The conventions are those of moe_ep.h: device pointers owned by the caller,
 * work enqueued on `stream` (a stream of the current device) without waiting,
 * launch shapes that depend on the size arguments alone (so every call can be
 * captured in a hipGraph and replayed on new contents), dense row-major
 * tensors, argument errors returned before anything is enqueued, padding rows
 * of expert-major buffers neither read nor written.  The library allocates
 * nothing and keeps no state; calls are independent of each other, but a
 * workspace must not be shared by calls that overlap in time.
 */
#ifndef MOE_BLOCK_H
#define MOE_BLOCK_H

#include "moe_ep.h"

#ifdef __cplusplus
extern "C" {
#endif

/* How moe_router_group_topk scores the experts of a token. */
typedef enum moe_score {
  MOE_SCORE_SOFTMAX = 0,      /* exp(l - max l) / sum exp(l - max l)       */
  MOE_SCORE_SIGMOID = 1       /* 1 / (1 + exp(-l))                         */
} moe_score;

/* The 16 values of a 4-bit weight code. */
typedef enum moe_w4_format {
  MOE_W4_INT4 = 0,            /* code - 8: -8 .. 7                         */
  MOE_W4_E2M1 = 1             /* OCP e2m1: sign, then 0 .5 1 1.5 2 3 4 6   */
} moe_w4_format;

/* ABI version of libmoe_block.so; bumped on any change of the functions here. */
int moe_block_abi_version(void);

/*
 * moe_add_rms_norm -- the residual's addition and the RMS norm in front of the
 * router and the experts:
 *   h[t]  = x[t] + residual[t], rounded to x_dt (h = x without a residual)
 *   y[t]  = h[t] * r[t] * weight,  r[t] = 1 / sqrt(mean_j h[t,j]^2 + eps)
 * in fp32 from the rounded h, so that a backward or a later layer that reads
 * h_out sees the values that were normed.
 *   x, residual (or NULL) [T,H] x_dt in {F32, BF16};  weight [H] w_dt in
 *   {F32, BF16}
 *   h_out [T,H] x_dt, or NULL; may be x or residual itself (in place)
 *   y [T,H] x_dt, or NULL; may be x or residual itself, not h_out
 *   y8 [T,H] e4m3fn with y8_scales [T,H/128] fp32, or both NULL: y quantised
 *   from fp32 with the recipe of moe_permute (rows that moe_permute_fp8 takes);
 *   where a group's y holds a NaN its scale and codes are NaN, and one whose
 *   largest magnitude is infinite has scale infinity, code NaN at its infinities
 *   and 0 elsewhere, so that no broken row leaves as numbers
 * At least one of h_out, y, y8 is given.  eps >= 0 and finite; a row of zeros
 * with eps = 0 gives NaN, in y and in y8.  The mean square is fp32's: a row
 * whose squares pass fp32's range has r = 0.
 * Limits: T <= 2^30, H % 8 == 0, H <= 16384, H % 128 == 0 with y8; x, residual, weight,
 * h_out, y and y8 16-byte aligned.
 */
moe_status moe_add_rms_norm(const void* x, const void* residual, moe_dtype x_dt, const void* weight,
                            moe_dtype w_dt, float eps, int T, int H, void* h_out, void* y, void* y8,
                            float* y8_scales, hipStream_t stream);

/* Device workspace bytes of moe_add_rms_norm_backward (0 for sizes it refuses). */
size_t moe_add_rms_norm_backward_workspace_bytes(int T, int H);

/*
 * moe_add_rms_norm_backward -- the gradients of moe_add_rms_norm, from the
 * saved h (h_out, or x without a residual) and dy = dL/dy:
 *   dx[t] = dh[t] + r * (weight dy - n * mean_j(weight_j dy_j n_j)), n = h r
 *           (the gradient of x and of residual alike; dh = dL/dh_out, the
 *           gradient that arrives on the residual stream, or NULL)
 *   d_weight = sum_t dy[t] * n[t]   (fp32; summed in a fixed order)
 *   dy, h, dh (or NULL), dx [T,H] dt in {F32, BF16}; weight [H] w_dt in {F32,
 *   BF16}; d_weight [H] fp32, written (zeros for T = 0).  dx may be dy, h or
 *   dh itself.
 *   workspace >= moe_add_rms_norm_backward_workspace_bytes(T, H) bytes,
 *   16-byte aligned.
 * Limits: as moe_add_rms_norm; every pointer 16-byte aligned.
 */
moe_status moe_add_rms_norm_backward(const void* dy, const void* h, const void* dh, moe_dtype dt,
                                     const void* weight, moe_dtype w_dt, float eps, int T, int H, void* dx,
                                     float* d_weight, void* workspace, size_t workspace_bytes,
                                     hipStream_t stream);

/*
 * moe_router_group_topk -- group-limited selection of K experts per token,
 * with sigmoid or softmax scores and a bias that balances the experts' load:
 *   s[t,e] = score(logits[t,:])            (moe_score)
 *   c[t,e] = s[t,e] + bias[e]              (c = s without a bias)
 *   the E experts form n_group groups of E/n_group neighbours; a group ranks by
 *   the sum of its group_top (1 or 2) largest c, and the topk_group best groups
 *   stay (ties: the lower group)
 *   topk_ids[t,:] = the K largest c among their experts, descending (ties: the
 *   lower id)
 *   topk_weights[t,k] = route_scale * s[t,id_k], divided by
 *   (sum_k s[t,id_k] + 1e-20) with renorm: the bias steers the choice only
 * Masks: a logit or a bias at or below -3.3e38 (so -inf, and the lowest finite
 * fp32 and bf16 value) excludes its expert; a masked logit scores 0 and takes
 * no part in the softmax.  Where fewer than K experts remain, the other ids
 * are -1 ("no route" to moe_dispatch_layout) with weight 0: a fully masked row
 * (a padded token) routes nowhere.  A NaN score ranks below every number and
 * above a masked expert.
 * Scores are fp32, but the choice is the one that fp64 scores give, with and
 * without a bias: rows whose candidates lie closer than fp32 can tell apart are
 * decided again in fp64.  Scores that are the same fp64 number tie, as those of
 * sigmoid logits above 37 (all 1) or of logits more than 746 below the largest
 * with softmax (all 0).
 *   logits [T,E] fp32; bias [E] fp32 or NULL; topk_ids [T,K] int32,
 *   topk_weights [T,K] fp32.
 * Limits: T <= 2^30, E <= 1024, 1 <= K <= 32, E % n_group == 0, n_group <= 64,
 * 1 <= topk_group <= n_group, K <= topk_group * (E / n_group).
 */
moe_status moe_router_group_topk(const float* logits, const float* bias, int T, int E, int K,
                                 moe_score score, int n_group, int topk_group, int group_top, int renorm,
                                 float route_scale, int32_t* topk_ids, float* topk_weights,
                                 hipStream_t stream);

/*
 * moe_router_group_topk_backward -- d_logits [T,E] from d_weights = dL/dtopk_weights
 * [T,K] and the forward's logits and ids (the scores are computed again; the
 * choice is constant, so the bias has no gradient):
 *   ds_k = route_scale * d_weights_k, with renorm
 *          route_scale * (d_weights_k - sum_j d_weights_j w_j / S) / S, where
 *          w_j = s[id_j], S = sum_j w_j + 1e-20
 *   sigmoid: d_logits[id_k] += ds_k s (1 - s);
 *   softmax: d_logits[e] = s_e (ds_e - sum_k ds_k w_k) over the whole row
 * Every element of d_logits is written (0 where nothing arrives).  Ids outside
 * [0, E) are no route; an id that occurs twice counts twice.
 * Limits: T <= 2^30, E <= 1024, 1 <= K <= 32.
 */
moe_status moe_router_group_topk_backward(const float* logits, const int32_t* topk_ids,
                                          const float* d_weights, int T, int E, int K, moe_score score,
                                          int renorm, float route_scale, float* d_logits,
                                          hipStream_t stream);

/*
 * moe_permute_fp8 -- moe_permute for rows that are in block FP8 already:
 *   buf[slot_of[t,k],:] = x8[t,:],  buf_scales[slot_of[t,k],:] = x8_scales[t,:]
 * for every (t,k) with 0 <= slot_of < rows_cap, copied bit for bit.
 *   x8 [T,H] e4m3fn, x8_scales [T,H/128] fp32 (as moe_add_rms_norm writes
 *   them); slot_of [T,K]; buf [rows_cap,H], buf_scales [rows_cap,H/128]
 * Limits: H % 128 == 0, H <= 2^25, K <= 64, T times the 2 KB parts of a row below
 * 2^31; x8, buf 16-byte aligned.
 */
moe_status moe_permute_fp8(const void* x8, const float* x8_scales, int T, int K, int H,
                           const int32_t* slot_of, int64_t rows_cap, void* buf, float* buf_scales,
                           hipStream_t stream);

/*
 * moe_pack_w4 -- 4-bit expert weights and their scales in the order in which
 * moe_grouped_gemv_w4 reads them; once per weight update.
 *   codes [L,N,K/2] uint8: byte b of row n holds the code of column 2b in its
 *   low and of column 2b+1 in its high nibble
 *   scales [L,N,K/group] s_dt in {F32, BF16}: the weight is code value * scale
 * The packed copies have the same sizes and may not overlap the sources:
 *   codes  [L][N/16][K/128][64][16 bytes]: 16 rows x 128 columns are 1 KB; piece
 *          l holds of row l & 15 the columns 32 s + 8 (l >> 4) + 0..7 as its
 *          dword s (INT4: column 2i in bits 4 i + 3 .. 4 i + 6, 2 i + 1 sixteen
 *          bits above, bit 32 being bit 0; E2M1: in column order)
 *   scales [L][N/16][K/128][16 rows][128/group]
 * Limits: N % 128 == 0, K % 128 == 0, N K <= 2^31, K <= 2^24, L <= 1024, group in
 * {32, 64, 128}; codes, codes_packed and scales_packed 16-byte aligned.
 */
moe_status moe_pack_w4(const void* codes, const void* scales, moe_dtype s_dt, moe_w4_format fmt, int L,
                       int N, int K, int group, void* codes_packed, void* scales_packed,
                       hipStream_t stream);

/*
 * moe_grouped_gemv_w4 -- the experts' products with 4-bit weights, for decode
 * steps that give an expert few rows:
 *   G[q,n] = sum_k A[q,k] W[e,n,k],  W[e,n,k] = value(code) * scale[e,n,k/group]
 * for the valid rows q of expert e (counts, offsets as moe_dispatch_layout
 * writes them; rows past rows_cap are skipped).  A is bf16, or block FP8 with a
 * scale per row and 128 columns.  The 4-bit values enter the matrix cores
 * exactly; scales multiply the fp32 sums of their group.
 *   a [rows_cap,K] a_dt in {BF16, FP8_E4M3}; a_scales [rows_cap,K/128] fp32
 *   for FP8, else NULL
 *   codes_packed, scales_packed: as written by moe_pack_w4 with the same fmt,
 *   s_dt, group, L, N, K
 *   epi MOE_EPI_STORE_G: out [rows_cap,N] = G (gate/up or down products);
 *   MOE_EPI_SILU_MUL: out [rows_cap,N/2] = SiLU(G[:, :N/2]) * G[:, N/2:]
 *   out_dt in {F32, BF16}
 * Every count is right; weights are read once per 32 rows of an expert, so this
 * is the form for few rows per expert (moe_grouped_gemm_w13 / _w2 for many).
 * A row with an infinite or NaN activation (or scale of it) has no finite value:
 * with INT4 codes and bf16 rows it is NaN, as may be finite rows whose sums over a
 * group pass 2^123 (codes ride as 16 + code).  Other rows are not touched by it.
 * Limits: N % 128 == 0, K % 128 == 0, N K <= 2^31, L N K < 2^39, K <= 2^24,
 * L <= 1024, group in {32, 64, 128}; a, codes_packed, scales_packed and out 16-byte aligned.
 */
moe_status moe_grouped_gemv_w4(const void* a, moe_dtype a_dt, const float* a_scales,
                               const void* codes_packed, const void* scales_packed, moe_dtype s_dt,
                               moe_w4_format fmt, int group, const int32_t* counts,
                               const int32_t* offsets, int L, int64_t rows_cap, int N, int K,
                               moe_w13_epilogue epi, void* out, moe_dtype out_dt, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_BLOCK_H */
