/*
 * moe_experts.h -- C ABI of what trains and serves the experts' weights of one
 * GPU's MoE share (moe_ep.h), in libmoe_experts.so:
 *
 *   serving in microscaled 4 bits (MX4):
 *     moe_quantize_mx4 -> moe_pack_mx4                       (the weights, once)
 *     moe_dispatch_layout -> moe_permute_mx4 -> moe_grouped_gemm_mx4 (twice)
 *       -> moe_combine                                       (each step)
 *   training:
 *     the share's backward -> moe_adamw_step
 *
 * MX4 is the OCP microscaling format with e2m1 elements: 32 neighbouring
 * columns of a row share one scale.
 *   codes  two a byte, the even column in the low nibble: sign, then
 *          0 .5 1 1.5 2 3 4 6
 *   scales one byte s per 32 columns (e8m0): 2^(s - 127); 255 is NaN
 *
 * The conventions are those of moe_ep.h: device pointers owned by the caller,
 * work enqueued on `stream` (a stream of the current device) without waiting,
 * launch shapes that depend on the size arguments alone (so every call can be
 * captured in a hipGraph and replayed on new contents), dense row-major
 * tensors, argument errors returned before anything is enqueued, padding rows
 * of expert-major buffers neither read nor written.  The library allocates
 * nothing and keeps no state; calls are independent of each other.
 */
#ifndef MOE_EXPERTS_H
#define MOE_EXPERTS_H

#include "moe_ep.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ABI version of libmoe_experts.so; bumped on any change of the functions here. */
int moe_experts_abi_version(void);

/*
 * moe_quantize_mx4 -- rows (activations or weights) to MX4.  Per 32 columns:
 *   s = 127 + the least e in [-127, 127] with max|x| < 7 * 2^e
 *   code = x / 2^e rounded to the nearest e2m1 value, ties to the even code
 * so nothing is off by more than half a step: 7 is where the next value of the
 * format (8) would begin, and everything below it rounds to 6 at most.  Codes
 * keep the sign of x, zeros included.  Columns of zeros have s = 0.  Where one
 * of the 32 is infinite or NaN, s is 255 and the codes are 0: a broken row
 * leaves as NaN, not as numbers.
 *   x [rows,K] x_dt in {F32, BF16}; codes [rows,K/2], scales [rows,K/32]
 *   values [rows,K] x_dt, or NULL: what the codes stand for (exact; infinite
 *   where that is 2^128 or more, of numbers from 3.5 * 2^126 on), for a training
 *   pass that sees the quantised rows; may be x itself
 * Limits: K % 32 == 0, rows * K <= 2^40; x, codes and values 16-byte aligned.
 */
moe_status moe_quantize_mx4(const void* x, moe_dtype x_dt, int64_t rows, int K, void* codes, void* scales,
                            void* values, hipStream_t stream);

/*
 * moe_permute_mx4 -- moe_permute into MX4 rows:
 *   (buf, buf_scales)[slot_of[t,k],:] = MX4 of x[t,:]
 * for every (t,k) with 0 <= slot_of < rows_cap, by the rule of
 * moe_quantize_mx4.
 *   x [T,H] x_dt in {F32, BF16}; slot_of [T,K]; buf [rows_cap,H/2],
 *   buf_scales [rows_cap,H/32]
 * Limits: H % 32 == 0, H <= 2^25, K <= 64, T * ceil(H / 1024) < 2^31; x and buf
 * 16-byte aligned.
 */
moe_status moe_permute_mx4(const void* x, moe_dtype x_dt, int T, int K, int H, const int32_t* slot_of,
                           int64_t rows_cap, void* buf, void* buf_scales, hipStream_t stream);

/*
 * moe_pack_mx4 -- MX4 expert weights in the order in which
 * moe_grouped_gemm_mx4 reads them; once per weight update.
 *   codes [L,N,K/2], scales [L,N,K/32], as moe_quantize_mx4 writes them.
 * The packed copies have the same sizes and may not overlap the sources:
 *   codes  [L][N/16][K/128][64][16 bytes]: 16 rows x 128 columns are 1 KB; piece
 *          l holds row l & 15, columns 32 (l >> 4) .. + 31
 *   scales [L][N/16] runs of K/128 * 64 bytes: for every four 128-column steps
 *          [64][4], then for what is left [64][1..3]: byte (l, j) is the scale of
 *          piece l in step j of the four
 * Limits: N % 16 == 0, K % 128 == 0, N K <= 2^31, K <= 2^24, L N K < 2^39,
 * L <= 1024; codes and codes_packed 16-byte, scales and scales_packed 4-byte
 * aligned.
 */
moe_status moe_pack_mx4(const void* codes, const void* scales, int L, int N, int K, void* codes_packed,
                        void* scales_packed, hipStream_t stream);

/*
 * moe_grouped_gemm_mx4 -- the experts' products of MX4 rows and MX4 weights:
 *   G[q,n] = sum_k A[q,k] W[e,n,k]
 * for the valid rows q of expert e (counts, offsets as moe_dispatch_layout
 * writes them; rows past rows_cap are skipped), with fp32 sums.  Any number of
 * rows an expert, from decode steps to prefill.
 *   a [rows_cap,K/2], a_scales [rows_cap,K/32]; codes_packed, scales_packed as
 *   written by moe_pack_mx4 with the same L, N, K
 *   epi MOE_EPI_STORE_G: out [rows_cap,N] = G
 *   epi MOE_EPI_SILU_MUL: out [rows_cap,N/2] = SiLU(G[:, :N/2]) * G[:, N/2:]
 *   out_dt F32 or BF16 with out_scales NULL; or, with MOE_EPI_SILU_MUL,
 *   MOE_FP8_E4M3 as the mark of a byte buffer: out [rows_cap,N/4] and out_scales
 *   [rows_cap,N/64] are MX4, quantised from the fp32 products by the rule of
 *   moe_quantize_mx4 (the rows of the next product)
 * A row with a NaN scale (255) is NaN, and so is a column of a weight with one;
 * other rows and columns are not touched by it.
 * Limits: N % 32 == 0 (N % 64 == 0 with MX4 out), K % 128 == 0, N K <= 2^31,
 * K <= 2^24, L N K < 2^39, L <= 1024, rows_cap <= 2^30; a, codes_packed and out
 * 16-byte, a_scales and scales_packed 4-byte aligned.
 */
moe_status moe_grouped_gemm_mx4(const void* a, const void* a_scales, const void* codes_packed,
                                const void* scales_packed, const int32_t* counts, const int32_t* offsets,
                                int L, int64_t rows_cap, int N, int K, moe_w13_epilogue epi, void* out,
                                moe_dtype out_dt, void* out_scales, hipStream_t stream);

/* One tensor of moe_adamw_step: n elements each, device pointers. */
typedef struct moe_adamw_tensor {
  void* param;                /* p_dt: read (without master) and written      */
  float* master;              /* fp32 copy of param that is updated, or NULL  */
  const void* grad;           /* g_dt                                         */
  void* exp_avg;              /* m: fp32, or e4m3fn codes                     */
  void* exp_avg_sq;           /* v: fp32, or e4m3fn codes of sqrt(v)          */
  float* exp_avg_scale;       /* [ceil(n/128)] with 8-bit states, else NULL   */
  float* exp_avg_sq_scale;    /* [ceil(n/128)] with 8-bit states, else NULL   */
  int64_t n;
} moe_adamw_tensor;

/* What a step does to every tensor alike. */
typedef struct moe_adamw_config {
  double lr, beta1, beta2, eps, weight_decay;
  int64_t step;               /* number of this update, 1 for the first       */
  const float* lr_device;     /* read when the step runs, in place of lr, or NULL   */
  const int64_t* step_device; /* likewise in place of step, or NULL           */
  const float* grad_scale;    /* device: factor of every gradient, or NULL    */
  uint32_t seed;              /* of the 8-bit states' rounding                */
} moe_adamw_config;

/*
 * moe_adamw_step -- one AdamW update of many tensors, in fp32:
 *   g = grad * grad_scale
 *   m = beta1 m + (1 - beta1) g,  v = beta2 v + (1 - beta2) g^2
 *   p = p - lr weight_decay p - lr / (1 - beta1^t) m / (sqrt(v / (1 - beta2^t)) + eps)
 * with p = master, of which param is then the rounded copy, or p = param.  An eps
 * above 0 counts as 2^-149, fp32's least number, at least.
 *   s_dt F32: m and v are fp32.
 *   s_dt FP8_E4M3: m and sqrt(v) are e4m3fn codes with one fp32 scale per 128
 *   neighbouring elements (value = code * scale, scale = max * fp32(1/448)
 *   of the block's finite values; 0 where that is below 1e-30).  The update uses the new m
 *   and v before they are rounded.  They are rounded at random, up with the
 *   probability of the place between two codes: a v that moves by a part in
 *   a thousand a step would otherwise stay where it is, codes being 6 to 12 %
 *   apart.  The place is taken in 2^-20 of a step (nearest, ties to even); it
 *   rounds up where 16 times a 16-bit number carries it past one step.  The two numbers
 *   of element i of tensor j are the high (m) and low half (v) of
 *     mix(lo(i) ^ key),  key = mix(mix(mix(seed) + lo(step)) + j), with i >= 2^32
 *     key = mix(key + hi(i)) once more
 *     mix(x): x = (x ^ x >> 16) * 0x9e3779b9, x = (x ^ x >> 15) * 0xbb67ae85,
 *             x ^ x >> 16, in 32 bits
 *   so a step can be repeated.  A sqrt(v) above 0 does not become 0.  An element
 *   whose new m (or v) is infinite or NaN gets the code NaN in it.
 * Nothing is changed where step_device holds a number below 1, or where
 * grad_scale is infinite or NaN (a step to be skipped).
 *   tensors[count] is host memory and read before the call returns; p_dt, g_dt
 *   in {F32, BF16}; master only with p_dt BF16, for all tensors or for none.
 * Limits: lr, eps and weight_decay finite and >= 0, beta1 and beta2 in [0, 1), step >= 1
 * (without step_device); 0 <= n <= 2^40; all device pointers 16-byte aligned (the
 * states' scales, lr_device and grad_scale 4, step_device 8).  Tensors of one call may not overlap.
 */
moe_status moe_adamw_step(const moe_adamw_tensor* tensors, int count, moe_dtype p_dt, moe_dtype g_dt,
                          moe_dtype s_dt, const moe_adamw_config* config, hipStream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_EXPERTS_H */
