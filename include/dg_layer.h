/*
 * dg_layer.h -- C ABI of the operators around the tensor-parallel GEMM of
 * dg.h: residual add with RMS norm (16- or 8-bit output, and its gradient),
 * products grouped by expert (forward and gradients), microscaled 4-bit
 * quantisation and the product of microscaled 4-bit tensors.
 *
 * Every call checks its arguments, enqueues its work on `stream` (a
 * cudaStream_t of the current device) and returns a dg_status (dg.h);
 * dg_layer_last_error() gives a message for the calling thread.  No call
 * synchronizes, allocates device memory or keeps state between calls except
 * the device's properties; every call may be captured into a CUDA graph.  The
 * calls may be used from several threads and on several streams at once:
 * all device memory that a call uses is its arguments'.
 *
 * `status`: one 64-bit word of device memory, zeroed once by the caller, that
 * the matrix-product kernels write if an internal pipeline wait runs out (they
 * stop instead of hanging).  dg_layer_check() reads and clears it.  One word
 * may serve any number of calls.
 */
#ifndef DG_LAYER_H_
#define DG_LAYER_H_

#include "dg.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Residual add and RMS norm over rows of `hidden` values:
 *     h = x + residual        rounded to the residual's type (h = x without one)
 *     y = h * rsqrt(mean(h^2) + eps) * weight
 * written as bf16 (y_type DG_TYPE_BF16), or in 8 bits (DG_TYPE_E4M3 / E5M2,
 * nearest even, saturating) as y / c with the row's own scale
 * c = max|y| / largest finite value (at least 2^-126; 1 for a row of zeros;
 * scale_out, one fp32 per row), or, with scale_in (one fp32 in device memory),
 * as y / *scale_in.
 * x: bf16; residual: NULL, or bf16 / fp32 (residual_type); sum_out: h in the
 * residual's type, required with a residual and may be the residual's own
 * memory (its rows may not overlap, nor share other values with x); weight: bf16 or fp32 (weight_type); rstd_out: NULL, or the rows'
 * fp32 reciprocal deviations, for the gradient.  ld_*: elements from row to
 * row; y, scale_out and rstd_out are densely packed.  Any hidden (rows
 * of no values have the scale 1 and rstd NaN, the mean of nothing); rows whose
 * pointers and pitches are 16-byte aligned with hidden % 8 == 0 take 16-byte
 * accesses.  Statistics and products are computed in fp32.  A NaN or
 * infinity in a row stays in its row and never enters a scale. */
int dg_layer_add_rms_norm(const void* x, int64_t ld_x, const void* residual, int64_t ld_residual,
                          int residual_type, const void* weight, int weight_type, void* y, int y_type,
                          void* sum_out, int64_t ld_sum, float* scale_out, const float* scale_in,
                          float* rstd_out, int64_t rows, int64_t hidden, float eps, void* stream);

/* Gradient of dg_layer_add_rms_norm with a bf16 output: with xh = h * rstd and
 * g = dy * weight,
 *     dx = rstd * (g - xh * mean(g * xh)) + dh,     dweight = sum over rows of dy * xh.
 * dy: bf16; h: the stored sum, bf16 or fp32 (h_type); dh: NULL or the gradient
 * that reaches h on its other way, in h's type; dx: in h's type (it is the
 * gradient of x and of the residual); dweight: in the weight's type.
 * workspace: dg_layer_add_rms_norm_backward_workspace() bytes, 16-byte
 * aligned.  The row sums of dweight are added in a fixed order (the same bits
 * every time). */
size_t dg_layer_add_rms_norm_backward_workspace(int64_t rows, int64_t hidden);
int dg_layer_add_rms_norm_backward(const void* dy, int64_t ld_dy, const void* h, int64_t ld_h, int h_type,
                                   const void* weight, int weight_type, const float* rstd, const void* dh,
                                   int64_t ld_dh, void* dx, void* dweight, void* workspace, int64_t rows,
                                   int64_t hidden, void* stream);

/* Products grouped by expert: rows ends[e-1] <= t < ends[e] of A (T x K) times
 * expert e's matrix,
 *     D[t, n] = scale_a[t] * scale_b[e, n] * sum_k A[t, k] * B[e, n, k]
 * (fp32 accumulation, the scales in fp32, also where scale_a scale_b alone is
 * beyond fp32's range, one rounding to D's type).  `ends`:
 * `experts` ascending int32 in device memory; values are clamped to
 * [previous end, T] on the device, rows past the last end are written as 0.
 * type: DG_TYPE_BF16, or DG_TYPE_E4M3 / E5M2 for A and B each.  b_n_major: 0 =
 * B's rows (fixed n) are contiguous along k, 1 (bf16 only) = contiguous along
 * n: element (e, n, k) at e * ld_e + k * ld_b + n.  ld_a, ld_b, ld_e (of two
 * experts and more) in elements; the pitches and pointers are multiples of 16
 * bytes.  scale_a / scale_b: NULL, or fp32 with strides in elements (0 = shared): scale_a[t * sa],
 * scale_b[e * sb_e + n * sb_n].  D: bf16 or fp32 (d_type), T x N densely packed.
 * N % 8 == 0 and K % 8 == 0 (bf16) or K % 16 == 0 (8 bits).  T, N, K <= 2^31 - 256;
 * experts <= 1024.  workspace: dg_layer_products_workspace() bytes of the
 * current device, 16-byte aligned, its first DG_LAYER_COUNTER_BYTES zeroed once
 * before its first use (each call leaves them zero, except one that
 * dg_layer_check() reports: zero them again after it); calls that may run at
 * the same time need different ones. */
#define DG_LAYER_COUNTER_BYTES ((size_t)2048)
size_t dg_layer_products_workspace(void);
int dg_layer_grouped_matmul(const void* A, int64_t ld_a, int a_type, const void* B, int64_t ld_b, int64_t ld_e,
                            int b_type, int b_n_major, const int32_t* ends, int experts, const float* scale_a,
                            int64_t sa, const float* scale_b, int64_t sb_e, int64_t sb_n, void* D, int d_type,
                            int64_t T, int64_t N, int64_t K, void* workspace, void* status, void* stream);

/* Gradient of the experts' matrices: dB[e, n, k] = sum over the rows t of
 * group e of dD[t, n] * A[t, k] (bf16 operands, fp32 accumulation; 0 for an
 * empty group), dB bf16 or fp32 (d_type), experts x N x K densely packed.
 * workspace: dg_layer_grouped_grad_workspace() bytes, 16-byte aligned;
 * products_workspace: as the workspace of dg_layer_grouped_matmul. */
size_t dg_layer_grouped_grad_workspace(int experts, int64_t N, int64_t K);
int dg_layer_grouped_weight_grad(const void* dD, int64_t ld_d, const void* A, int64_t ld_a, const int32_t* ends,
                                 int experts, void* dB, int d_type, int64_t T, int64_t N, int64_t K,
                                 void* workspace, void* products_workspace, void* status, void* stream);

/* Microscaled 4 bits (OCP MX, e2m1 elements, one e8m0 scale for each 32
 * columns): scale 2^E with E = floor(log2(max|x|)) - 2, at least -127; element
 * x / 2^E to the nearest code, ties to the even code, saturating at 6.  A block
 * of zeros has scale byte 0; a block with a NaN or an infinity has scale byte
 * 255 (NaN) and codes 0.
 *   codes   rows x cols / 2 bytes, densely packed, the even column in the low half
 *   scales  tiles of 128 rows x 4 scales (512 bytes): tile (i, j) at
 *           (i * 2 * ceil(cols / 256) + j) * 512, row r, scale s of it at
 *           (r % 32) * 16 + (r / 32) * 4 + s: the order in which the block-scaled
 *           tensor core instructions read them from tensor memory.  Absent
 *           rows and columns are written as 0.
 * cols % 32 == 0; x: bf16 or fp32 (x_type), 16-byte aligned rows. */
size_t dg_layer_mx4_scale_bytes(int64_t rows, int64_t cols);
int dg_layer_mx4_quantize(const void* x, int64_t ld_x, int x_type, void* codes, void* scales, int64_t rows,
                          int64_t cols, void* stream);
/* The values that the codes stand for, as bf16 (exact) or fp32, densely packed. */
int dg_layer_mx4_dequantize(const void* codes, const void* scales, void* y, int y_type, int64_t rows,
                            int64_t cols, void* stream);
/* D[m, n] = sum_k a[m, k] * b[n, k] over the values of two such tensors (M x K
 * and N x K), fp32 accumulation, D bf16 or fp32 (d_type), M x N densely
 * packed.  N % 8 == 0.  workspace as for dg_layer_grouped_matmul. */
int dg_layer_mx4_matmul(const void* a_codes, const void* a_scales, const void* b_codes, const void* b_scales,
                        void* D, int d_type, int64_t M, int64_t N, int64_t K, void* workspace, void* status,
                        void* stream);

/* Synchronize `stream`, read the status word and clear it: DG_OK, or
 * DG_ERR_HANG if a product's pipeline wait ran out since the last check. */
int dg_layer_check(void* status, void* stream);

const char* dg_layer_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* DG_LAYER_H_ */
