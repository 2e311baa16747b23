/*
 * sgemm_fp8.h -- the 8-bit part of libsgemm: matrices of 8-bit floating point
 * values with a scale for each block of 128, their product with FP32
 * accumulation, what produces them (a quantiser, an RMS norm with residual
 * addition) and a mixture-of-experts layer for a few tokens on such weights.
 *
 * Conventions are those of sgemm.h: row-major matrices, `ld` = row stride of
 * the stored matrix in elements, device pointers owned by the caller, work
 * enqueued on `stream` of the current device, -(argument index) for an invalid
 * argument before anything is launched, SGEMM_ERR_* otherwise, workspace from
 * the library's stream-ordered pool.  Every call can be captured in a CUDA
 * graph after one eager call of this part on the device, which sets up its
 * kernels.  Results are deterministic: no sum's order depends on scheduling.
 *
 * 8-bit matrices.  A stored R x C matrix has one code per element and one FP32
 * scale per group of block_rows x block_cols elements, 1 x 128, 128 x 1 or
 * 128 x 128 (the last group of a row or column may be short); element (r, c) is
 *     value(r, c) = code(r, c) * scale[(r / block_rows) * lds + c / block_cols].
 * Codes are E4M3 (1-4-3 bits, +-448, NaN, no infinity) or E5M2 (1-5-2 bits,
 * +-57344, infinities and NaN).
 */
#ifndef SGEMM_FP8_H
#define SGEMM_FP8_H

#include "sgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

enum sgemm_fp8_format { SGEMM_FP8_E4M3 = 0, SGEMM_FP8_E5M2 = 1 };

/* Element types of the matrices that are not 8-bit. */
enum sgemm_type { SGEMM_F32 = 0, SGEMM_BF16 = 1 };

/* Kernel variants of sgemm_fp8(), as sgemm_fp8_plan() reports them (sgemm_plan_t.variant; the
 * numbers follow those of enum sgemm_variant, whose NONE and SCALE are reported too). */
enum sgemm_fp8_variant {
    SGEMM_VARIANT_FP8_PAIR = 32,  /* CTA pairs, 256 x tile_n tiles (tile_n 64, 128 or 256), 128 k per tile */
    SGEMM_VARIANT_FP8_SHORT = 33  /* one CTA per 128 x tile_n tile (128 along the longer of M and N, tile_n 16, 32,
                                     64 or 128 along the other), K shared by a cluster of split_k CTAs */
};

/* A stored 8-bit matrix (its row and column counts come from the call). */
typedef struct sgemm_fp8_matrix_t {
    const void *data;     /* codes, row-major */
    int64_t ld;           /* row stride of the codes */
    const float *scale;   /* one per group, row-major */
    int64_t lds;          /* row stride of the scales */
    int format;           /* enum sgemm_fp8_format */
    int block_rows;       /* 1 or 128 */
    int block_cols;       /* 1 or 128 (not 1 x 1) */
} sgemm_fp8_matrix_t;

/*
 * sgemm_fp8 -- D = alpha * op(A) * op(B) + beta * C on 8-bit matrices, summed as
 *     D_ij = alpha * sum_g sA(i, g) sB(g, j) (sum_{k in group g} a_ik b_kj) + beta * C_ij
 * over the groups g of 128 consecutive k: the inner sums of code products on
 * the tensor cores in FP32, the outer sum in FP32 registers.
 *   - transA, transB, M, N, K and the stored shapes as in sgemm(); A and B must
 *     have groups of 128 along k: block_cols = 128 where k runs along the
 *     stored rows (A 'N', B 'T'), block_rows = 128 where it runs down the
 *     stored columns (A 'T', B 'N'); along the other dimension 1 or 128.
 *     So 'N','T' with 1 x 128 activations and 128 x 128 weights is a forward
 *     product, 'N','N' with the same weights the gradient of its inputs,
 *     'T','N' with 128 x 1 groups on both sides the gradient of the weights.
 *   - C and D: `type` (enum sgemm_type), row stride ldc and ldd.  D may be C
 *     (then ldd == ldc); otherwise no operand may overlap D.  beta == 0: C is
 *     not read and may be NULL.  alpha == 0 or K == 0: A and B are not read.
 *   - Errors per element, against the sum taken exactly: at most
 *     (K + 2) 2^-24 (|alpha| sum|a b| + |beta c|), then one rounding to `type`.
 *     In sum|a b| a subnormal code (below 2^-6 in E4M3, 2^-14 in E5M2, and not
 *     0) counts as the smallest normal one: the tensor cores align the products
 *     that they add by the codes' exponents.
 *     NaN codes, E5M2 infinities and non-finite scales give the values the
 *     formula gives.  The two scales of a pair are multiplied first, in FP32:
 *     a product beyond FLT_MAX is +-Inf (0 * Inf = NaN), one below 2^-126 has
 *     the bits of a subnormal number or is 0.  The bound is for elements whose
 *     pairs' products are zero or in between, and whose sum (before alpha) and
 *     its terms are.
 *   - Fast where both code arrays are 16-byte aligned with ld % 16 == 0 (or one
 *     row); others are first copied to aligned rows (in the workspace).
 * Arguments: 1 transA, 2 transB, 3 M, 4 N, 5 K, 6 alpha, 7 A, 8 B, 9 beta, 10 C,
 * 11 ldc, 12 D, 13 ldd, 14 type, 15 stream.  An unusable field of *A or *B
 * gives -7 or -8 (data or scale NULL where read, ld or lds too small, unknown
 * format or groups).  SGEMM_ERR_UNSUPPORTED: a dimension or leading dimension
 * >= 2^31, or a kernel forced that needs clusters of CTAs on a device without.
 */
int sgemm_fp8(char transA, char transB, int64_t M, int64_t N, int64_t K, float alpha,
              const sgemm_fp8_matrix_t *A, const sgemm_fp8_matrix_t *B,
              float beta, const void *C, int64_t ldc, void *D, int64_t ldd, int type,
              struct CUstream_st *stream);

/* What sgemm_fp8() would launch (sm_count as in sgemm_plan(); plan == NULL: -16). */
int sgemm_fp8_plan(char transA, char transB, int64_t M, int64_t N, int64_t K, float alpha,
                   const sgemm_fp8_matrix_t *A, const sgemm_fp8_matrix_t *B,
                   float beta, const void *C, int64_t ldc, const void *D, int64_t ldd, int type,
                   int sm_count, sgemm_plan_t *plan);

/*
 * Process-wide override of sgemm_fp8()'s choice of kernel, for tests and
 * benchmarks: variant = SGEMM_VARIANT_AUTO (0) restores it.  tile_n = 0 and
 * split = 0 keep the planner's own; a forced split (SHORT: 1, 2, 4 or 8) may
 * give a CTA no groups at all.  -1, -2, -3: an argument that names no kernel,
 * tile or split.
 */
int sgemm_fp8_set_override(int variant, int tile_n, int split);

/*
 * sgemm_fp8_quantize -- codes and scales of the rows x cols matrix X (type F32
 * or BF16), in groups of block_rows x block_cols elements.  For each group
 *     s = max(amax / top, 2^-126),  code = round(x * (1 / s)),
 * amax the largest finite |x| of the group, top the format's largest value,
 * the division and 1 / s rounded to FP32, codes to nearest with ties to even.
 * A NaN or infinite x becomes a NaN code.
 * Arguments: 1 rows, 2 cols, 3 X, 4 type, 5 ldx, 6 format, 7 block_rows,
 * 8 block_cols, 9 codes, 10 ldq, 11 scale, 12 lds, 13 stream.
 */
int sgemm_fp8_quantize(int64_t rows, int64_t cols, const void *X, int type, int64_t ldx, int format,
                       int block_rows, int block_cols, void *codes, int64_t ldq, float *scale, int64_t lds,
                       struct CUstream_st *stream);

/*
 * sgemm_fp8_rmsnorm -- for each row of X (and of the residual R when it is not
 * NULL), in FP32:
 *     h = x + r,   rstd = (mean(h^2) + eps)^(-1/2),   y = h * rstd * w,
 * and y in E4M3 with 1 x 128 groups as sgemm_fp8_quantize() gives them.
 *   - X, R, W (cols values), H and Y have `type`.  H (NULL: not wanted) receives
 *     h, Y (NULL: not wanted) y, rstd (NULL: not wanted) a float per row (NaN
 *     where cols is 0);
 *     codes NULL: no 8-bit output.  H may be X or R, with its row stride (-11
 *     otherwise).  The norm is of the unrounded sum.
 * Arguments: 1 rows, 2 cols, 3 type, 4 X, 5 ldx, 6 R, 7 ldr, 8 W, 9 eps, 10 H,
 * 11 ldh, 12 Y, 13 ldy, 14 codes, 15 ldq, 16 scale, 17 lds, 18 rstd, 19 stream.
 */
int sgemm_fp8_rmsnorm(int64_t rows, int64_t cols, int type, const void *X, int64_t ldx, const void *R, int64_t ldr,
                      const void *W, float eps, void *H, int64_t ldh, void *Y, int64_t ldy,
                      void *codes, int64_t ldq, float *scale, int64_t lds, float *rstd,
                      struct CUstream_st *stream);

/*
 * sgemm_fp8_rmsnorm_backward -- the gradients of y = h * rstd * w (the rounding
 * to 8 bits passed through):
 *     dx = rstd * (dy * w - h * rstd^2 * mean(dy * w * h)) + dh,
 *     dw = sum over the rows of dy * h * rstd,
 * dh being the gradient that reaches h past the norm (NULL: none).  dx is the
 * gradient of both x and r.  dY, H, W, dH and dX have `type`, rstd and dW are
 * FP32 (dW NULL: not wanted).  dX may be dY or dH, with its row stride (-13
 * otherwise).  cols <= 49152, else SGEMM_ERR_UNSUPPORTED.
 * Arguments: 1 rows, 2 cols, 3 type, 4 dY, 5 lddy, 6 H, 7 ldh, 8 W, 9 rstd,
 * 10 dH, 11 lddh, 12 dX, 13 lddx, 14 dW, 15 stream.
 */
int sgemm_fp8_rmsnorm_backward(int64_t rows, int64_t cols, int type, const void *dY, int64_t lddy,
                               const void *H, int64_t ldh, const void *W, const float *rstd,
                               const void *dH, int64_t lddh, void *dX, int64_t lddx, float *dW,
                               struct CUstream_st *stream);

/* The weights of `experts` experts: stored matrices one `stride` apart, groups of 128 x 128. */
typedef struct sgemm_fp8_experts_t {
    const void *data;      /* E4M3 codes; 16-byte aligned */
    int64_t ld;            /* row stride, a multiple of 16 */
    int64_t stride;        /* codes between consecutive experts, a multiple of 16 */
    const float *scale;
    int64_t lds;           /* row stride of the scales */
    int64_t stride_scale;  /* scales between consecutive experts */
} sgemm_fp8_experts_t;

/*
 * sgemm_fp8_moe -- a mixture-of-experts layer for a few tokens.  For token t:
 *     p = softmax(logits[t, :]),  J = the top_k largest logits (ties: lowest index),
 *     Y_t = sum_{e in J} c_e W2_e (silu(W1_e x_t) * (W3_e x_t)),
 * c_e = p_e, or p_e / sum_J p when renormalize is not 0; silu(a) = a / (1 + exp(-a)).
 *   - X: tokens x hidden, E4M3, 1 x 128 groups; gate (W1) and up (W3): inner x
 *     hidden per expert; down (W2): hidden x inner per expert.
 *   - The weights of the experts that some token chose are read once.  The
 *     products' sums are FP32; the inner values are kept as two 8-bit terms
 *     with a common scale (relative to the largest of 64 at most 2^-9.8 off,
 *     about as far as BF16) whatever `type` is.  The codes have no infinity:
 *     an inner value beyond FP32 counts as NaN.
 *   - An expert whose logit is -Inf is not chosen; a row whose logits are all
 *     -Inf gives zeros.  A row with a NaN or +Inf logit gives NaNs.  top_k == 0
 *     or inner == 0: zeros, and nothing is read.
 *   - tokens <= 64, experts <= 1024, top_k <= 16, hidden and inner multiples of 16
 *     (SGEMM_ERR_UNSUPPORTED otherwise; top_k <= experts, else -5).
 * Arguments: 1 tokens, 2 hidden, 3 inner, 4 experts, 5 top_k, 6 X, 7 logits,
 * 8 ldl, 9 renormalize, 10 gate, 11 up, 12 down, 13 Y, 14 ldy, 15 type, 16 stream.
 */
int sgemm_fp8_moe(int64_t tokens, int64_t hidden, int64_t inner, int64_t experts, int top_k,
                  const sgemm_fp8_matrix_t *X, const float *logits, int64_t ldl, int renormalize,
                  const sgemm_fp8_experts_t *gate, const sgemm_fp8_experts_t *up, const sgemm_fp8_experts_t *down,
                  void *Y, int64_t ldy, int type, struct CUstream_st *stream);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_FP8_H */
