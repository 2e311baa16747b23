/*
 * sgemm_linear.h -- the BF16 part of libsgemm: a layer's product with bias,
 * activation and residual, the gated form of a feed-forward block, and their
 * gradients.  What the backward pass needs of the values before the activation
 * can be kept as BF16 or as 8-bit codes with scales (sgemm_fp8.h).
 *
 * Conventions are those of sgemm.h and sgemm_fp8.h: row-major matrices, `ld` =
 * row stride in elements, device pointers owned by the caller, work enqueued on
 * `stream` of the current device, -(argument index) for an invalid argument
 * before anything is launched, SGEMM_ERR_* otherwise, workspace from the
 * library's stream-ordered pool.  Every call can be captured in a CUDA graph
 * after one eager call of this part on the device, which sets up its kernels.
 * Results are deterministic: no sum's order depends on scheduling.
 *
 * Matrices are BF16 where nothing else is said.  Inputs may start at any
 * element and have any row stride; they are read fastest where their first
 * element is 16-byte aligned and ld is a multiple of 8 (others are first copied
 * to aligned rows in the workspace), and outputs are written fastest there too.
 * No output may overlap an input or another output unless its call says so.
 *
 * Products are summed on the tensor cores in FP32: an element is at most
 * (K + 2) 2^-24 sum|a b| off before its activation and its one rounding to the
 * output's type.  For FP32 outputs and the scales of 8-bit values long sums are
 * made of several, which keeps random sums of up to 16384 terms within 1e-6; for
 * BF16 outputs parts of up to 16384 terms are summed whole, which are up to
 * 1e-4 too small where the terms have one sign.  So a result's last bits can depend on the other outputs
 * that are wanted, as they can on the sizes.
 */
#ifndef SGEMM_LINEAR_H
#define SGEMM_LINEAR_H

#include "sgemm_fp8.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Activations, in FP32.  Phi is the standard normal distribution's integral.  A
 * NaN gives NaN, and so does -infinity but in RELU (a product of infinity and
 * 0); derivatives at the infinities are their limits.
 */
enum sgemm_activation {
    SGEMM_ACT_NONE = 0,      /* a */
    SGEMM_ACT_RELU = 1,      /* a where a > 0, 0 where a <= 0; derivative 0 at 0 */
    SGEMM_ACT_SILU = 2,      /* a / (1 + exp(-a)) */
    SGEMM_ACT_GELU = 3,      /* a Phi(a) */
    SGEMM_ACT_GELU_TANH = 4  /* a / (1 + exp(-2 u)), u = sqrt(2 / pi) (a + 0.044715 a^3): a (1 + tanh u) / 2 */
};

/* Kernel variants of this part (sgemm_plan_t.variant). */
enum sgemm_linear_variant {
    SGEMM_VARIANT_LINEAR_PAIR = 40,  /* CTA pairs, 256 x tile_n tiles (tile_n 64, 128 or 256), 64 k per tile; with split_k > 1
                                        the K tiles of a tile are shared and a second kernel adds the sums */
    SGEMM_VARIANT_LINEAR_SHORT = 41  /* one CTA per tile_n x 128 tile (tile_n 16, 32, 64 or 128 rows, 128 columns), K
                                        shared by a cluster of split_k CTAs */
};

/*
 * A matrix that is kept for the backward pass.  scale NULL: BF16.  Otherwise
 * E4M3 codes with an FP32 scale per group of 128 elements of a row, as
 * sgemm_fp8_quantize() gives them for the FP32 values:
 *     value(r, c) = code(r, c) * scale[r * lds + c / 128].
 */
typedef struct sgemm_kept_t {
    void *data;
    int64_t ld;
    float *scale;
    int64_t lds;  /* row stride of the scales (not read without them) */
} sgemm_kept_t;

/*
 * sgemm_linear -- a layer:
 *     A = X W^T + bias,   Y = act(A) + R
 * for `tokens` rows of `inputs` values: X is tokens x inputs, W outputs x
 * inputs, bias has `outputs` values (NULL: none), R (NULL: none) and Y are
 * tokens x outputs.  Y has `type` (enum sgemm_type), everything else is BF16.
 * `kept` (NULL: not wanted) receives A, rounded from FP32.  Y may be R, with its
 * row stride, when it is BF16.  inputs == 0: A is the bias (or 0).
 * Arguments: 1 tokens, 2 inputs, 3 outputs, 4 X, 5 ldx, 6 W, 7 ldw, 8 bias,
 * 9 activation, 10 R, 11 ldr, 12 kept, 13 Y, 14 ldy, 15 type, 16 stream.
 * SGEMM_ERR_UNSUPPORTED: a dimension or leading dimension >= 2^31 - 1024.
 */
int sgemm_linear(int64_t tokens, int64_t inputs, int64_t outputs, const void *X, int64_t ldx, const void *W, int64_t ldw,
                 const void *bias, int activation, const void *R, int64_t ldr, const sgemm_kept_t *kept,
                 void *Y, int64_t ldy, int type, struct CUstream_st *stream);

/*
 * sgemm_linear_backward -- the gradients of a layer from that of its output:
 *     dA = dY * act'(A),  dX = dA W,  dW = dA^T X,  dbias = sum over the tokens of dA
 * (R's gradient is dY itself).  A is `kept` as sgemm_linear() left it, X a
 * matrix or one kept in 8 bits.  dX, dW and dbias may each be NULL (not
 * wanted); W is read for dX only, X for dW only, A only where there is an
 * activation.  dX is BF16, dW has `dw_type`, dbias is FP32 (the sum of FP32
 * values of dA).  dA is rounded to BF16 for the products where there is an
 * activation, and the values of an 8-bit X are: the tensor cores read BF16.
 * Arguments: 1 tokens, 2 inputs, 3 outputs, 4 dY, 5 lddy, 6 X, 7 W, 8 ldw,
 * 9 activation, 10 kept, 11 dX, 12 lddx, 13 dW, 14 lddw, 15 dw_type, 16 dbias, 17 stream.
 */
int sgemm_linear_backward(int64_t tokens, int64_t inputs, int64_t outputs, const void *dY, int64_t lddy,
                          const sgemm_kept_t *X, const void *W, int64_t ldw, int activation, const sgemm_kept_t *kept,
                          void *dX, int64_t lddx, void *dW, int64_t lddw, int dw_type, float *dbias,
                          struct CUstream_st *stream);

/*
 * sgemm_gated -- the first half of a gated feed-forward block:
 *     A = X G^T,  B = X U^T,  H = act(A) * B
 * in one kernel: X is tokens x inputs, G (gate) and U (up) outputs x inputs, H
 * tokens x outputs.  kept_gate and kept_up (both NULL: not wanted; both BF16 or
 * both 8-bit) receive A and B, rounded from FP32; H is of the unrounded values.
 * Arguments: 1 tokens, 2 inputs, 3 outputs, 4 X, 5 ldx, 6 gate, 7 ldg, 8 up,
 * 9 ldu, 10 activation, 11 kept_gate, 12 kept_up, 13 H, 14 ldh, 15 stream.
 */
int sgemm_gated(int64_t tokens, int64_t inputs, int64_t outputs, const void *X, int64_t ldx, const void *gate, int64_t ldg,
                const void *up, int64_t ldu, int activation, const sgemm_kept_t *kept_gate, const sgemm_kept_t *kept_up,
                void *H, int64_t ldh, struct CUstream_st *stream);

/*
 * sgemm_gated_backward -- its gradients from that of H:
 *     dA = dH * B * act'(A),  dB = dH * act(A),
 *     dX = dA G + dB U,  dG = dA^T X,  dU = dB^T X,
 * A and B as sgemm_gated() kept them, X a matrix or one kept in 8 bits.  dX,
 * the pair dG and dU, and H may each be NULL (not wanted): H receives act(A) * B
 * of the kept values, which the layer behind needs for its weight gradient.  dX
 * and H are BF16, dG and dU have `dw_type`.  dA, dB and the values of an 8-bit X
 * are rounded to BF16 for the products.
 * Arguments: 1 tokens, 2 inputs, 3 outputs, 4 dH, 5 lddh, 6 X, 7 gate, 8 ldg,
 * 9 up, 10 ldu, 11 activation, 12 kept_gate, 13 kept_up, 14 dX, 15 lddx, 16 dG,
 * 17 lddg, 18 dU, 19 lddu, 20 dw_type, 21 H, 22 ldh, 23 stream.
 */
int sgemm_gated_backward(int64_t tokens, int64_t inputs, int64_t outputs, const void *dH, int64_t lddh,
                         const sgemm_kept_t *X, const void *gate, int64_t ldg, const void *up, int64_t ldu, int activation,
                         const sgemm_kept_t *kept_gate, const sgemm_kept_t *kept_up, void *dX, int64_t lddx,
                         void *dG, int64_t lddg, void *dU, int64_t lddu, int dw_type, void *H, int64_t ldh,
                         struct CUstream_st *stream);

/*
 * The launch this part makes for a product of `rows` x `cols` over `K` of
 * aligned matrices (gated != 0: for sgemm_gated() with `cols` outputs; kept8 !=
 * 0: values are kept in 8 bits); sm_count as in sgemm_plan().  Arguments: 1 rows, 2 cols, 3 K,
 * 4 gated, 5 kept8, 6 sm_count, 7 plan.
 */
int sgemm_linear_plan(int64_t rows, int64_t cols, int64_t K, int gated, int kept8, int sm_count, sgemm_plan_t *plan);

/*
 * Process-wide override of this part's choice of kernel, for tests and
 * benchmarks: variant = SGEMM_VARIANT_AUTO (0) restores it.  tile_n = 0 and
 * split = 0 keep the planner's own; a forced split (SHORT: 1, 2, 4 or 8; PAIR: 1
 * to 32, where the call can share K) may give a CTA of the short-side kernel no
 * work at all.  A tile that a call cannot use (64 columns where a gated pair or
 * 8-bit values want more, 128 rows of a gated short one) is left to the
 * planner.  -1, -2, -3: an argument that names no kernel, tile or split.
 */
int sgemm_linear_set_override(int variant, int tile_n, int split);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_LINEAR_H */
