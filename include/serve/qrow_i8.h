/*
 * serve/qrow_i8.h -- C-ABI of libqrow.so, serving part 1: rows of 8-bit codes
 * with ONE fp32 scale each, and their product. Activation rows carry a scale
 * per token, weight rows a scale per output channel, so that the whole sum of
 * an output is an exact integer and the two scales are applied once.
 *
 * These are the formats of a projection kept at 8 bits, beside the packed
 * 4- to 6-bit rows and the Q8_K activation blocks of qrow.h.
 *
 * Conventions are those of qrow.h (device pointers, 16-byte aligned;
 * asynchronous calls on `stream`; 0 or a negative QR_E* code with nothing
 * launched on failure; nothing allocated), with one difference: activation
 * and output rows may be strided.
 *
 * Row layout: int8 codes[qr_i8_row_bytes(n)], the first n of them the row's,
 * zeros behind them up to the next multiple of 128; the scales are a separate
 * fp32 array. A row stands for scale * code.
 */
#ifndef QROW_I8_H
#define QROW_I8_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define QR_I8_MAX_IN 131072   /* longest row: 127 * 127 * n fits in 31 bits */

/* Bytes of one row of codes: n_per_row rounded up to a multiple of 128; 0 if
 * n_per_row is not in 1..QR_I8_MAX_IN. */
size_t qr_i8_row_bytes(int64_t n_per_row);

/*
 * qr_quantize_rows_i8 -- one scale per row, for tokens and channels alike.
 *  src      QR_F32 or QR_BF16 (enum of qrow.h): element type of x.
 *  x        [n_rows, n_per_row], row r at element r * x_stride
 *           (x_stride >= n_per_row, any alignment of the rows).
 *  codes    [n_rows, qr_i8_row_bytes(n_per_row)], written completely (zeros
 *           behind a row's codes).
 *  scales   [n_rows] fp32, written.
 * Per row: amax = max |x|; scale = amax / 127; code = rint(x * (127 / amax)),
 * in -127..127; every operation rounded to fp32 once, the rule of the Q8_K
 * blocks. An all-zero row (or one whose 127 / amax is not finite) gets scale
 * 0 and zero codes. A row that holds an infinity or a NaN gets scale NaN and
 * zero codes, so that the outputs made from it, and no others, are NaN.
 * Limits: 1 <= n_per_row <= QR_I8_MAX_IN; n_rows < 2^24. n_rows == 0 is a
 * no-op.
 */
int qr_quantize_rows_i8(int src, const void *x, int64_t n_rows,
                        int64_t n_per_row, int64_t x_stride, int8_t *codes,
                        float *scales, void *stream);

/*
 * qr_matmul_i8 -- y[t][r] = xd[t] * wd[r] * sum_k x[t][k] * w[r][k] + bias[r].
 *  w, wd    weight rows [n_out, qr_i8_row_bytes(n_in)] and their scales.
 *  x, xd    activation rows [n_tok, qr_i8_row_bytes(n_in)] and their scales.
 *  bias     fp32 [n_out], or NULL for none.
 *  dst, y   QR_F32 or QR_BF16; y is [n_tok, n_out], token t at element
 *           t * y_stride (y_stride >= n_out), written completely; what lies
 *           between n_out and y_stride is left as it was.
 * The sum is exact (int32); it is converted to fp32, multiplied with xd[t],
 * then wd[r], and the bias added, each rounded to fp32 once, then rounded to
 * dst: within 4 * 2^-24 of the magnitude |product| + |bias| before that last
 * rounding (2^-149 more where the product is subnormal; infinite only where
 * the product or the output is). The result does not depend on the launch
 * shape. Codes are read as they are: -128 is allowed in codes made elsewhere up
 * to n_in = 131071.
 * Codes behind n_in up to the row's end must be zero, as qr_quantize_rows_i8
 * writes them.
 * Limits: 1 <= n_in <= QR_I8_MAX_IN; n_out, n_tok < 2^31 - 256, and what one
 * launch holds: n_out <= 16 * (2^23 - 1) with up to 16 tokens, else
 * ceil(n_out / 256) * ceil(n_tok / 256) < 2^24. n_out == 0 or n_tok == 0 is a
 * no-op.
 */
int qr_matmul_i8(const int8_t *w, const float *wd, const int8_t *x,
                 const float *xd, const float *bias, int64_t n_out,
                 int64_t n_tok, int64_t n_in, int dst, void *y,
                 int64_t y_stride, void *stream);

/* Activations of qr_matmul_i8_ex and of the experts in qrow_moe.h. */
enum {
    QR_ACT_NONE = 0,
    QR_ACT_RELU = 1,
    QR_ACT_SILU = 2,       /* x / (1 + exp(-x))                              */
    QR_ACT_GELU = 3,       /* x / 2 * (1 + erf(x / sqrt 2))                  */
    QR_ACT_GELU_TANH = 4   /* x / 2 * (1 + tanh(sqrt(2 / pi) (x + 0.044715 x^3))) */
};

/* What qr_matmul_i8_ex does with its products. */
typedef struct {
    int64_t act;               /* QR_ACT_*                                       */
    const int8_t *up;          /* a second set of weight rows, or NULL           */
    const float *upd;          /* its scales                                     */
    const float *up_bias;      /* and its bias, or NULL                          */
    const void *residual;      /* added at the end, of type dst, or NULL         */
    int64_t residual_stride;   /* token t at element t * residual_stride         */
} qr_i8_epilogue;

/*
 * qr_matmul_i8_ex -- qr_matmul_i8 with an epilogue:
 *   y[t][r] = act(p(w)) * p(up) + residual[t][r],
 * p(w) = xd[t] * wd[r] * sum_k x[t][k] * w[r][k] + bias[r] as in qr_matmul_i8
 * and p(up) the same product with up [n_out, qr_i8_row_bytes(n_in)], upd and
 * up_bias (left out where up is NULL): a gated projection in one pass over x,
 * without the two products in memory.
 * epilogue   NULL: qr_matmul_i8.
 * residual   [n_tok, n_out] of type dst, rows residual_stride >= n_out elements
 *            apart. It may be y itself (the same pointer and stride: added in
 *            place); otherwise the two must not overlap (refused). y must not
 *            overlap the other operands either (not looked at).
 * Every step is in fp32: the two products each as in qr_matmul_i8; the
 * activation, within 8 * 2^-24 of |p| (and 2^-110 where exp overflows) for the
 * fp32 p = p(w) it is given, and where its result a is 2^-110 or more in
 * magnitude within 8 * 2^-24 (SILU), (36 + 2 p^2) * 2^-24 (GELU) or
 * (8 + 5 t) * 2^-24 (GELU_TANH, t = 2 sqrt(2 / pi) |p + 0.044715 p^3|) of |a|;
 * the gate's product and the residual's addition rounded once each; then the
 * rounding to dst.
 * Limits: those of qr_matmul_i8, with up and more than 16 tokens those for
 * 2 * n_out; act one of the above.
 */
int qr_matmul_i8_ex(const int8_t *w, const float *wd, const int8_t *x,
                    const float *xd, const float *bias,
                    const qr_i8_epilogue *epilogue, int64_t n_out,
                    int64_t n_tok, int64_t n_in, int dst, void *y,
                    int64_t y_stride, void *stream);

#ifdef __cplusplus
}
#endif
#endif
