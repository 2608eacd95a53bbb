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

#ifdef __cplusplus
}
#endif
#endif
