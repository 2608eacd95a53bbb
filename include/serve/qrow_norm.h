/*
 * serve/qrow_norm.h -- C-ABI of libqrow.so, serving part 3: a root-mean-square
 * norm with the residual's addition in front and 8-bit rows (qrow_i8.h) behind,
 * in one pass: what stands between two 8-bit products of a layer.
 *
 * Conventions are those of qrow_i8.h.
 */
#ifndef QROW_NORM_H
#define QROW_NORM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/*
 * qr_norm_rows_i8 -- per row of n values:
 *   s = x + residual                     (x alone without a residual)
 *   y = s / sqrt(mean(s^2) + eps) * weight
 *   scale = max |y| / 127, codes = rint(y * (127 / max |y|))
 *  src      QR_F32 or QR_BF16: element type of x, residual, sum and y.
 *  x, residual, sum, y   [n_rows, n], rows x_stride, residual_stride, sum_stride
 *           and y_stride elements apart (each >= n, any alignment of the rows).
 *           residual and sum are both given or both NULL: sum receives s. y is
 *           NULL or receives the normed rows.
 *  wtype, weight   QR_F32 or QR_BF16 and [n] of it, or NULL for ones.
 *  eps      finite, >= 0.
 *  codes, scales   [n_rows, qr_i8_row_bytes(n)] and [n_rows], written as
 *           qr_quantize_rows_i8 writes them.
 * Steps: s is rounded to fp32 and then to src, and the norm goes on from what
 * sum holds; the mean and f = 1 / sqrt(mean + eps) are taken in 64 bits; y is
 * s * f rounded to fp32, times the weight rounded to fp32 (and to src in y);
 * the codes are made from the fp32 y by the rule of qr_quantize_rows_i8. So the
 * codes are the same whatever the order of the sum, but for an f that the last
 * bits of a 64-bit sum move across a rounding. A row that holds an infinity or
 * a NaN, before or behind the norm, gets scale NaN and zero codes; so does an
 * all-zero row with eps 0.
 * sum may be x or residual, and y may be x, residual or neither (the same
 * pointer and stride: in place); apart from that no output may overlap an input
 * or another output (refused).
 * Limits: 1 <= n <= QR_I8_MAX_IN; n_rows < 2^24, and < 2^22 where n > 8192.
 * n_rows == 0 is a no-op.
 */
int qr_norm_rows_i8(int src, const void *x, int64_t x_stride,
                    const void *residual, int64_t residual_stride, int wtype,
                    const void *weight, double eps, int64_t n_rows, int64_t n,
                    void *sum, int64_t sum_stride, void *y, int64_t y_stride,
                    int8_t *codes, float *scales, void *stream);

#ifdef __cplusplus
}
#endif
#endif
