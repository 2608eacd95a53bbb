/*
 * serve/qrow_moe.h -- C-ABI of libqrow.so, serving part 4: a mixture of experts
 * in 8 bits. The router (which experts a token meets, with which weights) and
 * the experts of a few tokens: gated products, their weighted sum and the
 * residual.
 *
 * Conventions are those of qrow_kv8.h: nothing is copied to the host, so every
 * call can be captured into a graph and replayed with other tokens and other
 * choices in the same arrays; scratch memory is the caller's `workspace`
 * (256-byte aligned, not shared by calls that may overlap; contents do not
 * matter and are clobbered).
 */
#ifndef QROW_MOE_H
#define QROW_MOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define QR_MOE_MAX_EXPERTS 1024
#define QR_MOE_MAX_TOP_K 64
#define QR_MOE_MAX_PAIRS 8192   /* n_tok * top_k of one qr_moe_i8 call */

/* Scores of qr_moe_route. */
enum {
    QR_SCORE_SOFTMAX = 0,   /* over all experts */
    QR_SCORE_SIGMOID = 1    /* each by itself   */
};

/* Device scratch bytes that qr_moe_route needs (0 for invalid shapes too, which
 * the call reports). */
size_t qr_moe_route_workspace_bytes(int64_t n_experts, int64_t n_tok,
                                    int64_t n_in);

/*
 * qr_moe_route -- the top_k experts of every token and their weights.
 *  src, x   QR_F32 or QR_BF16; [n_tok, n_in], token t at element t * x_stride
 *           (>= n_in, any alignment of the rows).
 *  wtype, w QR_F32 or QR_BF16; the router's rows [n_experts, n_in].
 *  bias     fp32 [n_experts] or NULL: added to the scores for the choice alone.
 *           An expert whose bias is -infinity is never chosen.
 *  score    QR_SCORE_SOFTMAX or QR_SCORE_SIGMOID of the logits x . w[e].
 *  renorm   nonzero: a token's weights are divided by their sum (all zero where
 *           that is zero).
 *  factor   finite; multiplies the weights at the end.
 *  ids      int32 [n_tok, top_k], written: the experts with the largest score +
 *           bias, largest first, the lower index first among equals, a NaN
 *           before everything. -1 behind the experts that can be chosen.
 *  weights  fp32 [n_tok, top_k], written: their scores (without bias); 0 beside
 *           an id of -1.
 *  workspace 256-byte aligned, qr_moe_route_workspace_bytes bytes, of one call at
 *           a time. It, ids and weights overlap nothing else (not looked at).
 * Logits are sums in 64 bits of exact products, and scores, choice and weights
 * follow in 64 bits: the choice does not depend on the launch shape unless two
 * scores agree to some 2^-50. Weights are rounded to fp32 at the end. (For many
 * bf16 tokens, an expert that fp32 sums with their error bound already leave out
 * of a token's choice gets no 64-bit sum; choice and weights are the same.)
 * Limits: 1 <= n_experts <= QR_MOE_MAX_EXPERTS, 1 <= top_k <= min(n_experts,
 * QR_MOE_MAX_TOP_K), 1 <= n_in <= 131072, n_tok < 2^22. n_tok == 0 is a no-op.
 */
int qr_moe_route(int src, const void *x, int64_t x_stride, int wtype,
                 const void *w, const float *bias, int64_t n_experts,
                 int64_t n_tok, int64_t n_in, int64_t top_k, int score,
                 int renorm, float factor, int32_t *ids, float *weights,
                 void *workspace, size_t workspace_bytes, void *stream);

/* The experts' weights: rows of codes with a scale each (qr_quantize_rows_i8).
 * gate and up hold n_mid rows of qr_i8_row_bytes(n_in) bytes per expert, down
 * n_in rows of qr_i8_row_bytes(n_mid) bytes; expert e's rows of gate and up
 * begin at row e * expert_rows (n_mid where each is a tensor of its own,
 * 2 * n_mid where an expert's gate and up rows lie behind each other), of down
 * at row e * n_in. */
typedef struct {
    const int8_t *gate, *up, *down;
    const float *gated, *upd, *downd;   /* scales, one per row, the same rows */
    int64_t n_experts;                  /* 1..QR_MOE_MAX_EXPERTS              */
    int64_t n_in;                       /* 1..QR_I8_MAX_IN                    */
    int64_t n_mid;                      /* 1..QR_I8_MAX_IN                    */
    int64_t expert_rows;                /* >= n_mid                           */
} qr_moe;

/* Device scratch bytes that qr_moe_i8 needs (0 for invalid shapes too, which
 * the call reports). */
size_t qr_moe_i8_workspace_bytes(const qr_moe *m, int64_t n_tok,
                                 int64_t top_k);

/*
 * qr_moe_i8 -- the experts of a few tokens:
 *   y[t] = sum_j weights[t][j] * down_e(act(gate_e(x[t])) * up_e(x[t])) + residual[t],
 *   e = ids[t][j].
 *  x, xd    activation rows [n_tok, qr_i8_row_bytes(n_in)] and their scales
 *           (qr_norm_rows_i8, qr_quantize_rows_i8).
 *  ids      int32 [n_tok, top_k]. An id outside 0..n_experts-1 (-1 of a padded
 *           token, an expert held elsewhere) is no expert: its weight is not
 *           looked at and it adds nothing. The same expert twice counts twice.
 *  weights  fp32 [n_tok, top_k].
 *  act      QR_ACT_* of qrow_i8.h (QR_ACT_SILU as a rule).
 *  residual NULL, or [n_tok, n_in] of type dst, token t at element t *
 *           residual_stride (>= n_in). It may be y itself (the same pointer and
 *           stride); otherwise the two must not overlap (refused).
 *  dst, y   QR_F32 or QR_BF16; [n_tok, n_in], token t at element t * y_stride
 *           (>= n_in), written completely. y overlaps no other input (refused
 *           for x, xd, ids and weights; the experts' weights are not looked at).
 *  workspace 256-byte aligned, qr_moe_i8_workspace_bytes bytes, of one call at a
 *           time; overlaps nothing (refused for x, xd, ids, weights, residual and y).
 * Steps: gate and up products as in qr_matmul_i8, in fp32; act(gate) * up in 64
 * bits, rounded to fp32; these hidden rows are held in 8 bits with one fp32
 * scale per 64 channels (max / 127, codes rint(h * (127 / max)), the rule of
 * the Q8_K blocks: infinities and NaN give a scale of NaN). The down product
 * multiplies codes exactly; sums over blocks, its scales, the experts' weights
 * and the residual are fp32, an expert's terms in an order that n_tok, top_k
 * and n_mid fix together with the number of distinct experts met, a token's
 * experts in the order of their slots.
 * The operator is made for few tokens, whose time is that of the weights' way
 * through the chip. Gate and up pass once for up to 64 tokens of an expert. Down
 * passes once for up to 512 pairs of the call (whole tokens: 512 / top_k of them)
 * and up to 16 of an expert (32 where there are many and n_mid is 4096 or more).
 * More are right, up to the limit, and read the weights again: 128 tokens of 8
 * experts each read down twice, 1024 of them up to 16 times, however few of an
 * expert's pairs are among them.
 * Limits: 1 <= top_k <= QR_MOE_MAX_TOP_K, n_tok * top_k <= QR_MOE_MAX_PAIRS,
 * and those of qr_moe. n_tok == 0 is a no-op.
 */
int qr_moe_i8(const qr_moe *m, const int8_t *x, const float *xd,
              const int32_t *ids, const float *weights, int64_t n_tok,
              int64_t top_k, int act, const void *residual,
              int64_t residual_stride, int dst, void *y, int64_t y_stride,
              void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif
