/*
 * serve/qrow_kv8.h -- C-ABI of libqrow.so, serving part 2: a paged cache of
 * keys and values in 8 bits with one fp32 scale per block of tokens and head,
 * and causal attention over it.
 *
 * Conventions are those of qrow.h (device pointers, 16-byte aligned unless
 * noted; asynchronous calls on `stream`; 0 or a negative QR_E* code with
 * nothing launched on failure; nothing allocated: scratch memory is the
 * caller's `workspace`). Nothing is copied to the host, so every call can be
 * captured into a graph and replayed with other lengths in the same arrays.
 *
 * Cache layout (this library's): a block holds block_tokens consecutive
 * tokens of one sequence for all heads.
 *   k   [n_blocks][n_heads][block_tokens][head_dim] codes
 *   v   [n_blocks][n_heads][block_tokens/32][head_dim/2][4][2][8] codes: within
 *       a group of 32 tokens, byte (d/2)*64 + (t/8)*16 + (d%2)*8 + t%8 holds
 *       channel d of token t (eight tokens of one channel side by side, as the
 *       matrix instructions take them)
 *   kd, vd  [n_blocks][n_heads] scales, never negative; a code stands for
 *       scale * code.
 * Sequence s: its token p lies in block table[s * table_width + p /
 * block_tokens], at p % block_tokens.
 *
 * Sequences and rows: a call brings n_tok rows; sequence s owns the rows
 * cu[s] .. cu[s+1]-1 (cu: int32 [n_seq+1], not descending), which are its
 * LAST cu[s+1]-cu[s] tokens: row cu[s]+i is the token at position
 * kv_len[s] - (cu[s+1]-cu[s]) + i, kv_len[s] (int32 [n_seq]) counting the
 * sequence's tokens with the new ones. Rows before cu[0] and from cu[n_seq] on
 * belong to no sequence: they are not read and what the call would write there
 * is left as it was (parts of a batch, padded batches).
 *
 * What is not a token: a position below 0, one behind the table's width, one
 * whose table entry lies outside 0..n_blocks-1 (an evicted or unassigned
 * block), is absent: not written, read back as 0, not attended to. cu is
 * clamped to 0..n_tok. So no content of cu, kv_len or table makes a kernel
 * leave its buffers. cu, kv_len and table need 4-byte alignment.
 */
#ifndef QROW_KV8_H
#define QROW_KV8_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    int8_t *k, *v;         /* codes                                          */
    float *kd, *vd;        /* scales                                         */
    int64_t n_blocks;      /* 0 .. 2^31-1                                    */
    int64_t n_heads;       /* key/value heads, 1..1024                       */
    int64_t head_dim;      /* 64, 128 or 256                                 */
    int64_t block_tokens;  /* 32, 64 or 128                                  */
} qr_kv8;

/* Bytes of k (and of v): n_blocks * n_heads * block_tokens * head_dim; 0 for
 * an invalid description (the pointers are not looked at). */
size_t qr_kv8_code_bytes(const qr_kv8 *c);

/*
 * qr_kv8_append -- writes the rows' keys and values into their blocks.
 *  src      QR_F32 or QR_BF16: element type of k and v.
 *  k, v     [n_tok, n_heads, head_dim], token t at element t * k_stride (t *
 *           v_stride), a multiple of 8, at least n_heads * head_dim.
 * Per block and head, for k and v apart: amax = max |x| of the new tokens in
 * the block, cand = amax / 127 (0 if 1 / cand is not finite). In a block whose
 * first token is new the scale becomes cand. Otherwise scale = max(old, cand),
 * and where it grew the codes c of the tokens before become rint(c * (old /
 * scale)). The new codes are rint(x * (1 / scale)), clamped to -127..127 (0
 * where the scale is 0). Every operation is rounded
 * to fp32 once. A block that gets an infinity or a NaN gets scale NaN and zero
 * codes for its new tokens, and stays so until its first token is written again: the
 * rows that attend to it are NaN. Writing the same rows again leaves
 * the same bytes. Two rows must not fall on the same token of the same block
 * and no two workgroups on the same block: a block that is written belongs to
 * one sequence and stands once in its row of the table; blocks that are only
 * read may be shared. In a block whose first token is not among the rows, the
 * tokens before them are taken to be there already.
 * Limits: n_seq, n_tok and table_width < 2^31, and what one launch holds:
 * (n_tok / block_tokens + 2 * n_seq) * n_heads < 2^24. n_tok == 0 or n_seq == 0
 * is a no-op.
 */
int qr_kv8_append(const qr_kv8 *c, int src, const void *k, const void *v,
                  int64_t k_stride, int64_t v_stride, int64_t n_tok,
                  int64_t n_seq, const int32_t *cu, const int32_t *kv_len,
                  const int32_t *table, int64_t table_width, void *stream);

/*
 * qr_kv8_read -- the decoder: the values of the same rows, scale * code
 * rounded to fp32 and then to dst (QR_F32 or QR_BF16), into k and v [n_tok,
 * n_heads, head_dim] (strides and limits as in qr_kv8_append), which must not
 * overlap. With cu counting whole sequences it returns the whole cache of each.
 */
int qr_kv8_read(const qr_kv8 *c, int dst, void *k, void *v, int64_t k_stride,
                int64_t v_stride, int64_t n_tok, int64_t n_seq,
                const int32_t *cu, const int32_t *kv_len, const int32_t *table,
                int64_t table_width, void *stream);

/* Device scratch bytes that qr_attention_kv8 needs for this call (0 if none:
 * then workspace may be NULL; 0 for invalid shapes too, which the call
 * reports). */
size_t qr_attention_kv8_workspace_bytes(const qr_kv8 *c, int64_t n_q_heads,
                                        int64_t n_tok, int64_t n_seq,
                                        int64_t table_width);

/*
 * qr_attention_kv8 -- causal attention of the rows over their sequences:
 *   out[t][h] = sum_j softmax_j(scale * q[t][h] . K[j][h/g]) V[j][h/g],
 * g = n_q_heads / n_heads, over the positions j of the row's sequence up to
 * its own, p, and above p - window if window > 0. A row that sees no token
 * gets zeros.
 *  src      QR_F32 or QR_BF16: element type of q and out.
 *  q, out   [n_tok, n_q_heads, head_dim], token t at element t * q_stride (t *
 *           out_stride), a multiple of 8, at least n_q_heads * head_dim. They
 *           must not overlap (refused; parts of one buffer may lie side by
 *           side).
 *  n_q_heads  a positive multiple of n_heads (g: see the limits).
 *  scale    finite factor of the scores (1 / sqrt(head_dim) as a rule).
 *  window   0: all positions up to the row's own; else the last `window`.
 *  workspace  at least qr_attention_kv8_workspace_bytes(...) bytes, 256-byte
 *           aligned, not shared by calls that may overlap; contents do not
 *           matter and are clobbered.
 * Limits: 1 <= g <= 1024; n_tok * n_q_heads < 2^31; n_seq, n_tok and
 * table_width < 2^31, and what one launch holds: (n_tok * g / 128 + n_seq) *
 * n_heads < 2^24, with 16 in place of 128 where the sequences have up to 32
 * rows (tokens times g) on average.
 * Numerics: the codes are exact as fp16 matrix operands. bf16 queries are
 * exact there too (scaled by a power of two per row; elements below 2^-28 of
 * the row's largest lose bits); fp32 ones are split into two fp16 parts (22
 * bits). Scores, maxima, sums and outputs are fp32. The weights exp(s - max)
 * enter the second product in fp16 (bf16 rows; 2^-11 each) or as two fp16 parts
 * (fp32 rows; 2^-22), and to 2^-31 of the largest weight where those are
 * smaller, whatever the scales of the blocks (up to factors of 2^70 between
 * them); their sum is taken in fp32. Sums are held undivided, with weights of
 * up to 2^15: values above 2^112 / (tokens that the row sees) may give
 * infinities. The result does not depend on timing; which kernel and how many
 * splits of the tokens a call takes goes by its shapes (n_tok, n_seq, heads,
 * table_width): a table no wider than its sequences need is faster where they
 * are short, and gives the same result up to the order of sums. A batch that mixes
 * whole prompts with single tokens is right in one call and faster in two:
 * cu + s, kv_len + s and table + s * table_width describe the sequences from
 * s on, whose rows keep their numbers.
 */
int qr_attention_kv8(const qr_kv8 *c, int src, const void *q, int64_t q_stride,
                     int64_t n_q_heads, int64_t n_tok, int64_t n_seq,
                     const int32_t *cu, const int32_t *kv_len,
                     const int32_t *table, int64_t table_width, float scale,
                     int64_t window, void *out, int64_t out_stride,
                     void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif
