/*
 * pkv_window.h - attention over the paged KV cache behind a sliding window,
 * with a few first tokens (sinks) that stay visible: for decode (one new
 * token per sequence) and for prefill chunks, over contexts of up to
 * PKV_MAX_LONG_CONTEXT tokens.
 *
 * The query at position p sees token t when
 *   t <= p  and  (p - t < window  or  t < sinks),
 * window >= 1 (so a token always sees itself) and sinks >= 0. A window of the
 * whole context (any value >= max_seq_len) is full causal attention.
 *
 * Geometry, pools, block tables and dtypes are those of pkv.h and
 * pkv_prefill.h; a handle created with PKV_FLAG_LONG_CONTEXT raises
 * max_seq_len. Lists of int32 (seq_lens, cu_tokens, start_pos, rope_positions)
 * need 4-byte alignment only. Pages that hold no visible token are never
 * read and their block-table entries may hold anything (-1 after
 * pkv_sched_release). Inside a page that is read, tokens that no query of the
 * sequence sees may hold any bits, NaN and infinities included; visible K and
 * V are finite.
 *
 * An invalid page id is flagged and its tokens are skipped (weight 0); a row
 * all of whose visible tokens are skipped is 0.
 *
 * Arithmetic: BF16 products summed in FP32 on the tensor cores, softmax
 * statistics in FP32; probabilities and rotated queries enter their products
 * as the sum of three BF16 terms (24 bits), so the result is that of FP32
 * arithmetic on BF16 inputs.
 */
#ifndef PKV_WINDOW_H
#define PKV_WINDOW_H

#include <stdint.h>

#include "pkv.h"
#include "pkv_axes.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Decode attention: out[b][h][:] = sum_t softmax_t(q[b][h] . K_t / 8) V_t over
 * the tokens visible from position seq_lens[b] - 1 (q BF16 [batch][32][64],
 * out FP32 [batch][32][64]). Every visible page tile is read once, for the 4
 * query heads of its KV head.
 *
 * seq_lens[b] == 0 marks a padding row: nothing of it is read or written and
 * it is not flagged. A seq_len outside [0, max_seq_len] is skipped and
 * flagged.
 *
 * num_splits as in pkv_decode_attention, over the visible pages of a sequence
 * (0: the library chooses from the batch, the window and the handle).
 *
 * rope (NULL: none): queries are rotated in FP32 by pkv_axes.h's rule;
 * rope_positions is device int32 [num_axes][position_stride], entry [a][b]
 * the position of sequence b's new token on axis a, position_stride >= batch.
 * A position outside [0, rows) skips the sequence and flags it.
 *
 * Errors as pkv_decode_attention; INVALID_ARG also for window < 1, sinks < 0
 * and a bad rope (see pkv_axes.h). With PKV_FLAG_PDL the contract of pkv.h
 * holds, rope_positions being one of the tensors read before the wait. */
pkv_status pkv_window_attention(pkv_pool_t pool, int layer, const void* q, const void* k_pool,
                                const void* v_pool, const int32_t* block_tables,
                                const int32_t* seq_lens, float* out, int window, int sinks,
                                const pkv_axes_rope* rope, const int32_t* rope_positions,
                                int position_stride, int batch, int num_splits, void* stream);

/* Append and attend in one launch: k[b], v[b] (BF16 [batch][8][64]; the key
 * rotated like the query when rope is given) go into the slot of position
 * seq_lens[b] - 1, then pkv_window_attention. A sequence that is skipped is
 * not appended. */
pkv_status pkv_window_append_attend(pkv_pool_t pool, int layer, const void* q, const void* k,
                                    const void* v, void* k_pool, void* v_pool,
                                    const int32_t* block_tables, const int32_t* seq_lens,
                                    float* out, int window, int sinks,
                                    const pkv_axes_rope* rope, const int32_t* rope_positions,
                                    int position_stride, int batch, int num_splits,
                                    void* stream);

/* pkv_prefill_attention behind the window: the chunk token at position p
 * attends to the tokens visible from p. Its K/V must be in the pages already
 * (pkv_prefill_fill or pkv_prefill_fill_axes, earlier on the stream). V of
 * a token that some row of a 32-token tile (counted from the chunk's first
 * token) sees must be finite for the results of all rows of that tile; K that
 * is not finite concerns the rows that see it alone. Errors as pkv_prefill_attention,
 * INVALID_ARG also for window < 1 and sinks < 0. */
pkv_status pkv_window_prefill_attention(pkv_pool_t pool, int layer, const void* q,
                                        const void* k_pool, const void* v_pool,
                                        const int32_t* block_tables, const int32_t* cu_tokens,
                                        const int32_t* start_pos, float* out, int window,
                                        int sinks, int batch, int total_tokens,
                                        int max_chunk_tokens, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PKV_WINDOW_H */
