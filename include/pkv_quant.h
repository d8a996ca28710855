/*
 * pkv_quant.h - an 8-bit KV cache: keys and values quantised as they are
 * written into pages, read back, and attended over in place. It takes 0.508 of
 * the bytes of the BF16 cache; handles, block tables, windows and rotary
 * positions are those of pkv.h, pkv_window.h and pkv_axes.h, admission and
 * release those of pkv_sched.h.
 *
 * What it does not share: pkv_copy_pages and pkv_compact_pages move pages of two
 * BF16 pools and none of this one (pkv_compact_pages would rewrite the tables all
 * the same), so the copies that pkv_sched_fork and pkv_sched_compact ask for are
 * the caller's to make: page i is row i of the tensor, whole. Chunks of a prompt and
 * drafted trees attend over BF16 pools alone.
 *
 * Pool: kv_pool, one uint8 tensor [num_pages][8][PKV_QUANT_TILE_BYTES] for K
 * and V together (16-byte aligned). The tile of a (page, kv head):
 *   bytes    0 .. 1023   K codes [16 tokens][64 dims]
 *   bytes 1024 .. 2047   V codes [4 chunks][16 tokens][16 dims], chunk c holding
 *                        dims 16 c .. 16 c + 15
 *   bytes 2048 .. 2063   K exponent bytes [16 tokens]
 *   bytes 2064 .. 2079   V exponent bytes [16 tokens]
 * A code is an e4m3 number (1 sign, 4 exponent and 3 fraction bits, largest
 * 448, 0x7f and 0xff NaN) and stands for it times 2^(E - 127), E the exponent
 * byte of its token's K or V in that head, 3 <= E <= 247 (a tile that is
 * attended over or read back holds no other E at a token that counts).
 *
 * Quantising a row of 64 values x (BF16, or FP32 after rotation; finite):
 * values beyond 1.875 x 2^127 are taken as that; E - 127 is the least e >= -124
 * with max |x| <= 448 x 2^e; each code is x 2^-e rounded to nearest, ties to
 * even. So a tile's content is bit-defined, what it stands for is exact in
 * BF16, and the error of a value is at most 2^-4 of it, or 2^-10 x 2^e where
 * that is more. A NaN is stored as a NaN code and does not count in the
 * maximum.
 *
 * Calls are asynchronous on `stream` and follow the rules of pkv.h: one stream
 * per handle, host-detectable errors return INVALID_ARG (another current
 * device among them) and launch nothing, what is found wrong in device data is
 * skipped and flagged (pkv_get_error). All calls take long-context handles.
 */
#ifndef PKV_QUANT_H
#define PKV_QUANT_H

#include <stdint.h>

#include "pkv.h"
#include "pkv_axes.h"

#ifdef __cplusplus
extern "C" {
#endif

#define PKV_QUANT_TILE_BYTES 2080

/* Quantises k[i], v[i] (BF16 [total_tokens][8][64]) of every chunk token into
 * its page slot (the packing of pkv_prefill.h; a decode step's rows are chunks
 * of one token). rope (NULL: none): keys are rotated in FP32 by pkv_axes.h's
 * rule and quantised from FP32; rope_positions is device int32
 * [num_axes][position_stride], position_stride >= total_tokens.
 *
 * A token whose place is outside [0, max_seq_len), whose rotary position is
 * outside [0, rows) or whose page id is outside the pool is skipped and
 * flagged; errors otherwise as pkv_prefill_fill_axes. k, v must not overlap
 * kv_pool. With PKV_FLAG_PDL it may come right before a decode launch of the
 * handle (the limits are those of pkv.h). */
pkv_status pkv_quant_fill(pkv_pool_t pool, int layer, const void* k, const void* v, void* kv_pool,
                          const int32_t* block_tables, const int32_t* cu_tokens,
                          const int32_t* start_pos, const pkv_axes_rope* rope,
                          const int32_t* rope_positions, int position_stride, int batch,
                          int total_tokens, int max_chunk_tokens, void* stream);

/* Reads tokens start_pos[b] .. of every sequence back: k[i], v[i] (BF16
 * [total_tokens][8][64], written) get what row i's token stands for, exactly
 * (same packing). Rows of tokens that are skipped (as in pkv_quant_fill) and
 * rows that no sequence has are left as they were. */
pkv_status pkv_quant_read(pkv_pool_t pool, int layer, const void* kv_pool,
                          const int32_t* block_tables, const int32_t* cu_tokens,
                          const int32_t* start_pos, void* k, void* v, int batch, int total_tokens,
                          int max_chunk_tokens, void* stream);

/* pkv_window_attention over the 8-bit cache: softmax(q . K_t / 8) V_t with what
 * the tiles stand for, over the tokens visible from position seq_lens[b] - 1
 * (pkv_window.h: window, sinks, padding rows, invalid pages, num_splits, rope).
 * q is BF16, out FP32; queries, scores, softmax statistics, probabilities and
 * sums keep FP32's precision, so the result is that of FP32 arithmetic on the
 * cache's values: keys below 2^122 in magnitude, scores and the sums of a
 * sequence's |V| inside FP32's range. Two things end earlier than in FP32: a
 * query's dim (after rotation) is held to within 2^-39 of its head's largest, so
 * dims down to 2^-31 of that keep all bits of a BF16 value, and those below 2^-40
 * count as 0; a token whose weight is below 2^-118 of its head's largest counts
 * as 0. */
pkv_status pkv_quant_attention(pkv_pool_t pool, int layer, const void* q, const void* kv_pool,
                               const int32_t* block_tables, const int32_t* seq_lens, float* out,
                               int window, int sinks, const pkv_axes_rope* rope,
                               const int32_t* rope_positions, int position_stride, int batch,
                               int num_splits, void* stream);

/* Append and attend in one launch: the new token's k[b], v[b] (BF16
 * [batch][8][64]; the key rotated with rope) are quantised into the slot of
 * position seq_lens[b] - 1, then pkv_quant_attention, which sees them as
 * stored. A sequence that is skipped is not appended. */
pkv_status pkv_quant_append_attend(pkv_pool_t pool, int layer, const void* q, const void* k,
                                   const void* v, void* kv_pool, const int32_t* block_tables,
                                   const int32_t* seq_lens, float* out, int window, int sinks,
                                   const pkv_axes_rope* rope, const int32_t* rope_positions,
                                   int position_stride, int batch, int num_splits, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PKV_QUANT_H */
