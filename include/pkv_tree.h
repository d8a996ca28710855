/*
 * pkv_tree.h - drafted tokens over the paged KV cache (speculative decoding):
 * attention of a tree of drafted tokens per sequence, and the commit of the path
 * that was accepted.
 *
 * Sequence b has start_pos[b] committed tokens (0 allowed) and n_b = cu_tokens[b+1]
 * - cu_tokens[b] drafted ones, 0 <= n_b <= PKV_MAX_TREE, packed at rows
 * cu_tokens[b] .. of q, out and tree. Drafted token i of a sequence occupies the
 * slot of position start_pos[b] + i (pkv_prefill_fill, or pkv_prefill_fill_axes
 * with rotary positions of its depth in the tree, earlier on the stream), whatever
 * its depth.
 *
 * Geometry, pools, block tables and dtypes are those of pkv.h and pkv_prefill.h;
 * lists of int32 need 4-byte alignment only, tree 8-byte. Calls are asynchronous
 * on `stream`, one stream per handle; host-detectable errors return INVALID_ARG
 * (another current device among them) and launch nothing. Long-context handles
 * are taken.
 */
#ifndef PKV_TREE_H
#define PKV_TREE_H

#include <stdint.h>

#include "pkv.h"

#ifdef __cplusplus
extern "C" {
#endif

#define PKV_MAX_TREE 64

/* out[i][h][:] = sum_t softmax_t(q[i][h] . K_t / 8) V_t (q BF16
 * [total_tokens][32][64], already rotated; out FP32 [total_tokens][32][64]) for
 * every drafted token i of sequence b over
 *   - drafted token j of its sequence where bit j of tree[i] is set (device uint64
 *     [total_tokens]; bits from n_b on are ignored): its ancestors and itself in a
 *     tree, but any set may be given;
 *   - committed tokens t < start_pos[b] with p_i - t < window or t < sinks, where
 *     p_i = start_pos[b] + (bits that count) - 1, a tree token's position.
 * window >= 1 (any value >= max_seq_len: every committed token), sinks >= 0. A row
 * that sees nothing is 0.
 * The window hides committed tokens only: a drafted token that bit j names is seen
 * whatever its distance. So for window >= the drafted tokens of the longest path a
 * verified step sees what decode steps along that path would see one by one; behind a
 * shorter window it sees more, and no tree says otherwise (bits left out also move p_i,
 * and with it the window).
 *
 * Pages all of whose tokens no drafted token of the sequence sees and which hold no
 * drafted token are not read, their table entries may hold anything. In a page that
 * is read, K that is not finite concerns the rows that see it alone; V of committed
 * tokens inside some row's window or the sinks and of every drafted token must be
 * finite; tokens before every row's window or past the last drafted one may hold
 * any bits. An invalid page id is flagged and its tokens are skipped. A sequence
 * whose rows fall outside [0, total_tokens), with more than PKV_MAX_TREE tokens, or
 * whose tokens pass max_seq_len is skipped (its out rows are left as they were) and
 * flagged; rows of no sequence are left as they were.
 *
 * Arithmetic as pkv_window_attention: the result is that of FP32 arithmetic on BF16
 * inputs. */
pkv_status pkv_tree_attention(pkv_pool_t pool, int layer, const void* q, const void* k_pool,
                              const void* v_pool, const int32_t* block_tables,
                              const int32_t* cu_tokens, const int32_t* start_pos,
                              const uint64_t* tree, float* out, int window, int sinks, int batch,
                              int total_tokens, void* stream);

/* The accepted path: for every layer and every k < counts[b], K and V of drafted
 * token accepted[b][k] (device int32 [batch][max_accepted]) go to position
 * start_pos[b] + k, bit for bit; all are read before any is written, so any order
 * and repeated tokens are allowed. Slots behind the last accepted token keep what
 * they held. Afterwards the sequence has start_pos[b] + counts[b] tokens.
 *
 * 1 <= max_accepted <= PKV_MAX_TREE; 0 <= counts[b] <= max_accepted. A sequence with
 * a count or a token out of range ([0, PKV_MAX_TREE)), or places outside [0,
 * max_seq_len), is skipped whole and flagged; in a layer where a page id that it
 * needs is invalid it is skipped in that layer and flagged. With PKV_FLAG_PDL it may
 * come right before a decode launch of the handle (the limits are those of pkv.h). */
pkv_status pkv_tree_commit(pkv_pool_t pool, void* k_pool, void* v_pool,
                           const int32_t* block_tables, const int32_t* start_pos,
                           const int32_t* accepted, const int32_t* counts, int batch,
                           int max_accepted, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PKV_TREE_H */
