/*
 * pkv_axes.h - rotary position embedding by several position axes, for
 * prompts that mix text with images and video: a token has one position per
 * axis (time, height, width, ...), and each rotary pair turns by the angle of
 * the axis it belongs to. Text tokens carry the same position on every axis,
 * which is the ordinary rotary embedding of pkv.h.
 *
 * Pair i < 32 of a head is (x[i], x[i + 32]). With a = axis_of_pair[i], p the
 * token's position on axis a, c = cos[p][i] and s = sin[p][i]:
 *   x'[i] = x[i] c - x[i + 32] s,   x'[i + 32] = x[i + 32] c + x[i] s.
 * Each product and the sum are rounded in FP32 (no fused multiply-add). A key
 * is stored as BF16 rounded to nearest even, so a page's content is
 * bit-defined; pkv_prefill_fill_axes rounds queries the same way, the decode
 * entry points of pkv_window.h keep them in FP32.
 *
 * Rotary positions have nothing to do with the slot a token is stored in: that
 * follows from its place in the sequence, as everywhere in this library.
 */
#ifndef PKV_AXES_H
#define PKV_AXES_H

#include <stdint.h>

#include "pkv.h"

#ifdef __cplusplus
extern "C" {
#endif

#define PKV_MAX_AXES 4

/* The part of the rotation that a program keeps: cos and sin are device FP32
 * [rows][32] tables (16-byte aligned, owned by the caller, read-only here; the
 * base and any frequency scaling are the caller's choice). axis_of_pair is
 * host data, copied by every call: the axis of each pair, below num_axes,
 * in any order (sections one after the other, or interleaved). */
typedef struct {
  const float* cos;
  const float* sin;
  int rows;                   /* positions the tables cover, >= 1 */
  int num_axes;               /* 1 .. PKV_MAX_AXES */
  uint8_t axis_of_pair[32];
} pkv_axes_rope;

/* Prefill fill with rotation, one launch: for every chunk token (the packing
 * of pkv_prefill.h: cu_tokens, start_pos, total_tokens, max_chunk_tokens)
 *   q_out[i][h][:] = rotated q[i][h][:]   (BF16 [total_tokens][32][64])
 *   its page slot of k_pool gets the rotated k[i], that of v_pool v[i],
 * i.e. what pkv_prefill_attention and pkv_window_prefill_attention take.
 * rope_positions: device int32 [num_axes][position_stride], entry [a][i] the
 * position of packed row i on axis a; position_stride >= total_tokens.
 * rope_positions, cu_tokens and start_pos need 4-byte alignment only.
 * q_out may be q itself (rotated in place) but not overlap it otherwise; q
 * and q_out may both be NULL (keys and values only). k and v must not
 * overlap the pools or q_out.
 *
 * A token whose rotary position is outside [0, rows), whose place is outside
 * [0, max_seq_len) or whose page id is outside the pool is skipped (its q_out
 * row is left as it was) and flagged; errors otherwise as pkv_prefill_fill,
 * INVALID_ARG also for a null rope, null or misaligned tables or positions,
 * rows < 1, num_axes outside [1, 4], a pair's axis outside [0, num_axes) or
 * position_stride < total_tokens. With PKV_FLAG_PDL it may come right before a
 * decode launch of the handle (the limits are those of pkv.h). Takes
 * long-context handles. */
pkv_status pkv_prefill_fill_axes(pkv_pool_t pool, int layer, const void* q, const void* k,
                                 const void* v, void* q_out, void* k_pool, void* v_pool,
                                 const int32_t* block_tables, const int32_t* cu_tokens,
                                 const int32_t* start_pos, const pkv_axes_rope* rope,
                                 const int32_t* rope_positions, int position_stride, int batch,
                                 int total_tokens, int max_chunk_tokens, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PKV_AXES_H */
