/*
 * pkv_pages.h - copying pages of the shared KV pool on the device: the pages
 * that forked sequences do not share (pkv_sched_fork) and the moves that
 * compact a pool (pkv_sched_compact).
 *
 * src, dst: device int32 [n] page ids (4-byte aligned; the pools and tables 16,
 * as everywhere). A page may be the source of several pairs. A destination must
 * be named by one pair only and be no pair's source: pairs that break this are
 * skipped and flagged (PKV_ERR_OUT_OF_RANGE from pkv_get_error), the others are
 * carried out, so the result never depends on the order of the copies. Pairs
 * with an id outside [0, num_pages) are skipped and flagged; an id in range
 * counts as named even where the rest of its pair is bad.
 *
 * Calls are asynchronous on `stream`. Host-detectable errors (null or
 * misaligned pointers, n outside [0, num_pages], another current device)
 * return INVALID_ARG and launch nothing; n == 0 is a no-op. Both calls use
 * scratch of the handle, so they share its rule: one stream per handle. With
 * PKV_FLAG_PDL either may come right before a decode launch of the handle (the
 * limits are those of pkv.h). Takes long-context handles.
 */
#ifndef PKV_PAGES_H
#define PKV_PAGES_H

#include <stdint.h>

#include "pkv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Copies, in both pools, page src[i] to page dst[i]: the whole page, or with
 * tokens (device int32 [n], or NULL) the first tokens[i] tokens of every KV
 * head; the destination's other tokens are left as they were. A pair with
 * tokens[i] outside [0, 16] is skipped and flagged. Bit copy. */
pkv_status pkv_copy_pages(pkv_pool_t pool, const int32_t* src, const int32_t* dst,
                          const int32_t* tokens, void* k_pool, void* v_pool, int n,
                          void* stream);

/* Moves page src[i] to page dst[i] in both pools and rewrites every entry of
 * block_tables (all of [num_layers][max_batch][max_seq_len / 16]) that names
 * src[i] to dst[i]; other entries, -1 among them, stay. Here a source must be
 * named by one pair only as well (else its pairs are skipped and flagged, and
 * entries naming it stay). The source pages keep their content. */
pkv_status pkv_compact_pages(pkv_pool_t pool, const int32_t* src, const int32_t* dst,
                             void* k_pool, void* v_pool, int32_t* block_tables, int n,
                             void* stream);

#ifdef __cplusplus
}
#endif

#endif /* PKV_PAGES_H */
