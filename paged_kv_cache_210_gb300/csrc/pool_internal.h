// Internal to libpkv: the pool handle behind pkv_pool_t and the device error
// bits, shared by the decode (pkv.cu) and prefill (prefill.cu) sources.
#ifndef PKV_POOL_INTERNAL_H
#define PKV_POOL_INTERNAL_H

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "pkv.h"

// Resident blocks per SM of a windowed decode kernel's shapes.
struct WindowResidency {
  int blocks_per_sm;           // ticket merge
  int cluster_blocks_per_sm;   // cluster merge
};

struct pkv_pool {
  pkv_pool_config cfg;
  int device;
  int num_sms;
  int blocks_per_sm;           // resident decode blocks per SM (occupancy API)
  int cluster_blocks_per_sm;   // the same for the narrow cluster-merge kernel
  int wide_blocks_per_sm;      // the same for the wide cluster-merge kernel
  int max_cluster;     // largest cluster size (power of two <= 16) the device schedules
  // Partial sums of one launch: of decode calls [2][max_batch][32][max_splits], of drafted
  // trees [pkv_tree_slots][128]. A tree's attention is launched when all before it is
  // done, and a decode writes partials once the join before it is.
  float* part_o;     // [...][64]
  float2* part_ml;
  int* tickets;      // [2][max_batch][8]
  int* err;          // sticky error bits (PKV_DEV_ERR_*)
  int* seq_done;     // [max_batch]: layer completions per sequence (multi-layer launch)
  unsigned long long* page_marks;   // [num_pages] how often the call's pairs name a page:
                                    // low half as destination, high half as source
  int* page_to;                     // [num_pages] 1 + the pair that moves a page (0: none), of the
                                    // last compaction that named it; follows page_marks in one
                                    // allocation
  unsigned long long* prefill_next; // windowed prefill: tiles drawn, CTAs done (zero between
                                    // launches)
  WindowResidency window;           // the windowed decode over BF16 pages
  WindowResidency quant;            // ... and over 8-bit pages
  std::atomic<bool> pages_written{false};   // the handle's last page or fill call (pkv_pages.h,
                                            // pkv_axes.h) has had no decode launch after it
  int layer_clusters[5];   // resident clusters of the multi-layer kernel, S = 1, 2, 4, 8, 16
};

// Sticky device error bits; pkv_get_error maps TIMEOUT to
// PKV_ERR_DEVICE_TIMEOUT and the others to PKV_ERR_OUT_OF_RANGE.
enum : int {
  PKV_DEV_ERR_PAGE = 1,       // a page id outside [0, num_pages)
  PKV_DEV_ERR_POSITION = 2,   // a position outside [0, max_seq_len)
  PKV_DEV_ERR_SEQ_LEN = 4,    // a length outside [1, max_seq_len]
  PKV_DEV_ERR_TIMEOUT = 8,    // a bounded wait gave up
};

// Host helpers of the entry points.
inline bool pkv_aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Lists of int32 that the kernels read one by one.
inline bool pkv_aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

inline pkv_status pkv_check_launch() {
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

// Whether the handle is in the range of the entry points limited to
// 2,048-token contexts (their kernels hold a whole block-table row).
inline bool pkv_short_context(const pkv_pool* pool) { return pool->cfg.max_seq_len <= 2048; }

// Whether the next decode launch may start under the kernel before it
// (PKV_FLAG_PDL): it then reads tables and pages ahead of that kernel's end, so
// not if that may be the handle's own call that writes them.
inline bool pkv_starts_early(pkv_pool* pool) {
  return (pool->cfg.flags & PKV_FLAG_PDL) != 0 && !pool->pages_written.exchange(false);
}

// pkv.cu: a K or V pool of num_pages pages as the copy engine's 3-D tensor
// map (dim, kv head x 16 + token, page), boxes of one (page, kv head) tile
// with the 128-byte swizzle; false if the driver refuses it.
bool pkv_pool_tensor_map(const void* pool, int num_pages, CUtensorMap* map);

// layers.cu: the multi-layer kernel's attributes and, per cluster size, how
// many of its clusters the device holds at once (pool->layer_clusters).
bool pkv_layers_setup(pkv_pool* pool);

// window.cu, quant.cu: the windowed decode kernels' attributes and residency.
bool pkv_window_setup(pkv_pool* pool);
bool pkv_quant_setup(pkv_pool* pool);

// tree_few.cu: its kernel's attributes.
bool pkv_tree_few_setup();

// tree.cu: parts of 128 rows whose sums one call may keep.
size_t pkv_tree_slots(const pkv_pool* pool);

#endif  // PKV_POOL_INTERNAL_H
