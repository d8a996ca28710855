// Page copies and moves over the shared KV pool (declared in
// include/pkv_pages.h): what forked sequences copy of the pages they cannot
// share, and the moves and block-table rewrites that compact a pool.
//
// The work is memory traffic alone: 64 KiB per whole page pair (K and V, read
// and written), so HBM bounds it: 16,384 moves with their tables take 167 us
// (6.4 TB/s, 96 % of the measured copy rate); small calls are bound by their
// launch (128 pairs 2.5 us).
// Whether a pair may be carried out depends on the whole list (a destination
// must be named once and be nobody's source), so that is settled before any
// byte moves: no order of the blocks can change the result.

#include <cuda_runtime.h>
#include <stdint.h>

#include "pkv.h"
#include "pkv_pages.h"
#include "device_common.cuh"
#include "pool_internal.h"

using namespace pkv_dev;

namespace {

constexpr int kCopyThreads = 128;
constexpr int kPageVecs = kHkv * kPage * kRowBytes / 16;     // 16-byte vectors of a page: 1024
constexpr int kVecsPerThread = kPageVecs / kCopyThreads;     // 8

// Lists of up to this many pairs are checked by every copy block for itself, in
// one launch; longer ones are counted per page first, in two launches more (a
// memset and the counts), since the checks grow with n^2. Partial copies, the
// launches in a graph, checked and counted (us): 257 pairs 3.4 and 4.9, 800 6.3
// and 7.1, 1,024 7.3 and 8.1, 1,500 10.3 and 9.0.
constexpr int kScanPairs = 1024;

// How often each page is named: destinations in the low half of a page's
// count, sources in the high half.
__global__ void __launch_bounds__(256) mark_pages_kernel(const int32_t* src, const int32_t* dst,
                                                         int n, int num_pages,
                                                         unsigned long long* marks) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= n) return;
  const int s = src[i], d = dst[i];
  if (s >= 0 && s < num_pages) atomicAdd(&marks[s], 1ull << 32);
  if (d >= 0 && d < num_pages) atomicAdd(&marks[d], 1ull);
}

// One block per (pair, pool): 128 threads move the page's 16 KiB, 8 vectors
// of 16 bytes each, all loads before the first store. Vector j of a page is
// token (j / 8) % 16 of its KV head. kScan: the block reads the list itself;
// else the counts are in marks. page_to (compaction): 1 + the pair that moves
// its source, 0 for a pair that is skipped.
template <bool kScan>
__global__ void __launch_bounds__(kCopyThreads) copy_pages_kernel(
    const int32_t* __restrict__ src, const int32_t* __restrict__ dst,
    const int32_t* __restrict__ tokens, uint4* k_pool, uint4* v_pool, int n, int num_pages,
    const unsigned long long* __restrict__ marks, int* page_to, int* err) {
  const int i = blockIdx.x >> 1;
  uint4* pool = (blockIdx.x & 1) ? v_pool : k_pool;
  const int t = threadIdx.x;
  const int s = src[i], d = dst[i];
  const int count = tokens ? tokens[i] : kPage;
  bool ok = s >= 0 && s < num_pages && d >= 0 && d < num_pages && count >= 0 && count <= kPage;
  if (kScan) {
    bool clash = false;
    for (int j = t; j < n; j += kCopyThreads)
      clash |= src[j] == d || (j != i && (dst[j] == d || (page_to && src[j] == s)));
    ok = !__syncthreads_or(clash) && ok;
  } else if (ok) {
    ok = marks[d] == 1ull && (!page_to || (marks[s] >> 32) == 1ull);
  }
  // two pairs of one source are both skipped: they write the same
  if (page_to && t == 0 && !(blockIdx.x & 1) && s >= 0 && s < num_pages)
    page_to[s] = ok ? i + 1 : 0;
  if (!ok) {
    if (t == 0) set_error(err, PKV_DEV_ERR_PAGE);
    return;
  }
  const uint4* from = pool + static_cast<size_t>(s) * kPageVecs;
  uint4* to = pool + static_cast<size_t>(d) * kPageVecs;
  // this thread's vectors are t + 128 j: the same token of KV head j
  if (((t >> 3) & (kPage - 1)) >= count) return;
  uint4 v[kVecsPerThread];
  #pragma unroll
  for (int j = 0; j < kVecsPerThread; ++j) v[j] = __ldcs(from + t + j * kCopyThreads);
  #pragma unroll
  for (int j = 0; j < kVecsPerThread; ++j) __stcs(to + t + j * kCopyThreads, v[j]);
}
static_assert(kCopyThreads == kPage * 8, "a thread's vectors belong to one token");

// Entries naming a moved page take its new id, 4 entries per thread. What
// page_to holds for a page that no pair of this list names as its source is
// left from earlier lists: the pair it points to has another source.
__global__ void __launch_bounds__(256) rewrite_tables_kernel(
    const int32_t* __restrict__ src, const int32_t* __restrict__ dst, int n_pairs,
    int32_t* tables, size_t entries, int num_pages, const int* __restrict__ page_to) {
  const size_t at = (static_cast<size_t>(blockIdx.x) * 256 + threadIdx.x) * 4;
  if (at >= entries) return;
  const int n = static_cast<int>(min(entries - at, static_cast<size_t>(4)));
  int32_t id[4];
  bool moved = false;
  if (n == 4) {
    const int4 v = *reinterpret_cast<const int4*>(tables + at);
    id[0] = v.x; id[1] = v.y; id[2] = v.z; id[3] = v.w;
  } else {
    for (int e = 0; e < 4; ++e) id[e] = e < n ? tables[at + e] : -1;
  }
  #pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int pair = id[e] >= 0 && id[e] < num_pages ? page_to[id[e]] - 1 : -1;
    if (pair >= 0 && pair < n_pairs && src[pair] == id[e]) {
      id[e] = dst[pair];
      moved = true;
    }
  }
  if (!moved) return;
  if (n == 4) {
    *reinterpret_cast<int4*>(tables + at) = make_int4(id[0], id[1], id[2], id[3]);
  } else {
    for (int e = 0; e < n; ++e) tables[at + e] = id[e];
  }
}

pkv_status launch_copies(pkv_pool_t pool, const int32_t* src, const int32_t* dst,
                         const int32_t* tokens, void* k_pool, void* v_pool, int32_t* tables,
                         bool compact, int n, void* stream) {
  if (!pool) return PKV_ERR_INVALID_ARG;
  const pkv_pool_config& c = pool->cfg;
  if (n < 0 || n > c.num_pages) return PKV_ERR_INVALID_ARG;
  if (n == 0) return PKV_OK;
  if (!src || !dst || !k_pool || !v_pool || (compact && !tables)) return PKV_ERR_INVALID_ARG;
  if (!pkv_aligned4(src) || !pkv_aligned4(dst) || !pkv_aligned4(tokens) ||
      !pkv_aligned16(k_pool) || !pkv_aligned16(v_pool) || !pkv_aligned16(tables))
    return PKV_ERR_INVALID_ARG;
  if (n > (1 << 30)) return PKV_ERR_INVALID_ARG;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev != pool->device) return PKV_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  uint4* kp = static_cast<uint4*>(k_pool);
  uint4* vp = static_cast<uint4*>(v_pool);
  int* page_to = compact ? pool->page_to : nullptr;
  pool->pages_written = true;
  if (n <= kScanPairs) {
    copy_pages_kernel<true><<<2 * n, kCopyThreads, 0, st>>>(src, dst, tokens, kp, vp, n,
                                                            c.num_pages, nullptr, page_to,
                                                            pool->err);
  } else {
    const size_t scratch = static_cast<size_t>(c.num_pages) * sizeof(unsigned long long);
    if (cudaMemsetAsync(pool->page_marks, 0, scratch, st) != cudaSuccess) return PKV_ERR_CUDA;
    mark_pages_kernel<<<(n + 255) / 256, 256, 0, st>>>(src, dst, n, c.num_pages,
                                                       pool->page_marks);
    copy_pages_kernel<false><<<2 * n, kCopyThreads, 0, st>>>(
        src, dst, tokens, kp, vp, n, c.num_pages, pool->page_marks, page_to, pool->err);
  }
  if (compact) {
    const size_t entries = static_cast<size_t>(c.num_layers) * c.max_batch *
                           (c.max_seq_len / kPage);
    rewrite_tables_kernel<<<static_cast<unsigned>((entries + 1023) / 1024), 256, 0, st>>>(
        src, dst, n, tables, entries, c.num_pages, page_to);
  }
  return pkv_check_launch();
}

}  // namespace

extern "C" {

pkv_status pkv_copy_pages(pkv_pool_t pool, const int32_t* src, const int32_t* dst,
                          const int32_t* tokens, void* k_pool, void* v_pool, int n,
                          void* stream) {
  return launch_copies(pool, src, dst, tokens, k_pool, v_pool, nullptr, false, n, stream);
}

pkv_status pkv_compact_pages(pkv_pool_t pool, const int32_t* src, const int32_t* dst,
                             void* k_pool, void* v_pool, int32_t* block_tables, int n,
                             void* stream) {
  return launch_copies(pool, src, dst, nullptr, k_pool, v_pool, block_tables, true, n, stream);
}

}  // extern "C"
