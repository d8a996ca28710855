// Attention of drafted token trees over the paged KV cache for GB300 (sm_103a),
// and the commit of an accepted path (declared in include/pkv_tree.h).
//
// The attention kernel is prefill_tiles.cuh's. A tile is up to 32 drafted tokens
// of one sequence and KV head (128 rows) and a part of the keys they see: the
// sink pages, the window's and the drafted tokens' own. Trees are few rows over
// long contexts, so a tile's steps are split into parts of about equal length,
// as many as the device holds CTAs, and a second kernel joins the parts' sums.
//
// What bounds it: over long contexts the softmax warps, as in windowed prefill: a
// step of two CTAs takes about 2,000 cycles. Eight trees of 49 to 64 tokens over
// 20,000 to 32,700: 204 us, 462 TFLOP/s of score and value products counted once (254
// with parts of one length for a launch, a fifth of the CTAs idle at the end; 217 with
// the parts joined by the last of a tile, in the same launch). A small call is latency:
// of 32 trees of up to 16 tokens over up to 2,000, 21 us, a CTA needs 4.4 before its
// first scores (set-up, its share of the line, page ids, copies), 0.7 a step, 2 at a
// tile's end; the join 2.
//
// The commit moves 128-byte rows: 256 sequences of up to 8 tokens in 16 layers 20 us
// (3.8 TB/s; 2 more with divisions by a launch's number of heads), one of 4 tokens 2.1 us.
// What bounds it is latency: 4,096 blocks, 4.5 waves, that each wait for three loads one
// after the other, 44 % of their items tokens past the count; HBM is at 29 %, issue at 51 %.

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "pkv.h"
#include "pkv_tree.h"
#include "device_common.cuh"
#include "pool_internal.h"
#include "prefill_device.cuh"
#include "prefill_tiles.cuh"
#include "tree.cuh"

using namespace pkv_tree_dev;

namespace {

struct TreeJob {
  using Params = TreeParams;
  using Work = TreeWork;
  using View = TreeView;
  using Walk = TreeWalk<kTileTokens>;
  static constexpr bool kFewRows = true;
  static constexpr bool kParts = true;
  static constexpr bool kDrawn = false;
  static __device__ __forceinline__ bool is_whole(const Work& work) { return work.slot < 0; }
  static __device__ __forceinline__ void put_sums(const Work& work, const Params& prm, int r,
                                                  float m, float l) {
    prm.part_ml[static_cast<size_t>(work.slot) * kRows + r] = make_float2(m, l);
  }
  static __device__ __forceinline__ float4* part(const Work& work, const Params& prm) {
    return reinterpret_cast<float4*>(prm.part_o + static_cast<size_t>(work.slot) * kRows * kDim);
  }
  using Row = TreeRow;
};


// ---------------------------------------------------------------- commit
// A block per (sequence, layer, some KV heads: as many as its threads can hold the
// rows of). A thread's 16-byte vectors are (token, head, pool, chunk), all read
// before any is written.
constexpr int kCommitThreads = 256;
constexpr int kHeadVecs = 2 * kRowBytes / 16;                    // K and V of a token: 16
constexpr int kCommitItems = kMaxTree * kHeadVecs / kCommitThreads;   // 4

template <int heads>
__global__ void __launch_bounds__(kCommitThreads, 6) tree_commit_kernel(
    uint4* k_pool, uint4* v_pool, const int32_t* __restrict__ tables,
    const int32_t* __restrict__ start_pos, const int32_t* __restrict__ accepted,
    const int32_t* __restrict__ counts, int max_accepted, int max_batch, int table_stride,
    int num_pages, int max_seq_len, int* err) {
  const int b = blockIdx.y, layer = blockIdx.z;
  const int count = counts[b], start = start_pos[b];
  // item i of this thread: accepted token k(i)'s vector `vec` of head g(i)
  auto k_of = [&](int i) { return (threadIdx.x + i * kCommitThreads) / (heads * kHeadVecs); };
  int j[kCommitItems];
  #pragma unroll
  for (int i = 0; i < kCommitItems; ++i)        // not waiting for the count
    j[i] = k_of(i) < max_accepted ? accepted[static_cast<size_t>(b) * max_accepted + k_of(i)] : 0;
  if (count == 0) return;
  const bool reports = threadIdx.x == 0 && blockIdx.x == 0;
  if (count < 0 || count > max_accepted || start < 0 || start > max_seq_len - count) {
    if (reports) set_error(err, count < 0 || count > max_accepted ? PKV_DEV_ERR_SEQ_LEN
                                                                  : PKV_DEV_ERR_POSITION);
    return;
  }
  const int32_t* row = tables + (static_cast<size_t>(layer) * max_batch + b) * table_stride;
  int page[kCommitItems], dest[kCommitItems];
  int bad = 0;
  #pragma unroll
  for (int i = 0; i < kCommitItems; ++i) {
    page[i] = dest[i] = -1;
    if (k_of(i) >= count) continue;
    if (j[i] < 0 || j[i] >= kMaxTree || j[i] >= max_seq_len - start) {
      bad = PKV_DEV_ERR_POSITION;
      continue;
    }
    page[i] = row[(start + j[i]) / kPage];
    dest[i] = row[(start + k_of(i)) / kPage];
  }
  uint4 v[kCommitItems];
  #pragma unroll
  for (int i = 0; i < kCommitItems; ++i) {
    v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (k_of(i) >= count || bad) continue;
    if (page[i] < 0 || page[i] >= num_pages || dest[i] < 0 || dest[i] >= num_pages) {
      bad = PKV_DEV_ERR_PAGE;
      continue;
    }
    const int item = threadIdx.x + i * kCommitThreads;
    const int g = blockIdx.x * heads + item / kHeadVecs % heads;
    const uint4* pool = item / 8 % 2 ? v_pool : k_pool;
    v[i] = pool[((static_cast<size_t>(page[i]) * kHkv + g) * kPage + (start + j[i]) % kPage) * 8 +
                item % 8];
  }
  // every row is in registers, and the verdict is the block's
  if (bad) set_error(err, bad);
  if (__syncthreads_or(bad)) return;
  #pragma unroll
  for (int i = 0; i < kCommitItems; ++i) {
    if (k_of(i) >= count) continue;
    const int item = threadIdx.x + i * kCommitThreads;
    const int g = blockIdx.x * heads + item / kHeadVecs % heads;
    uint4* pool = item / 8 % 2 ? v_pool : k_pool;
    pool[((static_cast<size_t>(dest[i]) * kHkv + g) * kPage + (start + k_of(i)) % kPage) * 8 +
         item % 8] = v[i];
  }
}

// Whether the kernel for few rows takes the call: where it does so in clusters, or for
// up to 8 drafted tokens a sequence on average. Measured (us, this and the other kernel;
// sequences x drafted tokens, 2,000 committed): in clusters 1 x 8 7.4 and 12.9, 1 x 64
// 14.3 and 15.4, 3 x 16 11.6 and 14.2, 4 x 16 14.1 and 15.3, over 300 7.9 and 11.6, 1 x 8
// over 8,000 13.6 and 17.2; on the line 16 x 8 23.5 and 25.8, 32 x 8 36.6 and 40.4, 128 x
// 4 91 and 119, 256 x 8 over 1,000 126 and 139, 1 x 8 over 16,000 20.5 and 20.4, 8 x 8
// 59.5 and 60.7, 2 x 8 over 100,000 87.0 and 88.4; 8 x 16 22.5 and 19.3, 32 x 16 64 and
// 47.
bool few_rows(int batch, int total_tokens, int parts) {
  return parts > 0 || total_tokens <= 8ll * batch;
}

}  // namespace

size_t pkv_tree_slots(const pkv_pool* pool) {
  return static_cast<size_t>(2) * kCtasPerSm * pool->num_sms;
}

extern "C" {

pkv_status pkv_tree_attention(pkv_pool_t pool, int layer, const void* q, const void* k_pool,
                              const void* v_pool, const int32_t* block_tables,
                              const int32_t* cu_tokens, const int32_t* start_pos,
                              const uint64_t* tree, float* out, int window, int sinks, int batch,
                              int total_tokens, void* stream) {
  if (!pool) return PKV_ERR_INVALID_ARG;
  const pkv_pool_config& c = pool->cfg;
  if (layer < 0 || layer >= c.num_layers || batch < 0 || batch > c.max_batch ||
      total_tokens < 0 || window < 1 || sinks < 0)
    return PKV_ERR_INVALID_ARG;
  if (batch == 0 || total_tokens == 0) return PKV_OK;
  if (!q || !k_pool || !v_pool || !block_tables || !cu_tokens || !start_pos || !tree || !out ||
      !pkv_aligned16(q) || !pkv_aligned16(k_pool) || !pkv_aligned16(v_pool) ||
      !pkv_aligned16(block_tables) || !pkv_aligned4(cu_tokens) || !pkv_aligned4(start_pos) ||
      (reinterpret_cast<uintptr_t>(tree) & 7u) != 0 || !pkv_aligned16(out))
    return PKV_ERR_INVALID_ARG;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev != pool->device) return PKV_ERR_INVALID_ARG;
  if (!set_smem_attribute<TreeJob>(pool->device)) return PKV_ERR_CUDA;

  CUtensorMap tq, tk, tv;
  // what a row sees: the context, or the sinks, the window and whole pages around them
  const long long seen = std::min<long long>(c.max_seq_len, static_cast<long long>(window) + sinks +
                                                                kMaxTree + 2 * kPage);
  const int parts = pkv_tree_cluster(pool, batch, total_tokens, static_cast<int>(seen));
  const bool few = few_rows(batch, total_tokens, parts);
  const cuuint64_t dims[3] = {kDim, kHq, static_cast<cuuint64_t>(total_tokens)};
  const cuuint64_t strides[2] = {kRowBytes, static_cast<cuuint64_t>(kHq) * kRowBytes};
  const cuuint32_t box[3] = {kDim, kGroup, kTileTokens};
  if ((!few && !encode_bf16(&tq, q, 3, dims, strides, box)) ||
      !pkv_pool_tensor_map(k_pool, c.num_pages, &tk) ||
      !pkv_pool_tensor_map(v_pool, c.num_pages, &tv))
    return PKV_ERR_CUDA;
  const int stride = c.max_seq_len / kPage;
  const int wave = kCtasPerSm * pool->num_sms;
  TreeParams prm;
  prm.table = block_tables + static_cast<size_t>(layer) * c.max_batch * stride;
  prm.cu_tokens = cu_tokens;
  prm.start_pos = start_pos;
  prm.out = out;
  prm.err = pool->err;
  prm.num_pages = c.num_pages;
  prm.table_stride = stride;
  prm.max_seq_len = c.max_seq_len;
  prm.batch = batch;
  prm.total_tokens = total_tokens;
  prm.window = std::min(window, c.max_seq_len);
  prm.sinks = std::min(sinks, c.max_seq_len);
  prm.tree = reinterpret_cast<const unsigned long long*>(tree);
  prm.part_o = pool->part_o;
  prm.part_ml = pool->part_ml;
  set_wave(&prm, wave);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (few) return pkv_tree_few(pool, q, tk, tv, prm, parts, st);
  tile_attention_kernel<TreeJob><<<wave, kThreads, kSmemBytes<TreeJob>, st>>>(tq, tk, tv, prm);
  if (cudaGetLastError() != cudaSuccess) return PKV_ERR_CUDA;
  return launch_join<kTileTokens>(prm, st);
}

pkv_status pkv_tree_commit(pkv_pool_t pool, void* k_pool, void* v_pool,
                           const int32_t* block_tables, const int32_t* start_pos,
                           const int32_t* accepted, const int32_t* counts, int batch,
                           int max_accepted, void* stream) {
  if (!pool) return PKV_ERR_INVALID_ARG;
  const pkv_pool_config& c = pool->cfg;
  if (batch < 0 || batch > c.max_batch || max_accepted < 1 || max_accepted > kMaxTree)
    return PKV_ERR_INVALID_ARG;
  if (batch == 0) return PKV_OK;
  if (!k_pool || !v_pool || !block_tables || !start_pos || !accepted || !counts ||
      !pkv_aligned16(k_pool) || !pkv_aligned16(v_pool) || !pkv_aligned16(block_tables) ||
      !pkv_aligned4(start_pos) || !pkv_aligned4(accepted) || !pkv_aligned4(counts) ||
      c.num_layers > 65535)
    return PKV_ERR_INVALID_ARG;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev != pool->device) return PKV_ERR_INVALID_ARG;
  int heads = kHkv;
  while (heads > 1 && heads * max_accepted > kMaxTree) heads /= 2;
  const auto kernel = heads == 8   ? tree_commit_kernel<8>
                      : heads == 4 ? tree_commit_kernel<4>
                      : heads == 2 ? tree_commit_kernel<2>
                                   : tree_commit_kernel<1>;
  pool->pages_written = true;
  kernel<<<dim3(kHkv / heads, batch, c.num_layers), kCommitThreads, 0,
           static_cast<cudaStream_t>(stream)>>>(
      static_cast<uint4*>(k_pool), static_cast<uint4*>(v_pool), block_tables, start_pos, accepted,
      counts, max_accepted, c.max_batch, c.max_seq_len / kPage, c.num_pages, c.max_seq_len,
      pool->err);
  return pkv_check_launch();
}

}  // extern "C"
