// The 8-bit KV cache's fill and read-back (declared in include/pkv_quant.h).
//
// Both are memory traffic: 2,048 + 1,040 bytes a token either way (K and V of 8
// heads in BF16, and as codes with their exponents).

#include <cuda_runtime.h>
#include <stdint.h>

#include "pkv.h"
#include "pkv_quant.h"
#include "axes.cuh"
#include "device_common.cuh"
#include "pool_internal.h"
#include "quant.cuh"

using namespace pkv_dev;
using namespace pkv_axes_dev;
using namespace pkv_quant_dev;

namespace {

constexpr int kThreads = 256;
constexpr int kRowVecs = kHkv * kDim / 8;            // 16-byte vectors of a token's K (or V): 64
constexpr int kItems = kPage * kRowVecs / kThreads;  // of a page, per thread: 4
constexpr int kTileVecs = kQuantTile / 16;           // 130
constexpr int kPageVecs = kHkv * kTileVecs;

struct StoreParams {
  const int32_t* table;       // this layer's block tables [max_batch][table_stride]
  const int32_t* cu_tokens;
  const int32_t* start_pos;
  int* err;
  int table_stride;
  int num_pages;
  int max_seq_len;
  int max_chunk;
  int total_tokens;
};

// What a block does: tokens [first, first + count) of logical page `logical` of
// sequence blockIdx.y, whose packed rows start at `row`. The blocks of a
// sequence take the pages its chunk lies in, one each.
struct PageWork {
  int logical, page;
  int first, count;           // slots; count 0: nothing to do
  long long row;
};

__device__ __forceinline__ PageWork page_work(const StoreParams& prm) {
  PageWork w = {};
  const int b = blockIdx.y;
  const bool reports = threadIdx.x == 0;
  const int row0 = prm.cu_tokens[b];
  int n = prm.cu_tokens[b + 1] - row0;
  if (row0 < 0 || n < 0 || n > prm.total_tokens - row0) {   // rows outside the caller's buffers
    if (blockIdx.x == 0 && reports) set_error(prm.err, PKV_DEV_ERR_SEQ_LEN);
    return w;
  }
  if (n > prm.max_chunk) {
    if (blockIdx.x == 0 && reports) set_error(prm.err, PKV_DEV_ERR_SEQ_LEN);
    n = prm.max_chunk;
  }
  if (n == 0) return w;
  const int start = prm.start_pos[b];
  if (start < 0 || start >= prm.max_seq_len) {
    if (blockIdx.x == 0 && reports) set_error(prm.err, PKV_DEV_ERR_POSITION);
    return w;
  }
  if (n > prm.max_seq_len - start) {
    if (blockIdx.x == 0 && reports) set_error(prm.err, PKV_DEV_ERR_POSITION);
    n = prm.max_seq_len - start;
  }
  w.logical = start / kPage + blockIdx.x;
  const int from = max(start, w.logical * kPage);
  const int to = min(start + n, (w.logical + 1) * kPage);
  if (to <= from) return w;
  w.page = prm.table[static_cast<size_t>(b) * prm.table_stride + w.logical];
  if (w.page < 0 || w.page >= prm.num_pages) {
    if (reports) set_error(prm.err, PKV_DEV_ERR_PAGE);
    return w;
  }
  w.first = from % kPage;
  w.count = to - from;
  w.row = static_cast<long long>(row0) + (from - start);
  return w;
}

// A block per page. A thread's items are (token, head, chunk of 8 dims), the
// chunk fastest, so 8 lanes hold a row and a warp's loads are 512 contiguous
// bytes; all loads go out before the first is used. The tiles are put together
// in shared memory and leave as 16-byte vectors, the slots of this chunk's
// tokens alone.
template <bool kRope>
__global__ void __launch_bounds__(kThreads) quant_fill_kernel(
    const uint16_t* __restrict__ k, const uint16_t* __restrict__ v, uint8_t* pool,
    const StoreParams prm, const AxesArgs rope) {
  __shared__ __align__(16) uint8_t tiles[kHkv][kQuantTile];
  __shared__ float angles[kRope ? 2 : 1][kRope ? kPage : 1][kPairs];
  __shared__ uint32_t good_tokens;
  const PageWork w = page_work(prm);
  if (w.count == 0) return;
  uint4 kv[2][kItems];
  #pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const int item = threadIdx.x + i * kThreads;
    const int token = item / kRowVecs - w.first;       // of this page's
    if (token >= 0 && token < w.count) {
      const size_t at = static_cast<size_t>(w.row + token) * kRowVecs + item % kRowVecs;
      kv[0][i] = __ldcs(reinterpret_cast<const uint4*>(k) + at);
      kv[1][i] = __ldcs(reinterpret_cast<const uint4*>(v) + at);
    } else {
      kv[0][i] = kv[1][i] = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  uint32_t good = 0xffffu;
  if constexpr (kRope) {
    // a warp per token, lane i its pair i; a token whose position is outside
    // the tables is left out
    if (threadIdx.x == 0) good_tokens = 0u;
    __syncthreads();
    const int lane = threadIdx.x & 31;
    for (int t = threadIdx.x >> 5; t < w.count; t += kThreads / 32) {
      float c = 1.f, s = 0.f;
      const int p = pair_position(rope, w.row + t, lane);
      const bool ok = load_pair_angle(rope, p, lane, c, s);
      angles[0][w.first + t][lane] = c;
      angles[1][w.first + t][lane] = s;
      if (lane == 0) {
        if (ok) {
          atomicOr(&good_tokens, 1u << (w.first + t));
        } else {
          set_error(prm.err, PKV_DEV_ERR_POSITION);
        }
      }
    }
    __syncthreads();
    good = good_tokens;
  }
  #pragma unroll
  for (int i = 0; i < kItems; ++i) {
    const int item = threadIdx.x + i * kThreads;
    const int token = item / kRowVecs, head = item / 8 % kHkv, c = item % 8;
    uint8_t* tile = tiles[head];
    #pragma unroll
    for (int which = 0; which < 2; ++which) {
      float x[8];
      unpack8(kv[which][i], x);
      if (kRope && which == 0) {
        const uint4 own = kv[0][i];
        float partner[8], cs[8], sn[8];
        unpack8(make_uint4(__shfl_xor_sync(0xffffffffu, own.x, 4),
                           __shfl_xor_sync(0xffffffffu, own.y, 4),
                           __shfl_xor_sync(0xffffffffu, own.z, 4),
                           __shfl_xor_sync(0xffffffffu, own.w, 4)),
                partner);
        #pragma unroll
        for (int e = 0; e < 8; ++e) {
          cs[e] = angles[0][kRope ? token : 0][8 * (c & 3) + e];
          sn[e] = angles[kRope ? 1 : 0][kRope ? token : 0][8 * (c & 3) + e];
        }
        rotate8(x, partner, c >= 4, cs, sn);
      }
      uint2 codes;
      const uint32_t e = quantise_row(x, codes);
      *reinterpret_cast<uint2*>(tile + (which == 0 ? k_at(token, 8 * c) : v_at(token, 8 * c))) =
          codes;
      if (c == 0) tile[(which == 0 ? kKExp : kVExp) + token] = static_cast<uint8_t>(e);
    }
  }
  __syncthreads();
  const uint32_t mine = good & (((1u << w.count) - 1u) << w.first);
  uint4* to = reinterpret_cast<uint4*>(pool + static_cast<size_t>(w.page) * kHkv * kQuantTile);
  for (int i = threadIdx.x; i < kPageVecs; i += kThreads) {
    const int head = i / kTileVecs, vec = i % kTileVecs;
    const uint4 x = *reinterpret_cast<const uint4*>(tiles[head] + vec * 16);
    if (vec < kKExp / 16) {
      const int token = vec < kCodeBytes / 16 ? vec / (kDim / 16) : vec % kPage;
      if ((mine >> token) & 1u) to[i] = x;
    } else if (mine == 0xffffu) {
      to[i] = x;
    } else {
      uint8_t* bytes = reinterpret_cast<uint8_t*>(to + i);
      for (int t = w.first; t < w.first + w.count; ++t)
        if ((mine >> t) & 1u) bytes[t] = tiles[head][vec * 16 + t];
    }
  }
}

// A block per page. A thread's items are (head, chunk of 16 dims, token), the
// token fastest: a warp reads 512 contiguous bytes of V's codes and 32-byte
// pieces of K's, and writes 32-byte pieces of the rows.
__global__ void __launch_bounds__(kThreads) quant_read_kernel(
    const uint8_t* __restrict__ pool, uint16_t* k, uint16_t* v, const StoreParams prm) {
  constexpr int kReadItems = kPage * kHkv * kDim / 16 / kThreads;   // 2
  const PageWork w = page_work(prm);
  if (w.count == 0) return;
  uint4 codes[2][kReadItems];
  uint32_t exps[2][kReadItems];
  #pragma unroll
  for (int i = 0; i < kReadItems; ++i) {
    const int item = threadIdx.x + i * kThreads;
    const int slot = item % kPage, chunk = item / kPage % 4, head = item / (kPage * 4);
    if (slot < w.first || slot >= w.first + w.count) continue;
    const uint8_t* tile = pool + (static_cast<size_t>(w.page) * kHkv + head) * kQuantTile;
    codes[0][i] = *reinterpret_cast<const uint4*>(tile + k_at(slot, 16 * chunk));
    codes[1][i] = *reinterpret_cast<const uint4*>(tile + v_at(slot, 16 * chunk));
    exps[0][i] = tile[kKExp + slot];
    exps[1][i] = tile[kVExp + slot];
  }
  #pragma unroll
  for (int i = 0; i < kReadItems; ++i) {
    const int item = threadIdx.x + i * kThreads;
    const int slot = item % kPage, chunk = item / kPage % 4, head = item / (kPage * 4);
    if (slot < w.first || slot >= w.first + w.count) continue;
    const size_t at = (static_cast<size_t>(w.row + slot - w.first) * kHkv + head) * kDim + 16 * chunk;
    #pragma unroll
    for (int which = 0; which < 2; ++which) {
      const uint32_t c[4] = {codes[which][i].x, codes[which][i].y, codes[which][i].z,
                             codes[which][i].w};
      const float scale = scale_of(exps[which][i]);
      uint32_t out[8];
      #pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t h = e % 2 ? codes_to_half2<1>(c[e / 2]) : codes_to_half2<0>(c[e / 2]);
        float x0, x1;
        asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\t"
            "cvt.f32.f16 %1, u;\n\t}"
            : "=f"(x0), "=f"(x1)
            : "r"(h));
        out[e] = float2_to_bf16x2(x0 * scale, x1 * scale);   // exact
      }
      uint4* to = reinterpret_cast<uint4*>((which == 0 ? k : v) + at);
      to[0] = make_uint4(out[0], out[1], out[2], out[3]);
      to[1] = make_uint4(out[4], out[5], out[6], out[7]);
    }
  }
}

// What both calls check, and the launch's parameters; PKV_OK with *grid_x 0: nothing to do.
pkv_status check_store(pkv_pool_t pool, int layer, const void* k, const void* v,
                       const void* kv_pool, const int32_t* block_tables,
                       const int32_t* cu_tokens, const int32_t* start_pos, int batch,
                       int total_tokens, int max_chunk_tokens, StoreParams* prm, int* grid_x) {
  *grid_x = 0;
  if (!pool) return PKV_ERR_INVALID_ARG;
  const pkv_pool_config& c = pool->cfg;
  if (layer < 0 || layer >= c.num_layers || batch < 0 || batch > c.max_batch || total_tokens < 0)
    return PKV_ERR_INVALID_ARG;
  if (batch == 0 || total_tokens == 0) return PKV_OK;
  if (max_chunk_tokens < 1 || max_chunk_tokens > c.max_seq_len) return PKV_ERR_INVALID_ARG;
  if (!k || !v || !kv_pool || !block_tables || !cu_tokens || !start_pos)
    return PKV_ERR_INVALID_ARG;
  if (!pkv_aligned16(k) || !pkv_aligned16(v) || !pkv_aligned16(kv_pool) ||
      !pkv_aligned16(block_tables) || !pkv_aligned4(cu_tokens) || !pkv_aligned4(start_pos))
    return PKV_ERR_INVALID_ARG;
  const int stride = c.max_seq_len / kPage;
  prm->table = block_tables + static_cast<size_t>(layer) * c.max_batch * stride;
  prm->cu_tokens = cu_tokens;
  prm->start_pos = start_pos;
  prm->err = pool->err;
  prm->table_stride = stride;
  prm->num_pages = c.num_pages;
  prm->max_seq_len = c.max_seq_len;
  prm->max_chunk = max_chunk_tokens;
  prm->total_tokens = total_tokens;
  // the most pages that a chunk of so many tokens can lie in
  *grid_x = (max_chunk_tokens + kPage - 2) / kPage + 1;
  return PKV_OK;
}

bool on_device(const pkv_pool* pool) {
  int dev = -1;
  return cudaGetDevice(&dev) == cudaSuccess && dev == pool->device;
}

}  // namespace

extern "C" {

pkv_status pkv_quant_fill(pkv_pool_t pool, int layer, const void* k, const void* v, void* kv_pool,
                          const int32_t* block_tables, const int32_t* cu_tokens,
                          const int32_t* start_pos, const pkv_axes_rope* rope,
                          const int32_t* rope_positions, int position_stride, int batch,
                          int total_tokens, int max_chunk_tokens, void* stream) {
  StoreParams prm;
  int grid_x;
  pkv_status st = check_store(pool, layer, k, v, kv_pool, block_tables, cu_tokens, start_pos,
                              batch, total_tokens, max_chunk_tokens, &prm, &grid_x);
  if (st != PKV_OK || grid_x == 0) return st;
  AxesArgs axes = {};
  if (rope) {
    st = make_axes_args(rope, rope_positions, position_stride, total_tokens, &axes);
    if (st != PKV_OK) return st;
  }
  if (!on_device(pool)) return PKV_ERR_INVALID_ARG;
  pool->pages_written = true;
  const auto kernel = rope ? quant_fill_kernel<true> : quant_fill_kernel<false>;
  kernel<<<dim3(grid_x, batch), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v),
      static_cast<uint8_t*>(kv_pool), prm, axes);
  return pkv_check_launch();
}

pkv_status pkv_quant_read(pkv_pool_t pool, int layer, const void* kv_pool,
                          const int32_t* block_tables, const int32_t* cu_tokens,
                          const int32_t* start_pos, void* k, void* v, int batch, int total_tokens,
                          int max_chunk_tokens, void* stream) {
  StoreParams prm;
  int grid_x;
  const pkv_status st = check_store(pool, layer, k, v, kv_pool, block_tables, cu_tokens,
                                    start_pos, batch, total_tokens, max_chunk_tokens, &prm,
                                    &grid_x);
  if (st != PKV_OK || grid_x == 0) return st;
  if (!on_device(pool)) return PKV_ERR_INVALID_ARG;
  quant_read_kernel<<<dim3(grid_x, batch), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint8_t*>(kv_pool), static_cast<uint16_t*>(k), static_cast<uint16_t*>(v),
      prm);
  return pkv_check_launch();
}

}  // extern "C"
