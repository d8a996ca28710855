// The 8-bit KV cache's fill and read-back (declared in include/pkv_quant.h).
//
// Both are memory traffic: 2,048 + 1,040 bytes a token either way (K and V of 8
// heads in BF16, and as codes with their exponents). Reading 120,500 tokens back takes
// 58 us (6.4 TB/s, 96 % of the measured copy rate), 14,200 8.9 us; filling 14,200
// rotated tokens 9.4 us (4.7 TB/s), of which three dependent loads (the lists, the page
// id and the rotary positions, the angles) are 2; 77 tokens 2.2 and 2.0 us, all
// latency. The fill took 11.6 us with a branch on each row's clamp and on each token's
// angle before the next one's load, 10.7 with the latter alone; a block per whole page
// whose tiles are put together in shared memory 15.2. A reading block whose threads held
// 16 codes took 83 us for the long read (it wrote half sectors).

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

// A block takes the tokens of a page, 4 per warp, and some of the KV heads: 8 lanes
// hold a row, 8 dims each (of a key to be rotated, 4 dims and their 4 partners). Of one
// head a warp then moves 256 contiguous bytes of K's codes, four pieces of 64 bytes of
// V's and four of 128 bytes on the BF16 side.
constexpr int kThreads = 128;
constexpr int kWarpTokens = 32 / 8;
constexpr int kReadHeads = 2;                        // of a block
// KV heads of a fill block: 2 shorten a small call (77 tokens 2.2 us, with 4 2.5; 2,048
// 3.1 and 3.2), 4 have more loads in flight and the angles for more (6,144 tokens 5.1
// us, with 2 5.7; 16,384 10.5 and 11.1).
constexpr int kFewFillHeads = 2, kManyFillHeads = 4;
constexpr int kManyTokens = 4096;
static_assert(kThreads / 32 * kWarpTokens == kPage, "a block's warps cover a page");

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

// What a block does: slots [first, first + count) of a page of sequence blockIdx.y,
// whose packed rows start at `row`. The blocks of a sequence take the pages its
// chunk lies in.
struct PageWork {
  int page;                   // its id, not checked
  int first, count;           // count 0: nothing to do
  long long row;
};

__device__ __forceinline__ PageWork page_work(const StoreParams& prm, int index) {
  PageWork w = {};
  const int b = blockIdx.y;
  const bool reports = threadIdx.x == 0 && blockIdx.x == 0;
  const int row0 = prm.cu_tokens[b];
  int n = prm.cu_tokens[b + 1] - row0;
  const int start = prm.start_pos[b];
  if (row0 < 0 || n < 0 || n > prm.total_tokens - row0) {   // rows outside the caller's buffers
    if (reports) set_error(prm.err, PKV_DEV_ERR_SEQ_LEN);
    return w;
  }
  if (n > prm.max_chunk) {
    if (reports) set_error(prm.err, PKV_DEV_ERR_SEQ_LEN);
    n = prm.max_chunk;
  }
  if (n == 0) return w;
  if (start < 0 || start >= prm.max_seq_len || n > prm.max_seq_len - start) {
    if (reports) set_error(prm.err, PKV_DEV_ERR_POSITION);
    if (start < 0 || start >= prm.max_seq_len) return w;
    n = prm.max_seq_len - start;
  }
  const int logical = start / kPage + index;
  const int from = max(start, logical * kPage);
  const int to = min(start + n, (logical + 1) * kPage);
  if (to <= from) return w;
  w.page = prm.table[static_cast<size_t>(b) * prm.table_stride + logical];
  w.first = from % kPage;
  w.count = to - from;
  w.row = static_cast<long long>(row0) + (from - start);
  return w;
}

// The rows' loads and the rotary positions' go out before the page id is waited for,
// the angles' all at once.
template <bool kRope, int kFillHeads>
__global__ void __launch_bounds__(kThreads) quant_fill_kernel(
    const uint16_t* __restrict__ k, const uint16_t* __restrict__ v, uint8_t* pool,
    const StoreParams prm, const AxesArgs rope) {
  __shared__ float2 angles[kRope ? kThreads / 32 : 1][kRope ? kWarpTokens : 1][kPairs];
  constexpr int kGroups = kHkv / kFillHeads;
  const PageWork w = page_work(prm, blockIdx.x / kGroups);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp * kWarpTokens >= w.first + w.count || (warp + 1) * kWarpTokens <= w.first) return;
  const int head0 = blockIdx.x % kGroups * kFillHeads;
  const int slot = warp * kWarpTokens + lane / 8, c = lane % 8;
  bool valid = slot >= w.first && slot < w.first + w.count;
  const size_t from = static_cast<size_t>(w.row + slot - w.first) * (kHkv * kDim) + head0 * kDim;
  uint4 kv[2][kFillHeads];
  #pragma unroll
  for (int h = 0; h < kFillHeads; ++h) {
    kv[0][h] = kv[1][h] = make_uint4(0u, 0u, 0u, 0u);
    if (valid) {
      if constexpr (kRope) {
        const uint2* row = reinterpret_cast<const uint2*>(k + from + kDim * h);
        const uint2 lo = __ldcs(row + c), hi = __ldcs(row + 8 + c);
        kv[0][h] = make_uint4(lo.x, lo.y, hi.x, hi.y);
      } else {
        kv[0][h] = __ldcs(reinterpret_cast<const uint4*>(k + from + kDim * h) + c);
      }
      kv[1][h] = __ldcs(reinterpret_cast<const uint4*>(v + from + kDim * h) + c);
    }
  }
  float2 cs[2], sn[2];
  if constexpr (kRope) {
    // lane i fetches pair i's angle of each of the warp's tokens; a token whose
    // position is outside the tables is left out
    int pos[kWarpTokens];
    #pragma unroll
    for (int t = 0; t < kWarpTokens; ++t) {
      const int s = warp * kWarpTokens + t - w.first;
      pos[t] = s >= 0 && s < w.count ? pair_position(rope, w.row + s, lane) : 0;
    }
    bool all_good = true;
    #pragma unroll
    for (int t = 0; t < kWarpTokens; ++t) {
      if (!__all_sync(0xffffffffu, pos[t] >= 0 && pos[t] < rope.rows)) {
        all_good = false;
        pos[t] = 0;
        if (lane / 8 == t) valid = false;
      }
    }
    if (!all_good && lane == 0) set_error(prm.err, PKV_DEV_ERR_POSITION);
    float2 mine[kWarpTokens];
    #pragma unroll
    for (int t = 0; t < kWarpTokens; ++t) {
      const size_t at = static_cast<size_t>(pos[t]) * kPairs + lane;
      mine[t] = make_float2(__ldg(rope.cos + at), __ldg(rope.sin + at));
    }
    #pragma unroll
    for (int t = 0; t < kWarpTokens; ++t) angles[warp][t][lane] = mine[t];
    __syncwarp();
    #pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float4 a = *reinterpret_cast<const float4*>(&angles[warp][lane / 8][4 * c + 2 * e]);
      cs[e] = make_float2(a.x, a.z);
      sn[e] = make_float2(a.y, a.w);
    }
  }
  const bool good_page = w.page >= 0 && w.page < prm.num_pages;
  if (!good_page) {
    if (lane == 0) set_error(prm.err, PKV_DEV_ERR_PAGE);
    return;
  }
  uint8_t* tile = pool + (static_cast<size_t>(w.page) * kHkv + head0) * kQuantTile;
  #pragma unroll
  for (int which = 0; which < 2; ++which) {
    float2 x[kFillHeads][4];
    #pragma unroll
    for (int h = 0; h < kFillHeads; ++h) {
      unpack8(kv[which][h], x[h]);
      if (kRope && which == 0) rotate_halves(x[h], cs, sn);
    }
    uint2 codes[kFillHeads];
    uint32_t exps[kFillHeads];
    quantise_rows(x, codes, exps);
    if (valid) {
      #pragma unroll
      for (int h = 0; h < kFillHeads; ++h) {
        uint8_t* to = tile + h * kQuantTile;
        if (kRope && which == 0) {
          *reinterpret_cast<uint32_t*>(to + k_at(slot, 4 * c)) = codes[h].x;
          *reinterpret_cast<uint32_t*>(to + k_at(slot, kDim / 2 + 4 * c)) = codes[h].y;
        } else {
          *reinterpret_cast<uint2*>(to + (which == 0 ? k_at(slot, 8 * c) : v_at(slot, 8 * c))) =
              codes[h];
        }
        if (c == 0) to[(which == 0 ? kKExp : kVExp) + slot] = static_cast<uint8_t>(exps[h]);
      }
    }
  }
}

__global__ void __launch_bounds__(kThreads) quant_read_kernel(
    const uint8_t* __restrict__ pool, uint16_t* k, uint16_t* v, const StoreParams prm) {
  constexpr int kGroups = kHkv / kReadHeads;
  const PageWork w = page_work(prm, blockIdx.x / kGroups);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp * kWarpTokens >= w.first + w.count || (warp + 1) * kWarpTokens <= w.first) return;
  if (w.page < 0 || w.page >= prm.num_pages) {
    if (lane == 0) set_error(prm.err, PKV_DEV_ERR_PAGE);
    return;
  }
  const int head0 = blockIdx.x % kGroups * kReadHeads;
  const int slot = warp * kWarpTokens + lane / 8, c = lane % 8;
  if (slot < w.first || slot >= w.first + w.count) return;
  const uint8_t* tile = pool + (static_cast<size_t>(w.page) * kHkv + head0) * kQuantTile;
  uint2 codes[2][kReadHeads];
  uint32_t exps[2][kReadHeads];
  #pragma unroll
  for (int h = 0; h < kReadHeads; ++h, tile += kQuantTile) {
    codes[0][h] = __ldcs(reinterpret_cast<const uint2*>(tile + k_at(slot, 8 * c)));
    codes[1][h] = __ldcs(reinterpret_cast<const uint2*>(tile + v_at(slot, 8 * c)));
    exps[0][h] = tile[kKExp + slot];
    exps[1][h] = tile[kVExp + slot];
  }
  const size_t to = static_cast<size_t>(w.row + slot - w.first) * (kHkv * kDim / 8) + head0 * 8 + c;
  #pragma unroll
  for (int h = 0; h < kReadHeads; ++h) {
    #pragma unroll
    for (int which = 0; which < 2; ++which) {
      const float scale = scale_of(exps[which][h]);
      uint32_t out[4];
      #pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t two = e < 2 ? codes[which][h].x : codes[which][h].y;
        const uint32_t half2 = e % 2 ? codes_to_half2<1>(two) : codes_to_half2<0>(two);
        float x0, x1;
        asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\t"
            "cvt.f32.f16 %1, u;\n\t}"
            : "=f"(x0), "=f"(x1)
            : "r"(half2));
        out[e] = float2_to_bf16x2(x0 * scale, x1 * scale);   // exact
      }
      __stcs(reinterpret_cast<uint4*>(which == 0 ? k : v) + to + 8 * h,
             make_uint4(out[0], out[1], out[2], out[3]));
    }
  }
}

// What both calls check, and the launch's parameters; PKV_OK with *pages 0: nothing to do.
pkv_status check_store(pkv_pool_t pool, int layer, const void* k, const void* v,
                       const void* kv_pool, const int32_t* block_tables,
                       const int32_t* cu_tokens, const int32_t* start_pos, int batch,
                       int total_tokens, int max_chunk_tokens, StoreParams* prm, int* pages) {
  *pages = 0;
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
  *pages = (max_chunk_tokens + kPage - 2) / kPage + 1;
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
  int pages;
  pkv_status st = check_store(pool, layer, k, v, kv_pool, block_tables, cu_tokens, start_pos,
                              batch, total_tokens, max_chunk_tokens, &prm, &pages);
  if (st != PKV_OK || pages == 0) return st;
  AxesArgs axes = {};
  if (rope) {
    st = make_axes_args(rope, rope_positions, position_stride, total_tokens, &axes);
    if (st != PKV_OK) return st;
  }
  if (!on_device(pool)) return PKV_ERR_INVALID_ARG;
  pool->pages_written = true;
  const bool many = total_tokens >= kManyTokens;
  const int heads = many ? kManyFillHeads : kFewFillHeads;
  const auto kernel = many ? (rope ? quant_fill_kernel<true, kManyFillHeads>
                                   : quant_fill_kernel<false, kManyFillHeads>)
                           : (rope ? quant_fill_kernel<true, kFewFillHeads>
                                   : quant_fill_kernel<false, kFewFillHeads>);
  kernel<<<dim3(pages * (kHkv / heads), batch), kThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint16_t*>(k), static_cast<const uint16_t*>(v),
      static_cast<uint8_t*>(kv_pool), prm, axes);
  return pkv_check_launch();
}

pkv_status pkv_quant_read(pkv_pool_t pool, int layer, const void* kv_pool,
                          const int32_t* block_tables, const int32_t* cu_tokens,
                          const int32_t* start_pos, void* k, void* v, int batch, int total_tokens,
                          int max_chunk_tokens, void* stream) {
  StoreParams prm;
  int pages;
  const pkv_status st = check_store(pool, layer, k, v, kv_pool, block_tables, cu_tokens,
                                    start_pos, batch, total_tokens, max_chunk_tokens, &prm,
                                    &pages);
  if (st != PKV_OK || pages == 0) return st;
  if (!on_device(pool)) return PKV_ERR_INVALID_ARG;
  quant_read_kernel<<<dim3(pages * (kHkv / kReadHeads), batch), kThreads, 0,
                      static_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint8_t*>(kv_pool), static_cast<uint16_t*>(k), static_cast<uint16_t*>(v),
      prm);
  return pkv_check_launch();
}

}  // extern "C"
