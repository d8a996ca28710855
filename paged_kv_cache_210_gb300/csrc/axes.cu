// Prefill fill with rotation by several position axes (declared in
// include/pkv_axes.h): one pass reads a chunk's q, k and v, rotates q and k,
// writes q back and k and v into their pages.
//
// The work is memory traffic: 12 KiB per token (q, k, v read and written
// once) against 7.5 KFLOP, so HBM bounds it: eight 4,096-token prompts 60.4 us
// (6.6 TB/s, 99 % of the measured copy rate), eight of 1,536 to 2,048 tokens
// 28.3 us, of which the launch and the first loads are 2; a 77-token prompt 2.4
// us, all latency.

#include <cuda_runtime.h>
#include <stdint.h>

#include "pkv.h"
#include "pkv_axes.h"
#include "axes.cuh"
#include "device_common.cuh"
#include "pool_internal.h"

using namespace pkv_dev;
using namespace pkv_axes_dev;

namespace {

// Tokens per block (8: 31.0 us at eight 2,048-token prompts, 2: 28.3).
constexpr int kFillWarps = 2;

struct FillParams {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  uint16_t* q_out;
  uint16_t* k_pool;
  uint16_t* v_pool;
  const int32_t* table;       // this layer's block tables [max_batch][table_stride]
  const int32_t* cu_tokens;
  const int32_t* start_pos;
  int* err;
  int table_stride;
  int num_pages;
  int max_seq_len;
  int max_chunk;
  int total_tokens;
  AxesArgs rope;
};

// A warp per token. Lane i fetches pair i's cos and sin once and the lanes
// exchange them, so a token reads 256 bytes of tables whatever the axes of
// its pairs; lane (c, h) = (lane % 4, lane / 4) then rotates dims 8 c .. + 7
// with 32 + 8 c .. + 7 of q heads h, h + 8, h + 16, h + 24 and of KV head h, and
// copies two chunks of v: 12 loads of 16 bytes go out before the first use.
__global__ void __launch_bounds__(kFillWarps * 32) fill_axes_kernel(const FillParams prm) {
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.y;
  const int i = blockIdx.x * kFillWarps + warp;
  const int row0 = prm.cu_tokens[b];
  const int n = prm.cu_tokens[b + 1] - row0;
  if (row0 < 0 || n < 0 || n > prm.total_tokens - row0) {   // rows outside the caller's buffers
    if (i == 0 && lane == 0) set_error(prm.err, PKV_DEV_ERR_SEQ_LEN);
    return;
  }
  if (i == 0 && lane == 0 && n > prm.max_chunk) set_error(prm.err, PKV_DEV_ERR_SEQ_LEN);
  if (i >= n || i >= prm.max_chunk) return;
  const int start = prm.start_pos[b];
  if (start < 0 || start >= prm.max_seq_len || i >= prm.max_seq_len - start) {
    if (lane == 0) set_error(prm.err, PKV_DEV_ERR_POSITION);
    return;
  }
  const int pos = start + i;
  const long long row = static_cast<long long>(row0) + i;
  // the loads that depend on the row alone go out before the page id, the
  // positions and the angles are waited for
  const int page = prm.table[static_cast<size_t>(b) * prm.table_stride + pos / kPage];
  const int rope_pos = pair_position(prm.rope, row, lane);
  const int ch = lane & 3;
  const int h = lane >> 2;
  const bool has_q = prm.q != nullptr;
  const uint4* q4 = reinterpret_cast<const uint4*>(prm.q + (row * kHq + h) * kDim) + ch;
  const uint4* k4 = reinterpret_cast<const uint4*>(prm.k + (row * kHkv + h) * kDim) + ch;
  const uint4* v4 = reinterpret_cast<const uint4*>(prm.v + (row * kHkv + h) * kDim) + ch;
  constexpr int kHeadVecs = kDim / 8;                     // 16-byte vectors per head
  uint4 qlo[4], qhi[4];
  if (has_q) {
    #pragma unroll
    for (int e = 0; e < 4; ++e) {
      qlo[e] = q4[8 * e * kHeadVecs];
      qhi[e] = q4[8 * e * kHeadVecs + 4];
    }
  }
  uint4 klo = k4[0], khi = k4[4];
  const uint4 vlo = v4[0], vhi = v4[4];
  if (page < 0 || page >= prm.num_pages) {
    if (lane == 0) set_error(prm.err, PKV_DEV_ERR_PAGE);
    return;
  }
  float c, s;
  if (!load_pair_angle(prm.rope, rope_pos, lane, c, s)) {
    if (lane == 0) set_error(prm.err, PKV_DEV_ERR_POSITION);
    return;
  }
  float cs[8], sn[8];
  #pragma unroll
  for (int j = 0; j < 8; ++j) {
    cs[j] = __shfl_sync(0xffffffffu, c, 8 * ch + j);
    sn[j] = __shfl_sync(0xffffffffu, s, 8 * ch + j);
  }
  if (has_q) {
    uint4* o4 = reinterpret_cast<uint4*>(prm.q_out + (row * kHq + h) * kDim) + ch;
    #pragma unroll
    for (int e = 0; e < 4; ++e) {
      rotate_chunks(qlo[e], qhi[e], cs, sn);
      o4[8 * e * kHeadVecs] = qlo[e];
      o4[8 * e * kHeadVecs + 4] = qhi[e];
    }
  }
  rotate_chunks(klo, khi, cs, sn);
  const size_t at = ((static_cast<size_t>(page) * kHkv + h) * kPage + pos % kPage) * kDim;
  uint4* kd = reinterpret_cast<uint4*>(prm.k_pool + at) + ch;
  uint4* vd = reinterpret_cast<uint4*>(prm.v_pool + at) + ch;
  kd[0] = klo;
  kd[4] = khi;
  vd[0] = vlo;
  vd[4] = vhi;
}

}  // namespace

extern "C" pkv_status pkv_prefill_fill_axes(pkv_pool_t pool, int layer, const void* q,
                                            const void* k, const void* v, void* q_out,
                                            void* k_pool, void* v_pool,
                                            const int32_t* block_tables,
                                            const int32_t* cu_tokens, const int32_t* start_pos,
                                            const pkv_axes_rope* rope,
                                            const int32_t* rope_positions, int position_stride,
                                            int batch, int total_tokens, int max_chunk_tokens,
                                            void* stream) {
  if (!pool) return PKV_ERR_INVALID_ARG;
  const pkv_pool_config& c = pool->cfg;
  if (layer < 0 || layer >= c.num_layers || batch < 0 || batch > c.max_batch || total_tokens < 0)
    return PKV_ERR_INVALID_ARG;
  if (batch == 0 || total_tokens == 0) return PKV_OK;
  if (max_chunk_tokens < 1 || max_chunk_tokens > c.max_seq_len) return PKV_ERR_INVALID_ARG;
  if (!k || !v || !k_pool || !v_pool || !block_tables || !cu_tokens || !start_pos ||
      (q == nullptr) != (q_out == nullptr))
    return PKV_ERR_INVALID_ARG;
  if (!pkv_aligned16(q) || !pkv_aligned16(k) || !pkv_aligned16(v) || !pkv_aligned16(q_out) ||
      !pkv_aligned16(k_pool) || !pkv_aligned16(v_pool) || !pkv_aligned16(block_tables) ||
      !pkv_aligned4(cu_tokens) || !pkv_aligned4(start_pos))
    return PKV_ERR_INVALID_ARG;
  FillParams prm;
  const pkv_status st = make_axes_args(rope, rope_positions, position_stride, total_tokens,
                                       &prm.rope);
  if (st != PKV_OK) return st;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev != pool->device) return PKV_ERR_INVALID_ARG;
  const int stride = c.max_seq_len / kPage;
  prm.q = static_cast<const uint16_t*>(q);
  prm.k = static_cast<const uint16_t*>(k);
  prm.v = static_cast<const uint16_t*>(v);
  prm.q_out = static_cast<uint16_t*>(q_out);
  prm.k_pool = static_cast<uint16_t*>(k_pool);
  prm.v_pool = static_cast<uint16_t*>(v_pool);
  prm.table = block_tables + static_cast<size_t>(layer) * c.max_batch * stride;
  prm.cu_tokens = cu_tokens;
  prm.start_pos = start_pos;
  prm.err = pool->err;
  prm.table_stride = stride;
  prm.num_pages = c.num_pages;
  prm.max_seq_len = c.max_seq_len;
  prm.max_chunk = max_chunk_tokens;
  prm.total_tokens = total_tokens;
  pool->pages_written = true;
  fill_axes_kernel<<<dim3((max_chunk_tokens + kFillWarps - 1) / kFillWarps, batch),
                     kFillWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(prm);
  return pkv_check_launch();
}
