// Windowed prefill attention over the paged KV cache for GB300 (sm_103a): a
// chunk's tokens attend behind a sliding window, with sinks (declared in
// include/pkv_window.h).
//
// out_i = sum_t p_it V_t / sum_t p_it, p_it = 2^(q_i.K_t log2(e) / 8 - m_i), over
// the tokens visible from position p_i: one pass per 32-token query tile
// with a running maximum m_i and sum per row.
//
// The kernel is prefill_tiles.cuh's; here are its tiles: 32 tokens of a chunk and
// the pages they see.
//
// What bounds it: the softmax warps, two per scheduler, and of their time less
// the arithmetic (maximum, exponentials, sums, the split into three terms: 1,200
// cycles for two warps by itself, measured alone) than what a warp waits for in
// turn: its barriers, tensor memory, votes and instructions. A step of two CTAs
// takes about 2,000 cycles, against 1,024 of the tensor pipe (16 products of 32
// cycles each); a tile's start and end cost it some 4,000 more. The products are
// never waited for: every barrier of theirs is complete when it is first looked
// at. Two 4,096-token chunks behind a 4,096-token window: 463 us (596 TFLOP/s of
// score and value products counted once); eight prompts of up to 2,048 tokens
// behind 512: 111 us; sixteen of 512 tokens behind 128: 44.3 us. What was measured
// on the way, the first of these: 718 us as a plain port of the step loop; 696
// with the products issued by a converged warp (one thread in a divergent branch
// takes 55 cycles an issue for its operands); 654 with the split's subtractions
// in mixed precision; 613 with O summed in registers (192 a thread, setmaxnreg)
// instead of shared memory; 534 with one hand-over of P per step, one flag
// instead of a step's edge tests and failure paths placed out of line; 523 with
// page ids fetched ahead; 505 with barriers looked at ahead of their use and
// predicated arrivals; 472 with O joined behind the first half of P, when the
// products it waits for are long done; 483 with segments of two steps instead of
// four; 469 with steps of any four pages; 465 with the next tile looked up under
// the last product; 467 with no tile drawn that does not exist; 463 with the limit
// that a step's maximum is compared with kept between steps. The second: 159
// us up to the page ids, one CTA per tile; 134 with tiles drawn by resident CTAs,
// V cleared by its loader and results written through shared memory; 122 with
// word masks and a first tile that needs no draw; 112, and 111 with the last of
// the above, at the end. Slower: two threads per row (16 softmax warps per SM, by
// 10 %), and the first half of P taken against the running maximum before the
// step's own is known, done again for a row that outgrew it (by 12 %).

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "pkv.h"
#include "pkv_window.h"
#include "device_common.cuh"
#include "pool_internal.h"
#include "prefill_device.cuh"
#include "prefill_tiles.cuh"

using namespace pkv_tiles;

namespace {

struct WindowPrefillParams : TileParams {
  unsigned long long* next_tile;   // shared by the launch's CTAs; zero before and after it
  unsigned int* ctas_done;         // the same
  int tiles_max;              // tiles per sequence the launch covers
};

struct WindowWork {
  int b, g, row, count, bad_page;
  int p_first;    // position of the tile's first row
};

// What the tile (and each of its steps) sees of the sequence.
struct WindowView {
  int p_first;           // position of the tile's first token
  int n_keys;            // position of its last token + 1
  int lo;                // first key inside some row's window
  int sinks;
  int sink_pages;        // pages of sinks before the window's
  int win_page;          // the window's first page
  int n_pages;
  int n_steps;
  int plain_from, plain_to;   // steps whose keys every row sees

  __device__ WindowView(const WindowWork& work, const WindowPrefillParams& prm) {
    const int first = work.p_first, window = prm.window;
    p_first = first;
    n_keys = first + work.count;
    lo = max(first - window + 1, 0);
    sinks = prm.sinks;
    win_page = lo / kPage;
    sink_pages = min((sinks + kPage - 1) / kPage, win_page);
    n_pages = sink_pages + (n_keys + kPage - 1) / kPage - win_page;
    n_steps = (n_pages + kStepPages - 1) / kStepPages;
    const int hidden = n_keys - 1 - window;    // the last key outside some row's window
    const int whole_from = hidden < sinks ? 0 : sink_pages + hidden / kPage + 1 - win_page;
    const int whole_to = sink_pages + (first + 1) / kPage - win_page;
    plain_from = (whole_from + kStepPages - 1) / kStepPages;
    plain_to = whole_to / kStepPages;
  }
  static __device__ constexpr int first_step() { return 0; }
  __device__ bool has_page(int i) const { return i < n_pages; }
  // whether no row of the tile sees the key
  __device__ bool dead(int key) const { return key >= n_keys || (key >= sinks && key < lo); }
  // logical page i of the tile; past the last one (i >= n_pages) it has no key
  __device__ int page(int i) const { return i < sink_pages ? i : i - sink_pages + win_page; }
  // whether step j has keys that no row sees: past the last key, past the
  // sinks, or before the window
  __device__ bool has_dead(int j) const {
    return (j == n_steps - 1 && (n_pages % kStepPages != 0 || n_keys % kPage != 0)) ||
           (sinks < sink_pages * kPage && j == (sink_pages - 1) / kStepPages) ||
           (max(win_page * kPage, sinks) < lo && j == sink_pages / kStepPages);
  }
};

// The launch's tiles in the order they are drawn: 32 sequences at a time and, of
// those, heaviest first (the last tile of each sequence that has as many as any,
// then the one before it, ...). Only tiles that exist are numbered, so a draw
// costs the same whatever the launch's bounds are (a 32-token chunk under a bound
// of 131,072 takes 7 us; with every tile below the bound drawn, 238). Held by one
// warp, which asks for ever larger numbers; lane i looks after the i-th of the 32
// sequences, the next 32 sequences' lists are on their way meanwhile. (Numbered
// sequence by sequence, sixteen prompts of 512 tokens behind 128 took 48 us
// instead of 44.)
struct WindowWalk {
  int first = -32;                // the first of the 32 sequences
  int row0, rows, start;          // this lane's
  int tiles = 0;                  // ... 0 if it has none or its data is bad
  int top = 0, bottom = 0;        // tiles top - 1 .. bottom belong to the same sequences, ...
  uint32_t in = 0;                // ... these
  uint32_t before = 0, here = 0;  // tiles in front of those; how many they are
  int nth;                        // this lane's place among `in`, -1 if it is not one of them
  float per_level;                // 1 / the number of `in`
  int ahead_row0, ahead_end, ahead_start;

  __device__ __forceinline__ void fetch(const WindowPrefillParams& prm, int b) {
    ahead_row0 = ahead_end = ahead_start = 0;
    if (b < prm.batch) {
      ahead_row0 = prm.cu_tokens[b];
      ahead_end = prm.cu_tokens[b + 1];
      ahead_start = prm.start_pos[b];
    }
  }

  // Tile n: its sequence (with that one's first row, rows and position) and its
  // place in it. False past the last one. Called by a whole warp.
  __device__ __forceinline__ bool find(uint32_t n, const WindowPrefillParams& prm, int lane,
                                       int& b, int& tile, int& b_row0, int& b_rows,
                                       int& b_start) {
    while (n >= before + here) {
      before += here;
      top = bottom;
      while (top == 0) {
        first += 32;
        if (first >= prm.batch) return false;
        take(prm, lane);
        top = __reduce_max_sync(0xffffffffu, tiles);
      }
      in = __ballot_sync(0xffffffffu, tiles >= top);
      bottom = __reduce_max_sync(0xffffffffu, tiles < top ? tiles : 0);
      here = static_cast<uint32_t>(__popc(in) * (top - bottom));
      nth = (in >> lane & 1u) ? __popc(in & ((1u << lane) - 1u)) : -1;
      per_level = __fdividef(1.f, static_cast<float>(__popc(in)));
    }
    // down / count, exact: down < 2^20, so the product's error stays below a
    // quarter of 1 / count, and (down + 1/2) / count is half of it or more away
    // from an integer
    const int down = static_cast<int>(n - before);
    const int level = static_cast<int>((static_cast<float>(down) + 0.5f) * per_level);
    tile = top - 1 - level;
    const int from =
        __ffs(__ballot_sync(0xffffffffu, nth == down - level * __popc(in))) - 1;
    b = first + from;
    b_row0 = __shfl_sync(0xffffffffu, row0, from);
    b_rows = __shfl_sync(0xffffffffu, rows, from);
    b_start = __shfl_sync(0xffffffffu, start, from);
    return true;
  }

  // Tile `index` of the launch, the 8 KV heads of a tile in a row.
  __device__ __forceinline__ bool next(unsigned long long index, const WindowPrefillParams& prm,
                                       int lane, WindowWork& work) {
    int b, tile, b_row0, b_rows, b_start;
    if (!find(static_cast<uint32_t>(index / kHkv), prm, lane, b, tile, b_row0, b_rows, b_start))
      return false;
    work.b = b;
    work.g = static_cast<int>(index % kHkv);
    work.row = b_row0 + tile * kTileTokens;
    work.p_first = b_start + tile * kTileTokens;
    work.count = min(kTileTokens, b_rows - tile * kTileTokens);
    return true;
  }

  // The sequences fetched ahead; the first CTA reports those whose data is bad.
  __device__ __forceinline__ void take(const WindowPrefillParams& prm, int lane) {
    row0 = ahead_row0;
    rows = ahead_end - row0;
    start = ahead_start;
    // rows outside the caller's buffers
    const bool bad_rows = row0 < 0 || rows < 0 || rows > prm.total_tokens - row0;
    const bool bad_start = !bad_rows && rows > 0 &&
                           (start < 0 || start > prm.max_seq_len || rows > prm.max_seq_len - start);
    if (rarely(blockIdx.x == 0)) {
      if (bad_rows || rows > prm.tiles_max * kTileTokens) set_error(prm.err, PKV_DEV_ERR_SEQ_LEN);
      if (bad_start) set_error(prm.err, PKV_DEV_ERR_POSITION);
    }
    tiles = bad_rows || bad_start
                ? 0
                : min(rows / kTileTokens + (rows % kTileTokens != 0 ? 1 : 0), prm.tiles_max);
    fetch(prm, first + 32 + lane);
  }
};

struct WindowJob {
  using Params = WindowPrefillParams;
  using Work = WindowWork;
  using View = WindowView;
  using Walk = WindowWalk;
  static constexpr bool kFewRows = false;
  static constexpr bool kParts = false;
  static constexpr bool kDrawn = true;
  static __device__ constexpr bool is_whole(const Work&) { return true; }
  struct Row {
    int pos, window;
    __device__ Row(const Work& work, const Params& prm, int tok)
        : pos(work.p_first + tok), window(prm.window) {}
    // the keys of the page at `base` that the row sees (16 bits)
    __device__ __forceinline__ uint32_t seen(const View& view, int base) const {
      return low_bits32(pos + 1 - base) &
             (low_bits32(view.sinks - base) | ~low_bits32(pos - window + 1 - base));
    }
  };
};

}  // namespace

extern "C" pkv_status pkv_window_prefill_attention(
    pkv_pool_t pool, int layer, const void* q, const void* k_pool, const void* v_pool,
    const int32_t* block_tables, const int32_t* cu_tokens, const int32_t* start_pos, float* out,
    int window, int sinks, int batch, int total_tokens, int max_chunk_tokens, void* stream) {
  if (!pool) return PKV_ERR_INVALID_ARG;
  const pkv_pool_config& c = pool->cfg;
  if (layer < 0 || layer >= c.num_layers || batch < 0 || batch > c.max_batch ||
      total_tokens < 0 || window < 1 || sinks < 0)
    return PKV_ERR_INVALID_ARG;
  if (batch == 0 || total_tokens == 0) return PKV_OK;
  if (max_chunk_tokens < 1 || max_chunk_tokens > c.max_seq_len) return PKV_ERR_INVALID_ARG;
  if (!q || !k_pool || !v_pool || !block_tables || !cu_tokens || !start_pos || !out ||
      !pkv_aligned16(q) || !pkv_aligned16(k_pool) || !pkv_aligned16(v_pool) ||
      !pkv_aligned16(block_tables) || !pkv_aligned4(cu_tokens) || !pkv_aligned4(start_pos) ||
      !pkv_aligned16(out))
    return PKV_ERR_INVALID_ARG;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev != pool->device) return PKV_ERR_INVALID_ARG;
  if (!set_smem_attribute<WindowJob>(pool->device)) return PKV_ERR_CUDA;

  CUtensorMap tq, tk, tv;
  const cuuint64_t dims[3] = {kDim, kHq, static_cast<cuuint64_t>(total_tokens)};
  const cuuint64_t strides[2] = {kRowBytes, static_cast<cuuint64_t>(kHq) * kRowBytes};
  const cuuint32_t box[3] = {kDim, kGroup, kTileTokens};
  if (!encode_bf16(&tq, q, 3, dims, strides, box) ||
      !pkv_pool_tensor_map(k_pool, c.num_pages, &tk) ||
      !pkv_pool_tensor_map(v_pool, c.num_pages, &tv))
    return PKV_ERR_CUDA;
  const int stride = c.max_seq_len / kPage;
  WindowPrefillParams prm;
  prm.table = block_tables + static_cast<size_t>(layer) * c.max_batch * stride;
  prm.cu_tokens = cu_tokens;
  prm.start_pos = start_pos;
  prm.out = out;
  prm.err = pool->err;
  prm.num_pages = c.num_pages;
  prm.table_stride = stride;
  prm.max_seq_len = c.max_seq_len;
  prm.tiles_max = (max_chunk_tokens + kTileTokens - 1) / kTileTokens;
  prm.total_tokens = total_tokens;
  prm.window = std::min(window, c.max_seq_len);
  prm.sinks = std::min(sinks, c.max_seq_len);
  prm.batch = batch;
  // every CTA of a wave takes tiles until none is left; there are at most so many
  prm.next_tile = pool->prefill_next;
  prm.ctas_done = reinterpret_cast<unsigned int*>(pool->prefill_next + 1);
  const long long tiles = std::min(static_cast<long long>(prm.tiles_max) * batch,
                                   static_cast<long long>(total_tokens) / kTileTokens + batch);
  const int ctas =
      static_cast<int>(std::min<long long>(tiles * kHkv, kCtasPerSm * pool->num_sms));
  tile_attention_kernel<WindowJob>
      <<<ctas, kThreads, kSmemBytes<WindowJob>, static_cast<cudaStream_t>(stream)>>>(tq, tk, tv,
                                                                                 prm);
  return pkv_check_launch();
}
