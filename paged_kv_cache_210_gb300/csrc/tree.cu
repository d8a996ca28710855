// Attention of drafted token trees over the paged KV cache for GB300 (sm_103a),
// and the commit of an accepted path (declared in include/pkv_tree.h).
//
// The attention kernel is prefill_tiles.cuh's. A tile is up to 32 drafted tokens
// of one sequence and KV head (128 rows) and a part of the keys they see: the
// sink pages, the window's and the drafted tokens' own. Trees are few rows over
// long contexts, so a tile's steps are split into parts of about equal length,
// as many as the device holds CTAs, and a second kernel joins the parts' sums.

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

using namespace pkv_tiles;

namespace {

constexpr int kMaxTree = PKV_MAX_TREE;
// A tile's start and end cost a CTA about as much as two steps; a CTA is given no
// less than kLeastCost.
constexpr int kTileCost = 2;
constexpr int kLeastCost = 4;

struct TreeParams : TileParams {
  const unsigned long long* tree;   // [total] which drafted tokens each row sees
  float* part_o;                    // [2 wave][8][128][64] sums of parts, not divided
  float2* part_ml;                  // [2 wave][8][128] their exponent and sum of weights
  int wave;                         // CTAs of one wave, per KV head
};

struct TreeWork {
  int b, g, row, count, bad_page;
  int start;            // committed tokens
  int nodes;            // drafted tokens of the sequence
  int lo;               // first committed token inside some row's window
  int top;              // the largest position of a row
  int first_node;       // the tile's first drafted token
  int step, steps;      // its part
  int slot;             // of the part's sums; -1: all of the tile's steps
};

// The pages and steps a sequence lists: from the first token that a row at
// position start - 1 could see, so that they follow from its length alone. What
// no row sees of them is left out when they are read.
struct TreePages {
  int win_page, sink_pages, n_pages;
  __device__ TreePages(int start, int nodes, int window, int sinks) {
    win_page = max(start - window, 0) / kPage;
    sink_pages = min((sinks + kPage - 1) / kPage, win_page);
    n_pages = sink_pages + (start + nodes + kPage - 1) / kPage - win_page;
  }
  __device__ int steps() const { return (n_pages + kStepPages - 1) / kStepPages; }
};

struct TreeView {
  int win_page, sink_pages, n_pages;
  int n_keys, lo, sinks, start;
  int step0, n_steps;
  int plain_from, plain_to;

  __device__ TreeView(const TreeWork& work, const TreeParams& prm) {
    const TreePages pages(work.start, work.nodes, prm.window, prm.sinks);
    win_page = pages.win_page;
    sink_pages = pages.sink_pages;
    n_pages = pages.n_pages;
    start = work.start;
    n_keys = work.start + work.nodes;
    lo = work.lo;
    sinks = prm.sinks;
    step0 = work.step;
    n_steps = work.steps;
    const int hidden = work.top - prm.window;     // the last key outside some row's window
    const int whole_from = hidden < sinks ? 0 : sink_pages + hidden / kPage + 1 - win_page;
    const int whole_to = sink_pages + start / kPage - win_page;
    plain_from = (whole_from + kStepPages - 1) / kStepPages - step0;
    plain_to = whole_to / kStepPages - step0;
  }
  __device__ int first_step() const { return step0; }
  __device__ int page(int i) const { return i < sink_pages ? i : i - sink_pages + win_page; }
  // a page of the list with a token that some row may see
  __device__ bool has_page(int i) const {
    return i < n_pages && (i < sink_pages || (page(i) + 1) * kPage > lo || page(i) * kPage < sinks);
  }
  // whether no row sees the key: past the last drafted token, or between the sinks
  // and the window
  __device__ bool dead(int key) const { return key >= n_keys || (key >= sinks && key < lo); }
  // whether step j of the part has keys that no row sees
  __device__ bool has_dead(int j) const {
    const int from = (step0 + j) * kStepPages, to = from + kStepPages;
    return to > n_pages || (to == n_pages && n_keys % kPage != 0) ||
           (sinks < sink_pages * kPage && from < sink_pages && to >= sink_pages) ||
           (lo > max(win_page * kPage, sinks) && to > sink_pages &&
            from <= sink_pages + (lo - 1) / kPage - win_page);
  }
};

// How the launch's work is shared out. All tiles one after the other (sequence by
// sequence, a tile kTileCost before its steps) make a line of `total` places; of
// `ctas` CTAs per KV head number c takes [total c / ctas, total (c + 1) / ctas), so
// all take equally long whatever the lengths are, and a tile may be cut anywhere.
// (Parts of one length per launch left a fifth of the device idle: 8 trees of 64
// over 20,000 to 32,700 tokens took 254 us, shared out 205.)
//
// A CTA has at most one part of a tile that began before it, kept in slot 2 c, and
// one of a tile that goes on behind it, in slot 2 c + 1.
struct TreeShares {
  long long total;
  int ctas;
  __device__ void set(long long all, int wave) {
    total = all;
    ctas = static_cast<int>(min(max(total / kLeastCost, 1ll), static_cast<long long>(wave)));
  }
  __device__ long long begin(int c) const { return quotient(total * c, ctas); }
  // the last CTA that begins at or before `place`
  __device__ int owner(long long place) const {
    return static_cast<int>(quotient((place + 1) * ctas - 1, total));
  }
  // x / y, in 32 bits where they fit: a division in 64 is some 100 instructions on
  // the way to a CTA's first copy
  static __device__ long long quotient(long long x, long long y) {
    return (x | y) >> 32 ? x / y
                         : static_cast<long long>(static_cast<uint32_t>(x) / static_cast<uint32_t>(y));
  }
};

// The sequences of 32 lanes: what each brings, and where on the line.
struct TreeLane {
  int row0, nodes, start, steps;

  // Sequence b: steps 0 if there is none or its data is bad.
  __device__ __forceinline__ void load(const TreeParams& prm, int b, bool report) {
    steps = nodes = row0 = start = 0;
    if (b >= prm.batch) return;
    row0 = prm.cu_tokens[b];
    const int rows = prm.cu_tokens[b + 1] - row0;
    start = prm.start_pos[b];
    const bool bad_rows = row0 < 0 || rows < 0 || rows > prm.total_tokens - row0 || rows > kMaxTree;
    const bool bad_start = !bad_rows && rows > 0 &&
                           (start < 0 || start > prm.max_seq_len || rows > prm.max_seq_len - start);
    if (report) {
      if (bad_rows) set_error(prm.err, PKV_DEV_ERR_SEQ_LEN);
      if (bad_start) set_error(prm.err, PKV_DEV_ERR_POSITION);
    }
    if (bad_rows || bad_start || rows == 0) return;
    nodes = rows;
    steps = TreePages(start, nodes, prm.window, prm.sinks).steps();
  }
  __device__ __forceinline__ int tiles() const { return (nodes + kTileTokens - 1) / kTileTokens; }
  __device__ __forceinline__ int cost() const { return tiles() * (steps + kTileCost); }
};

// The sum of x over the lanes.
__device__ __forceinline__ long long warp_sum(long long x) {
  #pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// This CTA's parts, in the line's order. Held by one warp; lane i looks after the
// i-th of 32 sequences.
struct TreeWalk {
  TreeLane mine;
  TreeShares shares;
  bool planned = false;
  int cta, first;                 // its number; the first of the 32 sequences
  long long at, end;              // places that are left
  long long base;                 // where the 32 sequences begin
  int before_me, here;            // cost of earlier lanes' sequences; of all 32

  __device__ __forceinline__ void fetch(const TreeParams& prm, int lane) {
    mine.load(prm, lane, blockIdx.x == 0);
  }

  __device__ __forceinline__ void take(int lane) {
    int incl = mine.cost();       // 32 x 2 x (2^14 + 3) at most
    const int own = incl;
    #pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    here = __shfl_sync(0xffffffffu, incl, 31);
    before_me = incl - own;
  }

  __device__ __forceinline__ void plan(const TreeParams& prm, int lane) {
    planned = true;
    cta = blockIdx.x / kHkv;
    first = 0;
    base = 0;
    take(lane);
    long long total = here;
    if (prm.batch > 32) {
      long long rest = 0;
      for (int b = 32; b < prm.batch; b += 32) {
        TreeLane other;
        other.load(prm, b + lane, blockIdx.x == 0);
        rest += other.cost();
      }
      total += warp_sum(rest);
    }
    at = end = 0;
    if (total == 0) return;
    shares.set(total, prm.wave);
    if (cta >= shares.ctas) return;
    at = shares.begin(cta);
    end = shares.begin(cta + 1);
  }

  // The next part, false when there is none. Called by a whole warp.
  __device__ __forceinline__ bool next(unsigned long long, const TreeParams& prm, int lane,
                                       TreeWork& work) {
    if (!planned) plan(prm, lane);
    while (at < end) {
      if (at >= base + here) {
        base += here;
        first += 32;
        mine.load(prm, first + lane, false);
        take(lane);
        continue;
      }
      const int place = static_cast<int>(at - base);
      const int from = __ffs(__ballot_sync(0xffffffffu, place >= before_me &&
                                                            place < before_me + mine.cost())) - 1;
      const int steps = __shfl_sync(0xffffffffu, mine.steps, from);
      const int in = place - __shfl_sync(0xffffffffu, before_me, from);
      const int tile = in >= steps + kTileCost ? 1 : 0;
      const long long tile_at = at - (in - tile * (steps + kTileCost));   // the tile's place
      const int begin = max(static_cast<int>(at - tile_at) - kTileCost, 0);
      const int stop = static_cast<int>(min(max(end - tile_at - kTileCost, 0ll),
                                            static_cast<long long>(steps)));
      at = tile_at + steps + kTileCost;
      if (stop <= begin) continue;
      work.b = first + from;
      work.g = blockIdx.x % kHkv;
      work.start = __shfl_sync(0xffffffffu, mine.start, from);
      work.nodes = __shfl_sync(0xffffffffu, mine.nodes, from);
      const int row0 = __shfl_sync(0xffffffffu, mine.row0, from);
      work.first_node = tile * kTileTokens;
      work.row = row0 + work.first_node;
      work.count = min(kTileTokens, work.nodes - work.first_node);
      work.step = begin;
      work.steps = stop - begin;
      work.slot = begin == 0 && stop == steps
                      ? -1
                      : (2 * cta + (begin == 0 ? 1 : 0)) * kHkv + work.g;
      // the rows' positions, where the window hides committed tokens
      work.lo = 0;
      work.top = work.start + work.nodes - 1;
      if (work.top >= prm.window) {
        int least = kMaxTree, most = 0;
        for (int i = lane; i < work.nodes; i += 32) {
          const int n = __popcll(prm.tree[row0 + i] & low_nodes(work.nodes));
          least = min(least, n);
          most = max(most, n);
        }
        least = __reduce_min_sync(0xffffffffu, least);
        most = __reduce_max_sync(0xffffffffu, most);
        work.lo = min(max(work.start + least - prm.window, 0), work.start);
        work.top = work.start + most - 1;
      }
      return true;
    }
    return false;
  }

  static __device__ __forceinline__ unsigned long long low_nodes(int n) {
    return n >= 64 ? ~0ull : (1ull << n) - 1ull;
  }
};

struct TreeJob {
  using Params = TreeParams;
  using Work = TreeWork;
  using View = TreeView;
  using Walk = TreeWalk;
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
  struct Row {
    unsigned long long mask;
    int pos, window;
    __device__ Row(const Work& work, const Params& prm, int tok) {
      mask = __ldg(prm.tree + work.row + tok) & TreeWalk::low_nodes(work.nodes);
      pos = work.start + __popcll(mask) - 1;
      window = prm.window;
    }
    // the keys of the page at `base` that the row sees (16 bits)
    __device__ __forceinline__ uint32_t seen(const View& view, int base) const {
      const int at = base - view.start;                // the page's first drafted token, or before
      const uint32_t drafted =
          at >= 64 || at <= -kPage
              ? 0u
              : static_cast<uint32_t>(at >= 0 ? mask >> at : mask << -at);
      return ((low_bits32(view.sinks - base) | ~low_bits32(pos - window + 1 - base)) &
              low_bits32(-at)) | drafted;
    }
  };
};

// ---------------------------------------------------------------- parts joined
// 8 drafted tokens of a tile and KV head (32 rows) per block, 8 threads a row, two
// float4 each: sum_s 2^(m_s - M) o_s over the parts, divided by the same of l_s.
constexpr int kJoinThreads = 256;
constexpr int kJoinAhead = 8;       // parts whose sums are loaded at once

__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const TreeParams prm) {
  const int b = blockIdx.z, tile = blockIdx.y;
  const int g = blockIdx.x % kHkv, quarter = blockIdx.x / kHkv;
  // this launch must not complete before the one ahead of it, even if nothing is
  // to be joined: the launch after it waits for this one alone
  if (b == 0 && tile == 0 && blockIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
  // where the tile lies on the line, from the lists alone
  const int lane = threadIdx.x & 31;
  long long all = 0, before = 0;
  for (int s = 0; s < prm.batch; s += 32) {
    TreeLane other;
    other.load(prm, s + lane, false);
    all += other.cost();
    before += s + lane < b ? other.cost() : 0;
  }
  all = warp_sum(all);
  before = warp_sum(before);
  TreeLane seq;
  seq.load(prm, b, false);
  const int first_token = tile * kTileTokens + quarter * 8;
  if (first_token >= seq.nodes) return;
  TreeShares shares;
  shares.set(all, prm.wave);
  const long long from = before + tile * (seq.steps + kTileCost) + kTileCost;
  const int cta = shares.owner(from);
  const int parts = shares.owner(from + seq.steps - 1) - cta + 1;
  if (parts <= 1) return;
  const int r = threadIdx.x >> 3, lane8 = threadIdx.x & 7;
  const int token = first_token + (r >> 2);
  if (token >= seq.nodes) return;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int row = quarter * 32 + r;
  // part 0 in slot 2 cta + 1, part s in slot 2 (cta + s)
  auto slot = [&](int s) {
    return static_cast<size_t>((2 * (cta + s) + (s == 0 ? 1 : 0)) * kHkv + g) * kRows + row;
  };
  const float4* o = reinterpret_cast<const float4*>(prm.part_o) + lane8;
  float m = -INFINITY, l = 0.f;
  float4 sum[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int s = 0; s < parts; s += kJoinAhead) {
    float2 x[kJoinAhead];
    float4 v[kJoinAhead][2];
    #pragma unroll
    for (int e = 0; e < kJoinAhead; ++e) {
      const bool is = s + e < parts;
      const size_t at = is ? slot(s + e) : 0;
      x[e] = is ? __ldcg(prm.part_ml + at) : make_float2(-INFINITY, 0.f);
      #pragma unroll
      for (int h = 0; h < 2; ++h)
        v[e][h] = is ? __ldcg(o + at * (kDim / 4) + 8 * h)
                     : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float m_new = m;
    #pragma unroll
    for (int e = 0; e < kJoinAhead; ++e) m_new = fmaxf(m_new, x[e].x);
    if (m_new == -INFINITY) continue;
    const float a = fast_exp2(m - m_new);            // 0 while nothing was joined
    l *= a;
    #pragma unroll
    for (int h = 0; h < 2; ++h)
      sum[h] = make_float4(sum[h].x * a, sum[h].y * a, sum[h].z * a, sum[h].w * a);
    #pragma unroll
    for (int e = 0; e < kJoinAhead; ++e) {
      const float w = fast_exp2(x[e].x - m_new);     // 0 for an absent part
      l += w * x[e].y;
      #pragma unroll
      for (int h = 0; h < 2; ++h) {
        sum[h].x += w * v[e][h].x;
        sum[h].y += w * v[e][h].y;
        sum[h].z += w * v[e][h].z;
        sum[h].w += w * v[e][h].w;
      }
    }
    m = m_new;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  float4* to = reinterpret_cast<float4*>(
                   prm.out + ((static_cast<size_t>(seq.row0) + token) * kHq + g * kGroup +
                              (r & 3)) * kDim) + lane8;
  #pragma unroll
  for (int h = 0; h < 2; ++h)
    to[8 * h] = make_float4(sum[h].x * inv, sum[h].y * inv, sum[h].z * inv, sum[h].w * inv);
}

// ---------------------------------------------------------------- commit
// A block per (sequence, layer, some KV heads: as many as its threads can hold the
// rows of). A thread's 16-byte vectors are (token, head, pool, chunk), all read
// before any is written.
constexpr int kCommitThreads = 256;
constexpr int kHeadVecs = 2 * kRowBytes / 16;                    // K and V of a token: 16
constexpr int kCommitItems = kMaxTree * kHeadVecs / kCommitThreads;   // 4

__global__ void __launch_bounds__(kCommitThreads, 6) tree_commit_kernel(
    uint4* k_pool, uint4* v_pool, const int32_t* __restrict__ tables,
    const int32_t* __restrict__ start_pos, const int32_t* __restrict__ accepted,
    const int32_t* __restrict__ counts, int max_accepted, int max_batch, int table_stride,
    int num_pages, int max_seq_len, int heads, int* err) {
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
  const cuuint64_t dims[3] = {kDim, kHq, static_cast<cuuint64_t>(total_tokens)};
  const cuuint64_t strides[2] = {kRowBytes, static_cast<cuuint64_t>(kHq) * kRowBytes};
  const cuuint32_t box[3] = {kDim, kGroup, kTileTokens};
  if (!encode_bf16(&tq, q, 3, dims, strides, box) ||
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
  prm.next_tile = pool->prefill_next;
  prm.ctas_done = reinterpret_cast<unsigned int*>(pool->prefill_next + 1);
  prm.num_pages = c.num_pages;
  prm.table_stride = stride;
  prm.max_seq_len = c.max_seq_len;
  prm.batch = batch;
  prm.total_tokens = total_tokens;
  prm.window = std::min(window, c.max_seq_len);
  prm.sinks = std::min(sinks, c.max_seq_len);
  prm.tree = reinterpret_cast<const unsigned long long*>(tree);
  prm.part_o = pool->tree_part_o;
  prm.part_ml = pool->tree_part_ml;
  prm.wave = std::max(wave / kHkv, 1);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  tile_attention_kernel<TreeJob><<<wave, kThreads, kSmemBytes<TreeJob>, st>>>(tq, tk, tv, prm);
  if (cudaGetLastError() != cudaSuccess) return PKV_ERR_CUDA;
  // the join's blocks start as the attention's CTAs end, and wait for the last
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(kHkv * (kTileTokens / 8), total_tokens > kTileTokens ? 2 : 1, batch);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, tree_join_kernel, prm) != cudaSuccess) return PKV_ERR_CUDA;
  return pkv_check_launch();
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
  pool->pages_written = true;
  tree_commit_kernel<<<dim3(kHkv / heads, batch, c.num_layers), kCommitThreads, 0,
                       static_cast<cudaStream_t>(stream)>>>(
      static_cast<uint4*>(k_pool), static_cast<uint4*>(v_pool), block_tables, start_pos, accepted,
      counts, max_accepted, c.max_batch, c.max_seq_len / kPage, c.num_pages, c.max_seq_len,
      heads, pool->err);
  return pkv_check_launch();
}

}  // extern "C"
