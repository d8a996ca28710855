// Internal to libpkv: drafted token trees (include/pkv_tree.h), shared by the
// kernels for larger trees (tree.cu) and for few rows (tree_few.cu): what a tree
// sees, how a launch's work is shared out, and how parts are joined.
#ifndef PKV_TREE_CUH
#define PKV_TREE_CUH

#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "pkv.h"
#include "pkv_tree.h"
#include "device_common.cuh"
#include "pool_internal.h"
#include "prefill_tiles.cuh"

namespace pkv_tree_dev {

using namespace pkv_tiles;

constexpr int kMaxTree = PKV_MAX_TREE;
// A tile's start and end cost a CTA about as much as two steps; a CTA is given no
// less than kLeastCost.
constexpr int kTileCost = 2;
constexpr int kLeastCost = 2;
static_assert(kMaxTree % kTileTokens == 0, "whole tiles");

struct TreeParams : TileParams {
  const unsigned long long* tree;   // [total] which drafted tokens each row sees
  float* part_o;                    // [2 wave][8][rows][64] sums of parts, not divided
  float2* part_ml;                  // [2 wave][8][rows] their exponent and sum of weights
  int wave;                         // CTAs of one wave, per KV head
  unsigned long long per_wave;      // 2^64 / wave, rounded up
};

// The lowest n bits (n from 0 to 64).
__device__ __forceinline__ unsigned long long low_nodes(int n) {
  return n >= 64 ? ~0ull : (1ull << n) - 1ull;
}

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
  int whole_from, whole_to;       // pages whose tokens every row sees
  int plain_from, plain_to;       // steps of the part made of those

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
    whole_from = hidden < sinks ? 0 : sink_pages + hidden / kPage + 1 - win_page;
    whole_to = sink_pages + start / kPage - win_page;
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
// sequence, a tile kTileCost before its steps) make a line of `total` places (a short
// one counts as kLeastCost for every CTA); of the wave's CTAs per KV head number c
// takes [total c / wave, total (c + 1) / wave), so all take equally long whatever the
// lengths are, and a tile may be cut anywhere.
// (Parts of one length per launch left a fifth of the device idle: 8 trees of 64
// over 20,000 to 32,700 tokens took 254 us, shared out 205.)
//
// A CTA has at most one part of a tile that began before it, kept in slot 2 c, and
// one of a tile that goes on behind it, in slot 2 c + 1.
struct TreeShares {
  long long total;
  __device__ void set(long long all, const TreeParams& prm) {
    total = max(all, static_cast<long long>(prm.wave) * kLeastCost);
  }
  // total c / wave, rounded down: by the reciprocal, exact while total c < 2^64 /
  // wave (a division here is on the way to a CTA's first copy)
  __device__ long long begin(int c, const TreeParams& prm) const {
    return static_cast<long long>(__umul64hi(static_cast<unsigned long long>(total * c),
                                             prm.per_wave));
  }
  // the last CTA that begins at or before `place`
  __device__ int owner(long long place, const TreeParams& prm) const {
    return static_cast<int>(((place + 1) * prm.wave - 1) / total);
  }
};

// The sequences of 32 lanes: what each brings, with tiles of kTile tokens.
template <int kTile>
struct TreeLane {
  int row0, nodes, start, steps;

  // Sequence b: steps 0 if there is none or its data is bad.
  __device__ __forceinline__ void load(const TreeParams& prm, int b, bool report) {
    set(prm, lists(prm, b), report);
  }
  // The same in two parts, to have several sequences' lists on their way: its first
  // row, the row after its last, and its committed tokens.
  static __device__ __forceinline__ int3 lists(const TreeParams& prm, int b) {
    return b < prm.batch ? make_int3(prm.cu_tokens[b], prm.cu_tokens[b + 1], prm.start_pos[b])
                         : make_int3(0, 0, 0);
  }
  __device__ __forceinline__ void set(const TreeParams& prm, int3 lists, bool report) {
    steps = nodes = 0;
    row0 = lists.x;
    start = lists.z;
    const int rows = lists.y - row0;
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
  __device__ __forceinline__ int tiles() const { return (nodes + kTile - 1) / kTile; }
  __device__ __forceinline__ int cost() const { return tiles() * (steps + kTileCost); }
};

// The sum of x over the lanes.
__device__ __forceinline__ long long warp_sum(long long x) {
  #pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The positions of a sequence's rows, where the window hides committed tokens.
__device__ __forceinline__ void span_of_rows(const TreeParams& prm, int row0, int lane,
                                             TreeWork& work) {
  work.lo = 0;
  work.top = work.start + work.nodes - 1;
  if (work.top < prm.window) return;
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

// This CTA's parts, in the line's order. Held by one warp; lane i looks after the
// i-th of 32 sequences.
template <int kTile>
struct TreeWalk {
  TreeLane<kTile> mine;
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
    int incl = mine.cost();       // 32 x 16 x (2^14 + 3) at most
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
    int group = lane == 0 ? here : 0;     // cost of the lane-th 32 sequences (of the first 1,024)
    if (prm.batch > 32) {
      constexpr int kAhead = 4;
      long long rest = 0;
      for (int g = 1; g * 32 < prm.batch; g += kAhead) {
        int3 lists[kAhead];
        #pragma unroll
        for (int e = 0; e < kAhead; ++e)
          lists[e] = TreeLane<kTile>::lists(prm, (g + e) * 32 + lane);
        #pragma unroll
        for (int e = 0; e < kAhead; ++e) {
          TreeLane<kTile> other;
          other.set(prm, lists[e], blockIdx.x == 0);
          const int cost = __reduce_add_sync(0xffffffffu, other.cost());
          if (lane == g + e) group = cost;
          rest += cost;
        }
      }
      total += rest;
    }
    at = end = 0;
    shares.set(total, prm);
    if (cta >= prm.wave) return;
    at = shares.begin(cta, prm);
    end = min(shares.begin(cta + 1, prm), total);
    if (prm.batch > 32) {
      // on to the 32 sequences that hold the first place (or to the last of the 1,024)
      int incl = group;                   // 1,024 x 16 x (2^14 + 3) at most
      #pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      const uint32_t behind = __ballot_sync(0xffffffffu, at < incl);
      const int g = behind ? __ffs(behind) - 1 : 31;
      if (g > 0) {
        first = 32 * g;
        base = __shfl_sync(0xffffffffu, incl - group, g);
        mine.load(prm, first + lane, false);
        take(lane);
      }
    }
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
      // in / (steps + kTileCost), below 16: (in + 1/2) / d is 1 / (2 d) > 2^-16 away from
      // an integer, the error below 2^-18
      const int tile = static_cast<int>(__fdividef(static_cast<float>(in) + 0.5f,
                                                   static_cast<float>(steps + kTileCost)));
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
      work.first_node = tile * kTile;
      work.row = row0 + work.first_node;
      work.count = min(kTile, work.nodes - work.first_node);
      work.step = begin;
      work.steps = stop - begin;
      work.slot = begin == 0 && stop == steps
                      ? -1
                      : (2 * cta + (begin == 0 ? 1 : 0)) * kHkv + work.g;
      span_of_rows(prm, row0, lane, work);
      return true;
    }
    return false;
  }
};

// Part `rank` of `parts` of the launch's tile number `tile`, of up to 32 sequences;
// false if there are fewer tiles. A part may have no steps. Called by a whole warp.
template <int kTile>
__device__ __forceinline__ bool part_of_tile(const TreeParams& prm, const TreeLane<kTile>& mine,
                                             int tile, int rank, int parts, int lane,
                                             TreeWork& work) {
  int incl = mine.tiles();
  #pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  const uint32_t holds = __ballot_sync(0xffffffffu, tile < incl);
  if (holds == 0) return false;
  const int from = __ffs(holds) - 1;
  const int in = tile - __shfl_sync(0xffffffffu, incl - mine.tiles(), from);
  const int steps = __shfl_sync(0xffffffffu, mine.steps, from);
  const int row0 = __shfl_sync(0xffffffffu, mine.row0, from);
  work.b = from;
  work.start = __shfl_sync(0xffffffffu, mine.start, from);
  work.nodes = __shfl_sync(0xffffffffu, mine.nodes, from);
  work.first_node = in * kTile;
  work.row = row0 + work.first_node;
  work.count = min(kTile, work.nodes - work.first_node);
  work.step = steps * rank / parts;
  work.steps = steps * (rank + 1) / parts - work.step;
  work.slot = -1;
  span_of_rows(prm, row0, lane, work);
  return true;
}

// What one row sees.
struct TreeRow {
  unsigned long long mask;
  int pos, window;
  // the tile's token `tok`; or one whose entry of the tree is known
  __device__ TreeRow(const TreeWork& work, const TreeParams& prm, int tok)
      : TreeRow(work, prm, __ldg(prm.tree + work.row + tok)) {}
  __device__ TreeRow(const TreeWork& work, const TreeParams& prm, unsigned long long entry) {
    mask = entry & low_nodes(work.nodes);
    pos = work.start + __popcll(mask) - 1;
    window = prm.window;
  }
  // the keys of the page at `base` that the row sees (16 bits)
  __device__ __forceinline__ uint32_t seen(const TreeView& view, int base) const {
    const int at = base - view.start;                // the page's first drafted token, or before
    const uint32_t drafted =
        at >= 64 || at <= -kPage
            ? 0u
            : static_cast<uint32_t>(at >= 0 ? mask >> at : mask << -at);
    return ((low_bits32(view.sinks - base) | ~low_bits32(pos - window + 1 - base)) &
            low_bits32(-at)) | drafted;
  }
};

// ---------------------------------------------------------------- parts joined
// There are fewer cut tiles than CTAs: a block per CTA c and KV head looks where c
// begins and, if that is the first cut in its tile, joins the tile's rows, 8 threads a
// row, two float4 each: sum_s 2^(m_s - M) o_s over the parts, divided by the same of
// l_s. (With a block per sequence and tile, most of them without work, 4,096 trees
// of 2 took 1,018 us instead of 392, 128 of 4 over 2,000 tokens 102 instead of 93.)
constexpr int kJoinThreads = 256;
constexpr int kJoinAhead = 8;       // parts whose sums are loaded at once

template <int kTile>
__global__ void __launch_bounds__(kJoinThreads) tree_join_kernel(const TreeParams prm,
                                                                 int split) {
  constexpr int kWarps = kJoinThreads / 32;
  const int g = blockIdx.x % kHkv, c = blockIdx.x / (kHkv * split);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // this launch must not complete before the one ahead of it, even if nothing is
  // to be joined: the launch after it waits for this one alone
  if (c == 0) {
    if (blockIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  // the line's length, a thread's sequences being threadIdx.x, + 256, ...
  __shared__ long long sums[kWarps];
  __shared__ int scan[2][kWarps];
  __shared__ int4 found;              // row0, nodes, steps, place in the sequence
  TreeLane<kTile> seq;
  seq.load(prm, threadIdx.x, false);
  long long total = seq.cost();
  for (int s = threadIdx.x + kJoinThreads; s < prm.batch; s += kJoinThreads) {
    TreeLane<kTile> other;
    other.load(prm, s, false);
    total += other.cost();
  }
  total = warp_sum(total);
  if (lane == 0) sums[warp] = total;
  __syncthreads();
  total = 0;
  #pragma unroll
  for (int w = 0; w < kWarps; ++w) total += sums[w];
  TreeShares shares;
  shares.set(total, prm);
  const long long place = shares.begin(c, prm);
  if (place >= total) return;
  // the sequence that holds the place
  long long base = 0;
  for (int s0 = 0, turn = 0;; s0 += kJoinThreads, turn ^= 1) {
    if (s0 > 0) seq.load(prm, s0 + threadIdx.x, false);
    const int own = seq.cost();
    int incl = own;                   // 256 x 16 x (2^14 + 3) at most
    #pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    if (lane == 31) scan[turn][warp] = incl;
    __syncthreads();
    int group = 0;
    #pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) incl += scan[turn][w];
      group += scan[turn][w];
    }
    if (place < base + group) {       // the same decision in every thread
      const int in = static_cast<int>(place - base);
      if (in >= incl - own && in < incl)
        found = make_int4(seq.row0, seq.nodes, seq.steps, in - (incl - own));
      __syncthreads();
      break;
    }
    base += group;
  }
  const int row0 = found.x, nodes = found.y, steps = found.z;
  const int tile = found.w / (steps + kTileCost);
  const long long from = place - found.w + tile * (steps + kTileCost) + kTileCost;   // its steps
  // inside the tile's steps, and CTA c - 1 began at or before them
  if (place - from < 1 || place - from >= steps || shares.begin(c - 1, prm) - from >= 1) return;
  const int cta = c - 1;
  const int parts = shares.owner(from + steps - 1, prm) - cta + 1;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane8 = threadIdx.x & 7;
  const int rows = min(kTile, nodes - tile * kTile) * kGroup;
  for (int row = blockIdx.x / kHkv % split * (kJoinThreads / 8) + (threadIdx.x >> 3); row < rows;
       row += split * (kJoinThreads / 8)) {
    // part 0 in slot 2 cta + 1, part s in slot 2 (cta + s)
    auto slot = [&](int s) {
      const size_t at = (2 * (cta + s) + (s == 0 ? 1 : 0)) * kHkv + g;
      return at * (kTile * kGroup) + row;
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
                     prm.out + ((static_cast<size_t>(row0) + tile * kTile + (row >> 2)) * kHq +
                                g * kGroup + (row & 3)) * kDim) + lane8;
    #pragma unroll
    for (int h = 0; h < 2; ++h)
      to[8 * h] = make_float4(sum[h].x * inv, sum[h].y * inv, sum[h].z * inv, sum[h].w * inv);
  }
}

// ---------------------------------------------------------------- host
template <int kTile>
pkv_status launch_join(const TreeParams& prm, cudaStream_t st) {
  // the join's blocks start as the attention's CTAs end, and wait for the last
  cudaLaunchConfig_t cfg = {};
  // blocks that share a cut tile's rows: more where there are few tiles (one sequence
  // of 64, us: 4 blocks 15.6, 2 16.8, 1 21.3; 32 of up to 16: 21.4, 20.8, 21.1)
  const int split = kTile <= 8 ? 1 : prm.batch <= 2 ? 4 : 2;
  cfg.gridDim = dim3(prm.wave * kHkv * split);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, tree_join_kernel<kTile>, prm, split) != cudaSuccess)
    return PKV_ERR_CUDA;
  return pkv_check_launch();
}

// The wave of CTAs that shares a launch's work.
inline void set_wave(TreeParams* prm, int ctas) {
  prm->wave = std::max(ctas / kHkv, 2);
  prm->per_wave = ~0ull / static_cast<unsigned>(prm->wave) + 1;
}

}  // namespace pkv_tree_dev

// tree_few.cu: the attention of few rows per sequence (prm as tree.cu fills it), by
// clusters of so many blocks (0: none), as pkv_tree_cluster finds for a call whose
// sequences see up to seen_tokens.
int pkv_tree_cluster(const pkv_pool* pool, int batch, int total_tokens, int seen_tokens);
pkv_status pkv_tree_few(pkv_pool_t pool, const void* q, const CUtensorMap& tk,
                        const CUtensorMap& tv, pkv_tree_dev::TreeParams prm, int parts,
                        cudaStream_t st);

#endif  // PKV_TREE_CUH
