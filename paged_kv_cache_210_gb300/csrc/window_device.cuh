// Internal to libpkv: the windowed decode kernel, shared by the BF16 cache
// (window.cu) and the 8-bit cache (quant.cu). What differs between them is in
// their Tiles: how a page is copied, how a new row is written, a page's
// products, and the state that they leave.
//
// out = sum_t p_t V_t / sum_t p_t, p_t = 2^(q.K_t log2(e) / 8 - m), over the
// visible tokens: one pass with a running maximum m and sum.
//
// A sequence's visible pages are the sink pages [0, sp) and the window's
// pages [wf, n_pages); "page i" below counts through both. One block of 4
// warps per (sequence, kv head, split) serves the 4 query heads, so a page
// tile is read once; warp w takes pages w, w + 4, ... of its block's range
// through its own ring of stages, filled by the copy engine. Splits
// merge inside the launch: through a thread-block cluster's shared memory,
// or through global partials and a ticket.
#ifndef PKV_WINDOW_DEVICE_CUH
#define PKV_WINDOW_DEVICE_CUH

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "pkv.h"
#include "pkv_axes.h"
#include "axes.cuh"
#include "decode_device.cuh"
#include "device_common.cuh"
#include "pool_internal.h"

namespace pkv_window {

using namespace pkv_dev;
using namespace pkv_decode;
using namespace pkv_axes_dev;

constexpr int kWarps = 4;
constexpr int kThreadsW = kWarps * 32;
constexpr int kTries = 8;             // range sizes tried for a one-wave launch
constexpr int kHeld = 3;              // sequences per thread whose page count is kept

// Shared memory of the unit search.
struct UnitSearch {
  float pages[kWarps];
  int most[kWarps];
  int full[kWarps];
  uint32_t c12[kWarps], c34[kWarps];
  int count[2][kWarps];
  int seq, split, len;
  int4 unit;
};

template <class Tiles>
struct WindowSmem {
  typename Tiles::Ring warp[kWarps];
  unsigned long long bar[kWarps][Tiles::kStages];
  float m[kWarps][kGroup];
  float l[kWarps][kGroup];
  float acc[kWarps][kGroup][kDim];   // the warps' partial outputs (block merge)
  UnitSearch find;
  int last;
};

// + 1 KiB: the dynamic shared memory base is rounded up to 1024 bytes
template <class Tiles>
constexpr size_t kTicketSmemBytes = sizeof(WindowSmem<Tiles>) + 1024;
template <class Tiles>
constexpr size_t kClusterSmemBytes = sizeof(WindowSmem<Tiles>) + sizeof(AsyncInbox) + 1024;

struct WindowParams {
  const uint16_t* q;          // [B][32][64]
  const uint16_t* k_new;      // [B][8][64]   (fused only)
  const uint16_t* v_new;
  const int32_t* table;       // this layer's block tables: [max_batch][table_stride]
  const int32_t* seq_lens;    // [B]
  float* out;                 // [B][32][64]
  float* part_o;              // [max_batch][32][max_splits][64] (this layer's parity)
  float2* part_ml;            // [max_batch][32][max_splits]
  int* tickets;               // [max_batch][8]
  int* err;
  int num_pages;
  int table_stride;
  int max_seq_len;
  int max_splits;
  int num_splits;             // > 0: ranges per sequence (and gridDim.x); 0: units (below)
  int batch;
  int wave_units;             // units: > 0: batch <= 32 kHeld, try to keep to this many
  int range_div;              // units: ranges of about (the batch's pages) / range_div pages
  int least_pages;            // ranges have at least this many pages
  int window;                 // 1 .. max_seq_len
  int sinks;                  // 0 .. max_seq_len
  AxesArgs rope;
};

// The lowest n bits (n clamped to 0 .. 16).
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : n >= kPage ? 0xffffu : (1u << n) - 1u;
}

// The visible pages of a sequence: the sink pages [0, sinks) and the window's
// [window, window + count - sinks), `count` in all.
struct SeenPages {
  int sinks, window, count, first_token;
  __device__ SeenPages(int len, const WindowParams& prm) {
    first_token = max(len - prm.window, 0);
    window = first_token / kPage;
    sinks = min((prm.sinks + kPage - 1) / kPage, window);
    count = sinks + (len + kPage - 1) / kPage - window;
  }
};

// ---------------------------------------------------------------- units
// Larger batches launch a grid of (sequence, range) units instead of a fixed
// number of splits per sequence, whose blocks would be idle for short
// sequences and uneven for long ones. The range size comes from the lengths
// the launch finds; a sequence of p visible pages has ceil(p / range) units,
// the last of which may be short. With T the batch's visible pages:
//  * a batch that may fit one wave of resident blocks (wave_units > 0) takes
//    the smallest range of r0 (8 + k) / 8, r0 = T / wave_units, k < 8, whose
//    units fit it: a second wave of full ranges costs more than longer ranges
//    (32 full 1,024-token windows: 17.1 us in one wave, 20.6 in two);
//  * others take T / range_div, range_div 3/5 of a wave, but at least
//    least_pages (128 ragged sequences behind 1,024 tokens: 22.0 us; with 4/5
//    25.8, with 17/10 28.5).
// So there are fewer than batch + range_div units, or at most wave_units.
// They are handed out largest first (all full ranges, then the short ones by
// quarters of a range), so what does not fit the first wave is short (256
// ragged sequences behind 4,096 tokens: 106.5 us, in batch order 124.2). Each
// block finds its own unit: sums over the batch, the class of size the unit
// falls into, and a prefix sum within it. Padding rows have no units; a
// length out of range has one, which reports it.
//
// kBlock: the block's threads share the batch, kHeld sequences each kept in
// registers, the rest read again, and all of them call; otherwise (batch <=
// 32 kHeld) one warp calls, and does it all without a barrier. False past the
// last unit.
template <bool kBlock>
__device__ __forceinline__ bool find_unit(int u, const WindowParams& prm, UnitSearch& find, int& b,
                                          int& split, int& range, int& len) {
  constexpr int kGroupSize = kBlock ? kThreadsW : 32;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int me = kBlock ? static_cast<int>(threadIdx.x) : lane;
  auto pages_of = [&](int len) {
    return len == 0 ? 0 : len < 0 || len > prm.max_seq_len ? 1 : SeenPages(len, prm).count;
  };
  auto len_of = [&](int s) { return s < prm.batch ? prm.seq_lens[s] : 0; };
  int held_len[kHeld], held[kHeld];
  #pragma unroll
  for (int e = 0; e < kHeld; ++e) held_len[e] = len_of(me + e * kGroupSize);
  #pragma unroll
  for (int e = 0; e < kHeld; ++e)
    held[e] = prm.batch > e * kGroupSize ? pages_of(held_len[e]) : 0;
  auto each = [&](auto fn) {                  // for every sequence of this thread
    fn(held[0]);
    #pragma unroll
    for (int e = 1; e < kHeld; ++e)
      if (prm.batch > e * kGroupSize) fn(held[e]);
    if (kBlock)
      for (int s = me + kHeld * kGroupSize; s < prm.batch; s += kGroupSize) fn(pages_of(len_of(s)));
  };
  // ceil(p / r) by r's reciprocal, exact for p, r < 2^17 (the quotient of p + r -
  // 1/2 stays 1 / (2 r) away from integers, the errors are below 2^-21 of it);
  // adding 2^23 - 1/2 rounds it down into the low bits, without a conversion.
  auto ceil_of = [](int p, float r, float inv) {
    return __float_as_int(fmaf(static_cast<float>(p) + (r - 0.5f), inv, 8388607.5f)) - 0x4b000000;
  };
  float sum = 0.f;                            // pages: exact to 2^24, then to 2^-22 of itself
  int most = 0;
  if (!kBlock) {
    int pages = 0;
    each([&](int p) {
      pages += p;
      most = max(most, p);
    });
    sum = static_cast<float>(static_cast<int>(__reduce_add_sync(0xffffffffu, pages)));
    most = __reduce_max_sync(0xffffffffu, most);
  } else {
    each([&](int p) {
      sum += static_cast<float>(p);
      most = max(most, p);
    });
    #pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    most = __reduce_max_sync(0xffffffffu, most);
    if (lane == 0) {
      find.pages[warp] = sum;
      find.most[warp] = most;
    }
    __syncthreads();
    sum = 0.f;
    #pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      sum += find.pages[w];
      most = max(most, find.most[w]);
    }
  }
  // T / by, rounded up past the float error (ranges stay below 2^17 pages)
  auto share = [&](int by) {
    return static_cast<int>(fminf(__fdividef(sum, static_cast<float>(by)), 131070.f)) + 1;
  };
  range = max(prm.least_pages, share(prm.range_div));
  if (!kBlock) {
    const int r0 = max(prm.least_pages, share(prm.wave_units));
    #pragma unroll
    for (int k = kTries - 1; k >= 0; --k) {
      const int r = min((r0 * (kTries + k) + kTries - 1) / kTries, 131071);
      const float fr = static_cast<float>(r), inv = __fdividef(1.f, fr);
      int units = ceil_of(held[0], fr, inv);
      #pragma unroll
      for (int e = 1; e < kHeld; ++e)
        if (prm.batch > e * 32) units += ceil_of(held[e], fr, inv);
      if (static_cast<int>(__reduce_add_sync(0xffffffffu, units)) <= prm.wave_units) range = r;
    }
  }
  range = min(range, max(most, 1));
  const float f_range = static_cast<float>(range), inv_range = __fdividef(1.f, f_range);
  // a sequence's full ranges and the class of what is left: 1 (longest) .. 4, 0: nothing
  auto classify = [&](int p, int& full) {
    full = ceil_of(p + 1, f_range, inv_range) - 1;
    const int rest = p - full * range;
    return rest > 0 ? 5 - ceil_of(4 * rest, f_range, inv_range) : 0;
  };
  int full = 0;
  uint32_t c12 = 0, c34 = 0;                 // two 16-bit counts each (batch <= 65535)
  each([&](int p) {
    int f;
    const int c = classify(p, f);
    full += f;
    c12 += c == 1 ? 1u : c == 2 ? 0x10000u : 0u;
    c34 += c == 3 ? 1u : c == 4 ? 0x10000u : 0u;
  });
  full = __reduce_add_sync(0xffffffffu, full);
  c12 = __reduce_add_sync(0xffffffffu, c12);
  c34 = __reduce_add_sync(0xffffffffu, c34);
  if (kBlock) {
    if (lane == 0) {
      find.full[warp] = full;
      find.c12[warp] = c12;
      find.c34[warp] = c34;
    }
    __syncthreads();
    full = 0;
    c12 = c34 = 0;
    #pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      full += find.full[w];
      c12 += find.c12[w];
      c34 += find.c34[w];
    }
  }
  const int sizes[5] = {full, static_cast<int>(c12 & 0xffffu), static_cast<int>(c12 >> 16),
                        static_cast<int>(c34 & 0xffffu), static_cast<int>(c34 >> 16)};
  int cls = -1;
  #pragma unroll
  for (int c = 0; c < 5; ++c) {
    if (cls < 0) {
      if (u < sizes[c]) {
        cls = c;
      } else {
        u -= sizes[c];
      }
    }
  }
  if (cls < 0) return false;                 // the same decision in every thread
  int before = 0;
  for (int base = 0, turn = 0; base < prm.batch; base += kGroupSize, turn ^= 1) {
    const int e = base / kGroupSize;
    int pages = held[0], own_len = held_len[0];
    #pragma unroll
    for (int h = 1; h < kHeld; ++h) {
      pages = e == h ? held[h] : pages;
      own_len = e == h ? held_len[h] : own_len;
    }
    if (kBlock && e >= kHeld) {
      own_len = len_of(base + me);
      pages = pages_of(own_len);
    }
    int f;
    const int c = classify(pages, f);
    const int units = cls == 0 ? f : c == cls ? 1 : 0;
    int excl, total;                         // over the warp
    if (cls == 0) {
      int incl = units;
      #pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      total = __shfl_sync(0xffffffffu, incl, 31);
      excl = before + incl - units;
    } else {
      const uint32_t some = __ballot_sync(0xffffffffu, units != 0);
      total = __popc(some);
      excl = before + __popc(some & ((1u << lane) - 1u));
    }
    if (kBlock) {
      if (lane == 0) find.count[turn][warp] = total;
      __syncthreads();
      total = 0;
      #pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const int cw = find.count[turn][w];
        excl += w < warp ? cw : 0;
        total += cw;
      }
    }
    if (u < before + total) {                // the same decision in every thread
      const bool mine = u >= excl && u < excl + units;
      const int at = cls == 0 ? u - excl : f;
      if (kBlock) {
        if (mine) {
          find.seq = base + me;
          find.split = at;
          find.len = own_len;
        }
        __syncthreads();
        b = find.seq;
        split = find.split;
        len = find.len;
      } else {
        const int from = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
        b = base + from;
        split = __shfl_sync(0xffffffffu, at, from);
        len = __shfl_sync(0xffffffffu, own_len, from);
      }
      return true;
    }
    before += total;
  }
  return false;
}

// ---------------------------------------------------------------- decode
// kCluster: the splits of one (sequence, kv head) form one thread-block
// cluster (gridDim.x == cluster size); otherwise global partials and a ticket.
template <bool kFused, bool kCluster, bool kRope, class Tiles>
__global__ void __launch_bounds__(kThreadsW, kCluster ? 3 : 4)
window_decode_kernel(const __grid_constant__ typename Tiles::Source src,
                     const WindowParams prm) {
  constexpr int kStages = Tiles::kStages;
  constexpr int kPer = Tiles::kStagePages;      // pages of a stage: a group
  constexpr int kParts = Tiles::kParts;         // copies of a page
  static_assert(kPer == 1 || kParts == 1, "a group's valid pages are read off one vote");
  static_assert(kStages * kPer * kParts <= 32, "one lane per copy of the prefetch");
  using Smem = WindowSmem<Tiles>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem_base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Smem& sm = *reinterpret_cast<Smem*>(smem_base);
  AsyncInbox& inbox = *reinterpret_cast<AsyncInbox*>(smem_base + sizeof(Smem));

  const bool units = !kCluster && prm.num_splits == 0;   // grid (units x kv heads)
  int split = blockIdx.x;
  const int kvh = units ? blockIdx.x % kHkv : blockIdx.y;
  int b = blockIdx.z;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  typename Tiles::Ring& ws = sm.warp[warp];
  unsigned long long* bars = sm.bar[warp];
  if (lane == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&bars[s], 1);
    fence_mbar_init();
    if (warp == 1) Tiles::prefetch(src);   // warp 0 goes on to the unit search
  }
  // Before the wait (programmatic dependent launch) this block reads only
  // seq_lens, the block table, the rotary inputs and pool rows below the
  // appended position.
  // A block without work leaves at once, but the first one waits all the same:
  // a launch must not complete before the one ahead of it does, even if none
  // of its rows has work (the launch after it waits for this one alone).
  auto leave = [&]() {
    if (blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) pdl_wait();
  };
  int range = 0;
  int len;
  if (units) {
    const int u = static_cast<int>(blockIdx.x) / kHkv;
    bool found;
    if (prm.wave_units > 0) {
      // one warp searches: four doing the same compete for the issue slots
      if (warp == 0) {
        found = find_unit<false>(u, prm, sm.find, b, split, range, len);
        if (lane == 0)
          sm.find.unit = found ? make_int4(b, split, range, len) : make_int4(-1, 0, 0, 0);
      }
      __syncthreads();
      const int4 unit = sm.find.unit;
      found = unit.x >= 0;
      b = unit.x;
      split = unit.y;
      range = unit.z;
      len = unit.w;
    } else {
      found = find_unit<true>(u, prm, sm.find, b, split, range, len);
    }
    if (!found) {
      leave();
      return;
    }
  } else {
    len = prm.seq_lens[b];
  }
  if (len <= 0 || len > prm.max_seq_len) {               // a padding row (0), or a bad length
    if (len != 0 && split == 0 && kvh == 0 && threadIdx.x == 0) set_error(prm.err, kErrSeqLen);
    leave();
    return;
  }
  int rope_pos = 0;
  if (kRope) rope_pos = pair_position(prm.rope, b, lane);   // arrives with the page ids
  const SeenPages see(len, prm);
  const int sink_pages = see.sinks;
  const int win_page = see.window;
  const int win_lo = see.first_token;
  const int n_seen = see.count;                          // >= 1
  const int chunk = prm.num_splits > 0 ? (n_seen + prm.num_splits - 1) / prm.num_splits : range;
  const int n_splits = (n_seen + chunk - 1) / chunk;     // non-empty splits of this sequence
  if (kCluster) {
    if (n_splits == 1 && split > 0) return;   // the same decision in every block of the cluster
  } else {
    if (split >= n_splits) return;
  }
  const bool active = split < n_splits;       // an idle cluster block only joins the merge
  const int page_begin = active ? split * chunk : 0;
  const int page_end = active ? min(n_seen, page_begin + chunk) : 0;
  // This warp's pages: its page l is page page_begin + (kWarps j + warp) kPer + e
  // of the sequence's, l = kPer j + e; groups j < mine, pages l < my_pages.
  const int pages = page_end - page_begin;
  const int rounds = pages / (kWarps * kPer);
  const int my_pages =
      rounds * kPer + min(max(pages - (rounds * kWarps + warp) * kPer, 0), kPer);
  const int mine = (my_pages + kPer - 1) / kPer;
  const int new_slot = (len - 1) % kPage;     // slot of the appended token
  // the sequence's last page, if it is one of this warp's
  const int new_off = n_seen - 1 - page_begin;
  const bool has_new = new_off >= 0 && new_off < pages && new_off / kPer % kWarps == warp;
  const int j_new = has_new ? new_off / (kPer * kWarps) : -1;
  const int l_new = has_new ? j_new * kPer + new_off % kPer : -1;

  const int32_t* row = prm.table + static_cast<size_t>(b) * prm.table_stride;
  auto logical = [&](int l) {
    const int i = page_begin + (l / kPer * kWarps + warp) * kPer + l % kPer;
    return i < sink_pages ? i : i - sink_pages + win_page;
  };
  // Physical ids of 32 of this warp's pages, one per lane; the next 32 are
  // fetched while these are in use.
  auto fetch_ids = [&](int base) {
    const int l = base + lane;
    return l < my_pages ? __ldg(row + logical(l)) : -1;
  };
  int ids = fetch_ids(0);
  int ids_next = my_pages > 32 ? fetch_ids(32) : -1;
  auto good_id = [&](int phys) {
    return static_cast<unsigned>(phys) < static_cast<unsigned>(prm.num_pages);
  };
  float ang_c = 1.f, ang_s = 0.f;                        // the angle of pair `lane`
  if (kRope && !load_pair_angle(prm.rope, rope_pos, lane, ang_c, ang_s)) {
    if (split == 0 && kvh == 0 && threadIdx.x == 0) set_error(prm.err, kErrPosition);
    leave();
    return;                                              // every block of the sequence
  }

  if (kCluster && n_splits > 1) async_inbox_setup(inbox);
  __syncwarp();

  // Copy engine: the pages of group j into `stage`, one copy per lane. A page
  // whose only token is the appended one (fused) is not copied.
  uint32_t stage_bad = 0;                     // bit kPer s + e: page e of stage s is invalid
  bool some_bad = false;                      // some page had an invalid id
  auto issue_copy = [&](int j, int stage) {
    constexpr uint32_t kGroup1 = (1u << kPer) - 1u;
    const int l0 = j * kPer;
    const int there = min(my_pages - l0, kPer);
    if constexpr (kPer == 2) {
      // both pages there and nothing unusual: one lane issues both copies, all lanes
      // compute their addresses (operands of a lane's own take a loop over the lanes)
      const int p0 = __shfl_sync(0xffffffffu, ids, l0 & 31);
      const int p1 = __shfl_sync(0xffffffffu, ids, (l0 + 1) & 31);
      if (there == 2 && good_id(p0) && good_id(p1) && !some_bad &&
          !(kFused && j == j_new && new_slot == 0)) {
        if (elect_one()) {
          mbar_arrive_expect_tx(&bars[stage], 2 * Tiles::kCopyBytes);
          Tiles::copy(ws, stage, 0, src, 0, kvh, p0, &bars[stage]);
          Tiles::copy(ws, stage, 1, src, 0, kvh, p1, &bars[stage]);
        }
        __syncwarp();
        return;
      }
    }
    const int e = kPer == 1 ? 0 : lane;
    const int phys = __shfl_sync(0xffffffffu, ids, (l0 + e) & 31);
    const bool ok = good_id(phys);
    const uint32_t valid = kPer == 1 ? ok : __ballot_sync(0xffffffffu, e < there && ok);
    const uint32_t all = (1u << there) - 1u;
    stage_bad = (stage_bad & ~(kGroup1 << (kPer * stage))) | (all & ~valid) << (kPer * stage);
    uint32_t copied = valid;
    if (kFused && j == j_new && new_slot == 0) copied &= ~(1u << (l_new - l0));
    some_bad |= valid != all;
    if (valid != all && lane == 0) set_error(prm.err, kErrPage);
    if (lane >= kPer * kParts) return;
    if (copied) {
      if (lane == 0) mbar_arrive_expect_tx(&bars[stage], __popc(copied) * Tiles::kCopyBytes);
      // the expected bytes are set before any copy can land
      __syncwarp((1u << (kPer * kParts)) - 1u);
      if (kPer == 1 || (copied >> e & 1u))
        Tiles::copy(ws, stage, e, src, lane % kParts, kvh, phys, &bars[stage]);
    } else if (lane == 0) {
      mbar_arrive(&bars[stage]);
    }
  };
  // Fused: the appended row, one 16-byte chunk per lane (K in lanes 0..7, V
  // in 8..15). Loaded ahead of the pages and patched into the stage at its page's
  // turn; what comes before that (rotation, quantisation, the pool's copy) is done
  // there as well or, where the Tiles say so, while the first pages are on their way.
  auto load_new_row = [&]() {
    uint4 val = make_uint4(0u, 0u, 0u, 0u);
    if (lane < 16)
      val = __ldg(reinterpret_cast<const uint4*>(
          (lane >= 8 ? prm.v_new : prm.k_new) +
          (static_cast<size_t>(b) * kHkv + kvh) * kDim + (lane & 7) * 8));
    return val;
  };
  // Prefetch: the first groups' tiles at once, a lane per copy. The unfused
  // kernel defers the last page's group, whose newest row the kernel before this
  // one may be writing.
  const int n_prefetch = min(mine, kStages);
  const bool deferred = !kFused && j_new >= 0 && j_new < n_prefetch;
  {
    const int l = lane / kParts;
    const int j = l / kPer;
    const int phys = __shfl_sync(0xffffffffu, ids, l);
    const bool ok = good_id(phys);
    const bool serves = j < n_prefetch && l < my_pages && (kFused || j != j_new);
    const bool copies = serves && ok && !(kFused && l == l_new && new_slot == 0);
    const int held = min(my_pages, kStages * kPer);
    stage_bad = __ballot_sync(0xffffffffu, lane < held && !good_id(ids));
    some_bad = stage_bad != 0;
    const uint32_t all = __ballot_sync(0xffffffffu, copies && lane % kParts == 0);
    if (serves && lane % kParts == 0 && !ok) set_error(prm.err, kErrPage);
    if (j < n_prefetch && (kFused || j != j_new) && lane % (kPer * kParts) == 0) {
      const int n = __popc(all >> lane & ((1u << (kPer * kParts)) - 1u));
      if (n > 0) {
        mbar_arrive_expect_tx(&bars[j], n * Tiles::kCopyBytes);
      } else {
        mbar_arrive(&bars[j]);
      }
    }
    __syncwarp();
    if (copies) Tiles::copy(ws, j, l % kPer, src, lane % kParts, kvh, phys, &bars[j]);
  }
  pdl_wait();
  pdl_launch_dependents();
  if (deferred) issue_copy(j_new, j_new);
  // the new row's load goes out before the queries', so their latencies overlap
  uint4 new_row = make_uint4(0u, 0u, 0u, 0u);
  int new_page = -1;
  if (kFused && j_new >= 0) {
    new_row = load_new_row();
    new_page = __ldg(row + (len - 1) / kPage);
  }
  typename Tiles::Queries queries;
  Tiles::template load_queries<kRope>(
      prm.q + (static_cast<size_t>(b) * kHq + kvh * kGroup) * kDim, lane, ang_c, ang_s, queries);

  typename Tiles::NewRow made;
  if (kFused && j_new >= 0)
    made = Tiles::template make_row<kRope>(src, kvh, new_slot, new_page, good_id(new_page), new_row,
                                           ang_c, ang_s, lane);

  typename Tiles::State st;
  st.reset();
  // Groups seen whole: all their pages are there, inside the window (and valid);
  // the first one is one of the sequence's [whole_from, whole_from + whole).
  const int whole_from = sink_pages + (win_lo % kPage != 0 ? 1 : 0);
  const int whole_to = min(len / kPage - win_page + sink_pages, page_end);
  const unsigned whole = max(whole_to - kPer + 1 - whole_from, 0);
  int at = page_begin + warp * kPer;          // the group's first page
  int issued = n_prefetch;
  int consumed = 0;
  bool timed_out = false;
  int stage = 0;
  uint32_t phase = 0;
  constexpr uint32_t kAll = 0xffffffffu >> (32 - kPage * kPer);   // 16 bits a page
  // Group j has landed in `stage`: which of its tokens count. V rows that do not
  // are cleared (0 times what they hold must stay 0), and the appended row goes
  // over what the copy brought.
  auto make_ready = [&](int j, int stage, int at) {
    uint32_t seen = kAll;
    const bool with_new = kFused && j == j_new;
    if (static_cast<unsigned>(at - whole_from) >= whole || some_bad || with_new) {
      seen = 0;
      #pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const int t0 = logical(j * kPer + e) * kPage;
        uint32_t bits = 0xffffu;
        // a page inside the window, or one of sinks alone, is seen whole
        if (t0 + kPage > len || t0 < win_lo)
          bits = low_bits(len - t0) &
                 (low_bits(prm.sinks - t0) | (0xffffu & ~low_bits(win_lo - t0)));
        if ((stage_bad >> (kPer * stage + e)) & 1u) bits = 0;
        if (kPer > 1 && j * kPer + e >= my_pages) bits = 0;     // no page of this warp's
        seen |= bits << (kPage * e);
      }
    }
    if (seen != kAll || with_new) {
      Tiles::hide_rows(ws, stage, seen, lane);
      __syncwarp();
      if (with_new)
        Tiles::template put_row<kRope>(ws, stage, l_new % kPer, src, kvh, new_slot, new_page,
                                       good_id(new_page),
                                       (seen >> (l_new % kPer * kPage) & 0xffffu) != 0, made, lane);
      fence_proxy_async_smem();
      __syncwarp();
    }
    return seen;
  };
  // Every lane's reads of the stage are done: the group after those in flight.
  auto refill = [&](int j, int stage) {
    const int next = j + kStages;
    if (next >= mine) return;
    if ((next * kPer & 31) == 0) {
      ids = ids_next;
      ids_next = fetch_ids(next * kPer + 32);
    }
    issue_copy(next, stage);
    issued = next + 1;
  };
  for (int j = 0; j < mine; ++j, at += kWarps * kPer) {
    if (!__all_sync(0xffffffffu, mbar_wait(&bars[stage], phase))) {
      timed_out = true;
      break;
    }
    consumed = j + 1;
    const uint32_t seen = make_ready(j, stage, at);
    if (seen) Tiles::template attend<kRope>(ws, stage, seen, lane, queries, st);
    __syncwarp();
    refill(j, stage);
    if (++stage == kStages) {
      stage = 0;
      phase ^= 1u;
    }
  }
  if (timed_out) {
    // this warp's copies in flight land before the block exits (each wait bounded)
    for (int j = consumed; j < issued; ++j) mbar_wait(&bars[j % kStages], (j / kStages) & 1);
    if (lane == 0) set_error(prm.err, kErrTimeout);
    st.m_run = -INFINITY;
    st.l_run = 0.f;
  }

  Tiles::finish(sm, st, warp, lane);
  __syncthreads();
  float M, L;
  float2 O;
  block_merge_read<kWarps>(sm, M, L, O);
  float* out_kv = prm.out + (static_cast<size_t>(b) * kHq + kvh * kGroup) * kDim;
  if (kCluster && n_splits > 1) {
    cluster_merge_async(inbox, M, L, O, warp, lane, out_kv, prm.err);
    return;
  }
  if (n_splits == 1) {
    const float inv = L > 0.f ? 1.f / L : 0.f;
    *reinterpret_cast<float2*>(out_kv + warp * kDim + 2 * lane) = make_float2(O.x * inv, O.y * inv);
    return;
  }
  if constexpr (!kCluster)
    ticket_merge(sm, prm.part_o, prm.part_ml, prm.tickets, prm.max_splits, prm.out, b, kvh, split,
                 n_splits, M, L, O, warp, lane);
}

// ---------------------------------------------------------------- host
template <class Tiles>
using WindowKernel = void (*)(const typename Tiles::Source, const WindowParams);

template <class Tiles, bool kCluster>
WindowKernel<Tiles> window_kernel(bool fused, bool rope) {
  return fused ? (rope ? window_decode_kernel<true, kCluster, true, Tiles>
                       : window_decode_kernel<true, kCluster, false, Tiles>)
               : (rope ? window_decode_kernel<false, kCluster, true, Tiles>
                       : window_decode_kernel<false, kCluster, false, Tiles>);
}

// The launch: splits per sequence (a cluster, or a ticket), or units.
struct WindowPlan {
  int num_splits;   // 0: units
  bool cluster;
  int units;        // units in the grid
  int wave_units;
  int range_div;
  int least_pages;
};

// Small batches take a cluster per (sequence, kv head), whose merge is shorter
// than the ticket's, of the size that its tiles choose from the batch's rows (times
// 8 KV heads) and the slots of resident cluster blocks, while the pages a sequence
// can see are few for it or the blocks fill enough of the slots. Everything else
// takes units.
template <class Tiles>
WindowPlan plan_window(const pkv_pool* pool, const WindowResidency& res, int batch, int window,
                       int sinks, int num_splits) {
  const pkv_pool_config& c = pool->cfg;
  const int max_pages = c.max_seq_len / kPage;
  // the most pages a sequence can see
  const int seen = std::min(max_pages, (sinks + kPage - 1) / kPage + (window - 1) / kPage + 2);
  WindowPlan p = {};
  if (num_splits > 0) {
    p.num_splits = num_splits;
    p.cluster = num_splits >= 2 && num_splits <= pool->max_cluster;
    return p;
  }
  const long long rows = static_cast<long long>(batch) * kHkv;
  const long long cluster_slots =
      static_cast<long long>(res.cluster_blocks_per_sm) * pool->num_sms;
  constexpr int kBlockPages = kWarps * Tiles::kStagePages;      // of one turn of a block
  const int s = std::min({Tiles::cluster_size(rows, cluster_slots), pool->max_cluster,
                          c.max_splits, (seen + kBlockPages - 1) / kBlockPages});
  if (s >= 2 && rows * s <= cluster_slots &&
      (seen <= 4 * kBlockPages * s || Tiles::fills(rows * s, cluster_slots))) {
    p.num_splits = s;
    p.cluster = true;
    return p;
  }
  const int wave = std::max(1, res.blocks_per_sm * pool->num_sms / kHkv);
  const int fewest = (seen + c.max_splits - 1) / c.max_splits;   // keeps to max_splits ranges
  if (batch <= std::min(wave, 32 * kHeld)) p.wave_units = wave;
  p.range_div = std::max(1, 3 * wave / 5);
  p.least_pages = std::max(2 * kWarps, fewest);
  p.units = std::max(p.wave_units, batch + p.range_div);
  return p;
}

// src: the pool as the kernel takes it, once the arguments are known to be good.
template <class Tiles, bool kFused, class MakeSource>
pkv_status launch_window(pkv_pool_t pool, int layer, const void* q, const void* k, const void* v,
                         bool pools_good, const MakeSource& make_source,
                         const int32_t* block_tables, const int32_t* seq_lens, float* out,
                         int window, int sinks, const pkv_axes_rope* rope,
                         const int32_t* rope_positions,
                         int position_stride, int batch, int num_splits, void* stream) {
  if (!pool) return PKV_ERR_INVALID_ARG;
  const pkv_pool_config& c = pool->cfg;
  if (layer < 0 || layer >= c.num_layers || batch < 0 || batch > c.max_batch)
    return PKV_ERR_INVALID_ARG;
  if (num_splits < 0 || num_splits > c.max_splits || window < 1 || sinks < 0)
    return PKV_ERR_INVALID_ARG;
  if (batch == 0) return PKV_OK;
  if (!q || !pools_good || !block_tables || !seq_lens || !out || (kFused && (!k || !v)))
    return PKV_ERR_INVALID_ARG;
  if (!pkv_aligned16(q) || !pkv_aligned16(k) || !pkv_aligned16(v) ||
      !pkv_aligned16(block_tables) || !pkv_aligned4(seq_lens) ||
      !pkv_aligned16(out))
    return PKV_ERR_INVALID_ARG;
  WindowParams prm = {};
  if (rope) {
    const pkv_status st = make_axes_args(rope, rope_positions, position_stride, batch, &prm.rope);
    if (st != PKV_OK) return st;
  }
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev != pool->device) return PKV_ERR_INVALID_ARG;

  const int max_pages = c.max_seq_len / kPage;
  const size_t parity = layer & 1;
  prm.q = static_cast<const uint16_t*>(q);
  prm.k_new = static_cast<const uint16_t*>(k);
  prm.v_new = static_cast<const uint16_t*>(v);
  prm.table = block_tables + static_cast<size_t>(layer) * c.max_batch * max_pages;
  prm.seq_lens = seq_lens;
  prm.out = out;
  prm.part_o = pool->part_o + parity * c.max_batch * kHq * c.max_splits * kDim;
  prm.part_ml = pool->part_ml + parity * c.max_batch * kHq * c.max_splits;
  prm.tickets = pool->tickets + parity * c.max_batch * kHkv;
  prm.err = pool->err;
  prm.num_pages = c.num_pages;
  prm.table_stride = max_pages;
  prm.max_seq_len = c.max_seq_len;
  prm.max_splits = c.max_splits;
  prm.window = std::min(window, c.max_seq_len);
  prm.sinks = std::min(sinks, c.max_seq_len);
  const WindowPlan plan = plan_window<Tiles>(pool, Tiles::residency(pool), batch, prm.window,
                                             prm.sinks, num_splits);
  const bool cluster = plan.cluster;
  prm.num_splits = plan.num_splits;
  prm.batch = batch;
  prm.wave_units = plan.wave_units;
  prm.range_div = plan.range_div;
  prm.least_pages = plan.least_pages;

  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = plan.num_splits > 0 ? dim3(plan.num_splits, kHkv, batch)
                                    : dim3(plan.units * kHkv, 1, 1);
  cfg.blockDim = dim3(kThreadsW, 1, 1);
  cfg.dynamicSmemBytes = cluster ? kClusterSmemBytes<Tiles> : kTicketSmemBytes<Tiles>;
  cfg.stream = static_cast<cudaStream_t>(stream);
  typename Tiles::Source src;
  if (!make_source(src)) return PKV_ERR_CUDA;
  cudaLaunchAttribute attrs[2];
  int n_attrs = 0;
  if (cluster) {
    attrs[n_attrs].id = cudaLaunchAttributeClusterDimension;
    attrs[n_attrs].val.clusterDim.x = prm.num_splits;
    attrs[n_attrs].val.clusterDim.y = 1;
    attrs[n_attrs].val.clusterDim.z = 1;
    ++n_attrs;
  }
  if (pkv_starts_early(pool)) {
    attrs[n_attrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[n_attrs].val.programmaticStreamSerializationAllowed = 1;
    ++n_attrs;
  }
  cfg.attrs = attrs;
  cfg.numAttrs = n_attrs;
  const WindowKernel<Tiles> kernel = cluster ? window_kernel<Tiles, true>(kFused, rope != nullptr)
                                             : window_kernel<Tiles, false>(kFused, rope != nullptr);
  if (cudaLaunchKernelEx(&cfg, kernel, src, prm) != cudaSuccess) return PKV_ERR_CUDA;
  return pkv_check_launch();
}

// The kernels' attributes, and how many of their blocks an SM holds.
template <class Tiles>
bool setup_window(WindowResidency* res) {
  bool ok = true;
  for (int v = 0; v < 4 && ok; ++v) {
    const WindowKernel<Tiles> ticket = window_kernel<Tiles, false>(v & 1, v & 2);
    const WindowKernel<Tiles> cluster = window_kernel<Tiles, true>(v & 1, v & 2);
    ok = cudaFuncSetAttribute(ticket, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(kTicketSmemBytes<Tiles>)) == cudaSuccess &&
         cudaFuncSetAttribute(cluster, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(kClusterSmemBytes<Tiles>)) == cudaSuccess &&
         cudaFuncSetAttribute(cluster, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) ==
             cudaSuccess;
  }
  ok = ok && cudaOccupancyMaxActiveBlocksPerMultiprocessor(
                 &res->blocks_per_sm, window_kernel<Tiles, false>(true, true), kThreadsW,
                 kTicketSmemBytes<Tiles>) == cudaSuccess;
  ok = ok && cudaOccupancyMaxActiveBlocksPerMultiprocessor(
                 &res->cluster_blocks_per_sm, window_kernel<Tiles, true>(true, true), kThreadsW,
                 kClusterSmemBytes<Tiles>) == cudaSuccess;
  if (res->blocks_per_sm < 1) res->blocks_per_sm = 1;
  if (res->cluster_blocks_per_sm < 1) res->cluster_blocks_per_sm = 1;
  return ok;
}

}  // namespace pkv_window

#endif  // PKV_WINDOW_DEVICE_CUH
