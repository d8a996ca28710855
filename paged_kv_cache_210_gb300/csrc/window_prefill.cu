// Windowed prefill attention over the paged KV cache for GB300 (sm_103a): a
// chunk's tokens attend behind a sliding window, with sinks (declared in
// include/pkv_window.h).
//
// out_i = sum_t p_it V_t / sum_t p_it, p_it = 2^(q_i.K_t log2(e) / 8 - m_i), over
// the tokens visible from position p_i: one pass per 64-token query tile
// with a running maximum m_i and sum per row.
//
// Like the full-context kernel (prefill.cu) one CTA takes a (sequence, kv
// head, 64-token tile): 256 rows (token x 4 heads) in two halves of 128, K and
// V steps of 64 keys (4 pages) brought by two loader warps, scores and
// values on tcgen05 with accumulators in tensor memory, and eight softmax
// warps with one row per thread. What the window changes:
//  * the steps of a tile are those that hold a visible key: the sink steps and
//    the window's steps. Pages in them without a visible token, or with an
//    invalid id, are read as a page past the pool's end, which the copy
//    engine fills with zeros, so every step moves the same bytes;
//  * page ids come straight from the block table, one step ahead, so the
//    context's length does not appear in shared memory;
//  * a step's row masks are 64-bit words, built only in steps on an edge (the
//    diagonal, the window's start, the sinks' end) or with an invalid page;
//  * probabilities enter the value product as three BF16 terms (24 bits): a
//    score tile of 64 columns becomes 96 columns of P, so two tiles per row
//    half are held (2 x 2 x 96 columns, and 2 x 64 for O, fill the 512). A
//    tile is free again once its value product is done, which takes less
//    than the softmax of the other tile.

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <algorithm>
#include <mutex>

#include "pkv.h"
#include "pkv_window.h"
#include "device_common.cuh"
#include "pool_internal.h"
#include "prefill_device.cuh"

using namespace pkv_dev;
using namespace pkv_prefill_dev;

namespace {

constexpr int kRowHalves = 2;                        // MMAs of M = 128 rows per CTA
constexpr int kHalfRows = 128;
constexpr int kRows = kRowHalves * kHalfRows;        // 256 rows: token x head
constexpr int kTileTokens = kRows / kGroup;          // 64 query tokens per CTA
constexpr int kStepKeys = 64;                        // keys per step: the S MMA's N
constexpr int kStepPages = kStepKeys / kPage;        // 4
constexpr int kSoftmaxWarps = 4 * kRowHalves;        // one per (lane quarter, row half)
constexpr int kSoftmaxThreads = kSoftmaxWarps * 32;
constexpr int kLoadWarp = kSoftmaxWarps;             // Q and K copies, then V (+ 1)
constexpr int kScoreWarp = kSoftmaxWarps + 2;
constexpr int kValueWarp0 = kSoftmaxWarps + 3;       // one per row half
constexpr int kThreads = kSoftmaxThreads + 96 + 32 * kRowHalves;
constexpr int kKStages = 6;
constexpr int kVStages = 5;
constexpr int kSTiles = 2;                           // score (then P) tiles per row half
constexpr int kTileCols = 96;                        // S: 64 columns; P: 3 parts x 32 columns
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemO = kSTiles * kRowHalves * kTileCols;   // O of row half h at + 64 h
static_assert(kTmemO + kRowHalves * kDim == kTmemCols, "tensor memory is filled exactly");
constexpr float kRescaleLog2 = 8.f;                  // lazy max: p <= 2^8
constexpr uint32_t kStepBytes = kStepKeys * kRowBytes;

struct WindowPrefillSmem {                           // every tile 1024-byte aligned
  uint8_t q[kRows * kRowBytes];                      // 32 KiB
  uint8_t k[kKStages][kStepBytes];                   // 6 x 8 KiB
  uint8_t v[kVStages][kStepBytes];                   // 5 x 8 KiB
  unsigned long long bar_q, bar_k[kKStages], bar_v[kVStages], bar_s[kSTiles], bar_p[kSTiles];
  unsigned long long bar_o[kSTiles];                 // P(j) V(j) done, per tile
  unsigned long long k_free[kKStages], v_free[kVStages];
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(offsetof(WindowPrefillSmem, k) % 1024 == 0 &&
                  offsetof(WindowPrefillSmem, v) % 1024 == 0,
              "swizzled tiles start on 1024-byte boundaries");
constexpr size_t kSmemBytes = sizeof(WindowPrefillSmem) + 1024;   // + room to align the base
static_assert(kSmemBytes <= 227 * 1024, "one CTA's shared memory");

struct WindowPrefillParams {
  const int32_t* table;       // this layer's block tables [max_batch][table_stride]
  const int32_t* cu_tokens;   // [batch + 1]
  const int32_t* start_pos;   // [batch]
  float* out;                 // [total][32][64]
  int* err;
  int num_pages;
  int table_stride;
  int max_seq_len;
  int tiles_max;              // gridDim.y: tiles per sequence the launch covers
  int total_tokens;
  int window;                 // 1 .. max_seq_len
  int sinks;                  // 0 .. max_seq_len
};

// The lowest n bits of 64 (n clamped to 0 .. 64).
__device__ __forceinline__ unsigned long long low_bits64(int n) {
  return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull;
}

// What the tile (and each of its steps) sees of the sequence.
struct TileView {
  int p_first, p_last;   // positions of the tile's first and last token
  int n_keys;            // p_last + 1
  int lo;                // first key inside some row's window
  int sink_steps;        // steps of sinks before the window's
  int win_step;          // the window's first step
  int n_steps;
  int sinks;

  __device__ TileView(int first, int count, int window, int sinks_) {
    p_first = first;
    p_last = first + count - 1;
    n_keys = p_last + 1;
    lo = max(p_first - window + 1, 0);
    sinks = sinks_;
    win_step = lo / kStepKeys;
    sink_steps = min((sinks + kStepKeys - 1) / kStepKeys, win_step);
    n_steps = sink_steps + (n_keys + kStepKeys - 1) / kStepKeys - win_step;
  }
  __device__ int step(int j) const { return j < sink_steps ? j : j - sink_steps + win_step; }
  // whether logical page lp holds a key that some row sees
  __device__ bool wants(int lp) const {
    return lp * kPage < n_keys && ((lp + 1) * kPage > lo || lp * kPage < sinks);
  }
};

__global__ void __launch_bounds__(kThreads, 1) window_prefill_kernel(
    const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
    const __grid_constant__ CUtensorMap tmap_v, const WindowPrefillParams prm) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  WindowPrefillSmem& sm = *reinterpret_cast<WindowPrefillSmem*>(smem_raw + pad);

  const int tile = prm.tiles_max - 1 - static_cast<int>(blockIdx.y);   // heaviest first
  const int g = blockIdx.x;
  const int b = blockIdx.z;
  const int tid = threadIdx.x;
  const int warp = tid >> 5;

  const int row0 = prm.cu_tokens[b];
  const int n = prm.cu_tokens[b + 1] - row0;
  const int start = prm.start_pos[b];
  if (row0 < 0 || n < 0 || n > prm.total_tokens - row0) {   // rows outside the caller's buffers
    if (blockIdx.y == 0 && g == 0 && tid == 0) set_error(prm.err, PKV_DEV_ERR_SEQ_LEN);
    return;
  }
  if (blockIdx.y == 0 && g == 0 && tid == 0 && n > prm.tiles_max * kTileTokens)
    set_error(prm.err, PKV_DEV_ERR_SEQ_LEN);
  if (tile * kTileTokens >= n) return;                 // the whole CTA, before any allocation
  if (start < 0 || start > prm.max_seq_len || n > prm.max_seq_len - start) {
    if (tid == 0) set_error(prm.err, PKV_DEV_ERR_POSITION);
    return;
  }
  const int t_valid = min(kTileTokens, n - tile * kTileTokens);
  const TileView view(start + tile * kTileTokens, t_valid, prm.window, prm.sinks);
  const int n_steps = view.n_steps;
  const int32_t* trow = prm.table + static_cast<size_t>(b) * prm.table_stride;

  // invalid ids among the pages that count are flagged once, here
  bool bad_page = false;
  for (int i = tid; i < n_steps * kStepPages; i += kThreads) {
    const int lp = view.step(i / kStepPages) * kStepPages + i % kStepPages;
    if (!view.wants(lp)) continue;
    const int id = __ldg(trow + lp);
    bad_page |= id < 0 || id >= prm.num_pages;
  }
  if (bad_page) set_error(prm.err, PKV_DEV_ERR_PAGE);

  if (tid == 0) {
    mbar_init(&sm.bar_q, 1);
    for (int i = 0; i < kKStages; ++i) mbar_init(&sm.bar_k[i], 1);
    for (int i = 0; i < kVStages; ++i) mbar_init(&sm.bar_v[i], 1);
    for (int i = 0; i < kSTiles; ++i) mbar_init(&sm.bar_s[i], 1);
    for (int i = 0; i < kSTiles; ++i) mbar_init(&sm.bar_p[i], kSoftmaxThreads);
    // the value barriers complete once both row halves' issuers committed
    for (int i = 0; i < kSTiles; ++i) mbar_init(&sm.bar_o[i], kRowHalves);
    for (int i = 0; i < kKStages; ++i) mbar_init(&sm.k_free[i], 1);
    for (int i = 0; i < kVStages; ++i) mbar_init(&sm.v_free[i], kRowHalves);
    sm.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(&sm.tmem_base, kTmemCols);
  tc_fence_before();
  const bool any_bad_page = __syncthreads_or(bad_page);
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  volatile int* abort_flag = &sm.abort_flag;

  if (warp == kLoadWarp || warp == kLoadWarp + 1) {
    // ------------------------------------------------------------ copy engine
    // Lanes 0..3 copy the step's 4 pages in one instruction once lane 0 saw
    // the stage free. A page that does not count is copied from past the
    // pool's end: zeros.
    const int lane = lane_of(tid);
    const bool is_v = warp != kLoadWarp;
    const CUtensorMap* map = is_v ? &tmap_v : &tmap_k;
    const int stages = is_v ? kVStages : kKStages;
    if (lane == 0) {
      asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
      if (!is_v) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_q))
                     : "memory");
        mbar_arrive_expect_tx(&sm.bar_q, kRows * kRowBytes);
        tma_load_3d(sm.q, &tmap_q, 0, g * kGroup, row0 + tile * kTileTokens, &sm.bar_q);
      }
    }
    auto page_of = [&](int j) {
      int id = prm.num_pages;
      if (j < n_steps && lane < kStepPages) {
        const int lp = view.step(j) * kStepPages + lane;
        if (view.wants(lp)) id = __ldg(trow + lp);
        if (id < 0 || id >= prm.num_pages) id = prm.num_pages;
      }
      return id;
    };
    int page = page_of(0);
    int issued = 0;
    bool ok = true;
    for (int j = 0; j < n_steps; ++j) {
      const int st = j % stages;
      unsigned long long* full = is_v ? &sm.bar_v[st] : &sm.bar_k[st];
      const int next_page = page_of(j + 1);
      bool good = true;
      if (lane == 0) {
        good = *abort_flag == 0;
        if (good && j >= stages)
          good = mbar_wait(is_v ? &sm.v_free[st] : &sm.k_free[st], ((j - stages) / stages) & 1);
        if (good) mbar_arrive_expect_tx(full, kStepBytes);
      }
      if (!__shfl_sync(0xffffffffu, good ? 1 : 0, 0)) {
        ok = false;
        break;
      }
      if (lane < kStepPages)
        tma_load_3d((is_v ? sm.v[st] : sm.k[st]) + lane * kPage * kRowBytes, map, 0, g * kPage,
                    page, full);
      __syncwarp();
      page = next_page;
      ++issued;
    }
    if (lane == 0) {
      if (!ok) {
        *abort_flag = 1;
        set_error(prm.err, PKV_DEV_ERR_TIMEOUT);
      }
      // every copy issued lands before the CTA frees its memory (bounded waits)
      if (!is_v) mbar_wait(&sm.bar_q, 0);
      for (int s = 0; s < stages; ++s) {
        const int uses = (issued - s + stages - 1) / stages;
        if (uses > 0) mbar_wait(is_v ? &sm.bar_v[s] : &sm.bar_k[s], (uses - 1) & 1);
      }
    }
  } else if (warp >= kScoreWarp) {
    // ------------------------------------------------------------ tensor cores
    // One issuing thread for the scores, one per row half for the values.
    if (lane_of(tid) == 0) {
      const bool scores = warp == kScoreWarp;
      const int half = warp - kValueWarp0;
      int issued = 0;
      bool ok = true;
      if (scores) {
        const uint32_t idesc_s = instr_desc(kHalfRows, kStepKeys, false);
        const uint64_t q_desc = smem_desc_sw128(smem_u32(sm.q), 16, 1024);
        ok = mbar_wait(&sm.bar_q, 0);
        for (int j = 0; ok && j < n_steps; ++j) {
          // S(j) = Q K(j)^T into tile j % 2, once K(j) landed and P(j - 2) V(j - 2),
          // which reads that tile, is done
          if (*abort_flag || !mbar_wait(&sm.bar_k[j % kKStages], (j / kKStages) & 1) ||
              (j >= kSTiles &&
               !mbar_wait(&sm.bar_o[j % kSTiles], ((j - kSTiles) / kSTiles) & 1))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t k_desc = smem_desc_sw128(smem_u32(sm.k[j % kKStages]), 16, 1024);
          #pragma unroll
          for (int kk = 0; kk < kDim / 16; ++kk) {
            #pragma unroll
            for (int h = 0; h < kRowHalves; ++h)
              mma_bf16(tmem + ((j % kSTiles) * kRowHalves + h) * kTileCols,
                       q_desc + h * (kHalfRows * kRowBytes >> 4) + kk * 2, k_desc + kk * 2,
                       idesc_s, kk > 0);
          }
          mma_commit(&sm.bar_s[j % kSTiles]);
          mma_commit(&sm.k_free[j % kKStages]);
          ++issued;
        }
      } else {
        const uint32_t idesc_o = instr_desc(kHalfRows, kDim, true);
        for (int j = 0; ok && j < n_steps; ++j) {
          // O += P(j) V(j), P's three parts 32 columns apart, 16 keys per 8 columns
          if (*abort_flag || !mbar_wait(&sm.bar_p[j % kSTiles], (j / kSTiles) & 1) ||
              !mbar_wait(&sm.bar_v[j % kVStages], (j / kVStages) & 1)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t v_desc = smem_desc_sw128(smem_u32(sm.v[j % kVStages]), 8192, 1024);
          const uint32_t p_tile = tmem + ((j % kSTiles) * kRowHalves + half) * kTileCols;
          const uint32_t o_tile = tmem + kTmemO + half * kDim;
          #pragma unroll
          for (int part = 0; part < 3; ++part) {
            #pragma unroll
            for (int kk = 0; kk < kStepKeys / 16; ++kk)
              mma_bf16_tmem_a(o_tile, p_tile + part * 32 + kk * 8,
                              v_desc + kk * (16 * kRowBytes >> 4), idesc_o,
                              (j > 0 || kk > 0 || part > 0) ? 1u : 0u);
          }
          mma_commit(&sm.bar_o[j % kSTiles]);
          mma_commit(&sm.v_free[j % kVStages]);
          ++issued;
        }
      }
      if (!ok) {
        *abort_flag = 1;
        set_error(prm.err, PKV_DEV_ERR_TIMEOUT);
      }
      // every product this thread issued completes before the CTA frees its memory
      if (scores) {
        for (int t = 0; t < kSTiles; ++t) {
          const int uses = (issued - t + kSTiles - 1) / kSTiles;
          if (uses > 0) mbar_wait(&sm.bar_s[t], (uses - 1) & 1);
        }
      } else if (issued > 0) {
        mbar_wait(&sm.bar_o[(issued - 1) % kSTiles], ((issued - 1) / kSTiles) & 1);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax warps
    const int rh = warp >> 2;                           // row half
    const int r = (warp & 3) * 32 + (tid & 31);         // its MMA row = tensor-memory lane
    const int tok = (rh * kHalfRows + r) >> 2;          // token of the tile, head r & 3
    const uint32_t o_col = kTmemO + rh * kDim;
    const int pos = view.p_first + min(tok, t_valid - 1);   // rows past the chunk mirror its last
    const float c = 1.4426950408889634f * 0.125f;       // log2(e) / sqrt(64)
    const uint32_t lane_addr = static_cast<uint32_t>((warp & 3) * 32) << 16;
    float m_run = -INFINITY, l_run = 0.f;
    bool ok = true;
    for (int j = 0; j < n_steps; ++j) {
      // one verdict per warp (the tensor-memory accesses below are warp-wide)
      if (!__all_sync(0xffffffffu, *abort_flag == 0 &&
                                       mbar_wait(&sm.bar_s[j % kSTiles], (j / kSTiles) & 1))) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t st_tile = tmem + lane_addr + ((j % kSTiles) * kRowHalves + rh) * kTileCols;
      uint32_t sv[64];                                   // the row's 64 keys of the step
      {
        uint32_t (&a)[32] = *reinterpret_cast<uint32_t(*)[32]>(&sv[0]);
        uint32_t (&b2)[32] = *reinterpret_cast<uint32_t(*)[32]>(&sv[32]);
        tmem_ld32(st_tile, a);
        tmem_ld32(st_tile + 32, b2);
      }
      const int key0 = view.step(j) * kStepKeys;
      // some key of the step is hidden from some row
      const bool edge = key0 + kStepKeys - 1 > view.p_first ||
                        (key0 <= view.p_last - prm.window && key0 + kStepKeys > view.sinks);
      if (edge || any_bad_page) {
        unsigned long long seen =
            low_bits64(pos + 1 - key0) &
            (low_bits64(view.sinks - key0) | ~low_bits64(pos - prm.window + 1 - key0));
        if (any_bad_page) {
          for (int e = 0; e < kStepPages; ++e) {
            const int lp = key0 / kPage + e;
            const int id = view.wants(lp) ? __ldg(trow + lp) : -1;
            if (id < 0 || id >= prm.num_pages) seen &= ~(0xffffull << (16 * e));
          }
        }
        const uint32_t w0 = static_cast<uint32_t>(seen), w1 = static_cast<uint32_t>(seen >> 32);
        #pragma unroll
        for (int i = 0; i < 32; ++i) {
          if (!((w0 >> i) & 1u)) sv[i] = __float_as_uint(-INFINITY);
          if (!((w1 >> i) & 1u)) sv[i + 32] = __float_as_uint(-INFINITY);
        }
      }
      float mx8[8];
      #pragma unroll
      for (int e = 0; e < 8; ++e) mx8[e] = __uint_as_float(sv[e]);
      #pragma unroll
      for (int i = 8; i < 64; ++i) mx8[i & 7] = fmaxf(mx8[i & 7], __uint_as_float(sv[i]));
      const float m_step = fmaxf(fmaxf(fmaxf(mx8[0], mx8[1]), fmaxf(mx8[2], mx8[3])),
                                 fmaxf(fmaxf(mx8[4], mx8[5]), fmaxf(mx8[6], mx8[7]))) * c;
      float alpha = 1.f;
      const bool grow = m_step > m_run + kRescaleLog2;   // false while nothing was visible
      if (grow) {
        alpha = fast_exp2(m_run - m_step);
        m_run = m_step;
        l_run *= alpha;
      }
      {
        const float mu = m_run == -INFINITY ? 0.f : m_run;
        const float2 c2 = make_float2(c, c);
        const float2 nm2 = make_float2(-mu, -mu);
        const float2 neg1 = make_float2(-1.f, -1.f);
        float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                         make_float2(0.f, 0.f)};
        #pragma unroll
        for (int kh = 0; kh < 2; ++kh) {
          uint32_t hi[16], mid[16], lo[16];
          #pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const int k = kh * 32 + i;
            const float2 x = __ffma2_rn(
                make_float2(__uint_as_float(sv[k]), __uint_as_float(sv[k + 1])), c2, nm2);
            const float2 pp = make_float2(fast_exp2(x.x), fast_exp2(x.y));
            acc[(i >> 1) & 3] = __fadd2_rn(acc[(i >> 1) & 3], pp);
            // p = hi + mid + lo: two truncated parts, the rest rounded
            const uint32_t b0 = __float_as_uint(pp.x), b1 = __float_as_uint(pp.y);
            hi[i / 2] = __byte_perm(b0, b1, 0x7632);
            const float2 r1 = __ffma2_rn(make_float2(__uint_as_float(b0 & 0xffff0000u),
                                                     __uint_as_float(b1 & 0xffff0000u)),
                                         neg1, pp);
            const uint32_t c0 = __float_as_uint(r1.x), c1 = __float_as_uint(r1.y);
            mid[i / 2] = __byte_perm(c0, c1, 0x7632);
            const float2 r2 = __ffma2_rn(make_float2(__uint_as_float(c0 & 0xffff0000u),
                                                     __uint_as_float(c1 & 0xffff0000u)),
                                         neg1, r1);
            lo[i / 2] = float2_to_bf16x2(r2.x, r2.y);
          }
          // the scores of both halves are in registers already: P may overwrite them
          tmem_st16(st_tile + kh * 16, hi);
          tmem_st16(st_tile + 32 + kh * 16, mid);
          tmem_st16(st_tile + 64 + kh * 16, lo);
        }
        const float2 a = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
        l_run += a.x + a.y;
      }

      // a row that grew its max rescales its O, once P(j - 1) V(j - 1) is done
      bool failed = false;
      if (j > 0 && __any_sync(0xffffffffu, grow)) {
        failed = !__all_sync(0xffffffffu,
                             mbar_wait(&sm.bar_o[(j - 1) % kSTiles], ((j - 1) / kSTiles) & 1));
        tc_fence_after();
        if (!failed) {
          #pragma unroll
          for (int dh = 0; dh < 2; ++dh) {
            uint32_t ov[32];
            tmem_ld32(tmem + lane_addr + o_col + dh * 32, ov);
            #pragma unroll
            for (int d = 0; d < 32; ++d) ov[d] = __float_as_uint(__uint_as_float(ov[d]) * alpha);
            tmem_st32(tmem + lane_addr + o_col + dh * 32, ov);
          }
        }
      }
      // V rows that no row of the tile sees, in pages that were read (zero, so
      // that p = 0 times them stays 0): past the last key, or between the
      // sinks and the window
      const bool dead_tail = key0 + kStepKeys > view.n_keys;
      const bool dead_gap = max(key0, view.sinks) < min(key0 + kStepKeys, view.lo);
      if (!failed && (dead_tail || dead_gap)) {
        if (__all_sync(0xffffffffu, mbar_wait(&sm.bar_v[j % kVStages], (j / kVStages) & 1))) {
          for (int idx = tid; idx < kStepKeys * 8; idx += kSoftmaxThreads) {
            const int key = key0 + (idx >> 3);
            if (key >= view.n_keys || (key >= view.sinks && key < view.lo))
              *reinterpret_cast<uint4*>(sm.v[j % kVStages] + idx * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        } else {
          failed = true;
        }
      }
      if (failed) {
        ok = false;
        break;
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&sm.bar_p[j % kSTiles]);
    }
    if (!ok) {
      *abort_flag = 1;
      set_error(prm.err, PKV_DEV_ERR_TIMEOUT);
    }
    const bool done = ok && !*abort_flag &&
                      mbar_wait(&sm.bar_o[(n_steps - 1) % kSTiles], ((n_steps - 1) / kSTiles) & 1);
    if (__all_sync(0xffffffffu, done)) {
      tc_fence_after();
      const float inv = l_run > 0.f ? 1.f / l_run : 0.f;
      float* dst = prm.out + ((static_cast<size_t>(row0) + tile * kTileTokens + tok) * kHq +
                              g * kGroup + (r & 3)) * kDim;
      #pragma unroll
      for (int dh = 0; dh < 2; ++dh) {
        uint32_t ov[32];
        tmem_ld32(tmem + lane_addr + o_col + dh * 32, ov);
        if (tok < t_valid) {
          #pragma unroll
          for (int d = 0; d < 32; d += 4)
            *reinterpret_cast<float4*>(dst + dh * 32 + d) =
                make_float4(__uint_as_float(ov[d]) * inv, __uint_as_float(ov[d + 1]) * inv,
                            __uint_as_float(ov[d + 2]) * inv, __uint_as_float(ov[d + 3]) * inv);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ---------------------------------------------------------------- host
bool set_smem_attribute(int device) {
  constexpr int kMaxDevices = 64;
  static std::mutex lock;
  static bool done[kMaxDevices] = {};
  if (device < 0 || device >= kMaxDevices) return false;
  std::lock_guard<std::mutex> guard(lock);
  if (!done[device]) {
    if (cudaFuncSetAttribute(window_prefill_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSmemBytes)) != cudaSuccess)
      return false;
    done[device] = true;
  }
  return true;
}

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
      !pkv_aligned16(block_tables) || !pkv_aligned16(cu_tokens) || !pkv_aligned16(start_pos) ||
      !pkv_aligned16(out))
    return PKV_ERR_INVALID_ARG;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev != pool->device) return PKV_ERR_INVALID_ARG;
  if (!set_smem_attribute(pool->device)) return PKV_ERR_CUDA;

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
  window_prefill_kernel<<<dim3(kHkv, prm.tiles_max, batch), kThreads, kSmemBytes,
                          static_cast<cudaStream_t>(stream)>>>(tq, tk, tv, prm);
  return pkv_check_launch();
}
