// Internal to libpkv: attention of query tiles over paged K and V on tcgen05,
// the kernel behind windowed prefill (window_prefill.cu) and drafted trees
// (tree.cu). A job says which tiles there are, what each sees of its sequence
// and where its results go.
//
// out_i = sum_t p_it V_t / sum_t p_it, p_it = 2^(q_i.K_t log2(e) / 8 - m_i), over
// the tokens that row i sees: one pass per 32-token query tile with a running
// maximum m_i and sum per row.
//
// Like the full-context kernel (prefill.cu) a CTA takes the rows (token x 4
// heads) of a query tile of one (sequence, kv head), K and V come in steps of
// 64 keys (4 pages) by two loader warps, scores and values run on tcgen05 with
// accumulators in tensor memory, and the softmax warps hold one row per
// thread. What is different, and why:
//  * a tile's steps are its visible pages, the sinks' and then the window's, four
//    at a time wherever they lie (steps aligned to 64 tokens, with one more for
//    four sinks, took 4 % longer behind 512 and 3 % behind 4,096 tokens). What
//    the last step lacks, and pages with an invalid id, are read as a page past
//    the pool's end, which the copy engine fills with zeros, so every step
//    moves the same bytes;
//  * page ids come straight from the block table, eight steps at a time, so
//    the context's length does not appear in shared memory;
//  * a tile has 32 tokens (128 rows), two CTAs share an SM, and the CTAs of one
//    wave draw their tiles from a counter: behind a window a tile is a few
//    steps long, so the next tile's copies and scores run under the last one's
//    end, and each CTA's start and end under the other's steps;
//  * rows of V that no row of the tile sees are cleared by the V loader before
//    it completes a stage, and a step's row masks are two 32-bit words, built
//    only in steps on an edge (the diagonal, the window's start, the sinks'
//    end) or with an invalid page;
//  * probabilities enter the value product as three BF16 terms (24 bits) in
//    columns of their own (S 64, P 96 and O 64 of the CTA's 256), so the next
//    step's scores are computed as soon as this step's are in registers;
//  * O leaves tensor memory every kSegment steps and is added up in FP32 in
//    registers: a tensor-core sum drops the bits below its accumulator's last
//    one, always downwards, 12 times a step, which over a 4,096-token window
//    came to 1.5e-5 of the output. With segments of four steps it is 1.1e-6
//    (472 us in the first case below, then), of two 6.4e-7 (483 us), of one
//    4.4e-7 (506 us).
//
// What a job brings:
//   Work                  a tile, as the K loader hands it to the other warps: b
//                         (sequence), g (KV head), row (its first of q and out),
//                         count (rows, 1 .. 32; 0: the end), bad_page (some page
//                         that counts has an invalid id), and what its view needs
//   Params, View          its parameters, what a tile sees: pages
//                         (has_page, page, n_pages), steps (first_step, n_steps;
//                         plain_from, plain_to and has_dead count from the first),
//                         keys that no row sees (dead)
//   Walk, kDrawn          tile number -> Work, numbers ever larger, drawn from a
//                         counter by the launch's CTAs (Params: next_tile, ctas_done);
//                         or the walk shares the tiles out and takes no number
//   Row                   what one row sees of a page
//   kFewRows              tiles may leave whole softmax warps without rows
//   kParts, is_whole, ... a tile may be a part of its rows' keys
#ifndef PKV_PREFILL_TILES_CUH
#define PKV_PREFILL_TILES_CUH

#include <cuda.h>
#include <cuda_runtime.h>
#include <float.h>
#include <stddef.h>
#include <stdint.h>

#include <mutex>

#include "pkv.h"
#include "device_common.cuh"
#include "pool_internal.h"
#include "prefill_device.cuh"

namespace pkv_tiles {

using namespace pkv_dev;
using namespace pkv_prefill_dev;

constexpr int kRows = 128;                           // an MMA's M: token x head
constexpr int kTileTokens = kRows / kGroup;          // 32 query tokens per CTA
constexpr int kStepKeys = 64;                        // keys per step: the S MMA's N
constexpr int kStepPages = kStepKeys / kPage;        // 4
constexpr int kHalfKeys = kStepKeys / 2;             // keys of one P hand-over
constexpr int kSoftmaxWarps = 4;                     // one per tensor-memory lane quarter
constexpr int kLoadWarp = 4;                         // Q and K copies, then V (+ 1)
constexpr int kScoreWarp = 6;                        // S products; then the value products (+ 1)
constexpr int kThreads = 8 * 32;
constexpr int kQBuffers = 2;
constexpr int kWorkSlots = 4;                        // tiles the loaders may be ahead by
constexpr int kKStages = 4;
constexpr int kVStages = 3;
constexpr int kCtasPerSm = 2;                        // they share an SM's 512 columns
constexpr uint32_t kTmemCols = 512 / kCtasPerSm;
constexpr uint32_t kTmemP = kStepKeys;               // after S: two halves of P ...
constexpr uint32_t kPartCols = kHalfKeys / 2;        // ... of three parts, two keys per column
constexpr uint32_t kTmemO = kTmemP + 2 * 3 * kPartCols;
static_assert(kTmemO + kDim <= kTmemCols, "S, P and O fit the CTA's tensor memory");
constexpr float kRescaleLog2 = 8.f;                  // lazy max: p <= 2^8
constexpr int kSegment = 2;                          // steps whose O stays in tensor memory
// Registers a thread, once the roles are taken: 128 at launch, shared by the
// CTA's two warpgroups.
constexpr int kSoftmaxRegs = 192;
constexpr int kOtherRegs = 64;
static_assert(kSoftmaxRegs + kOtherRegs <= 2 * 128, "the launch's registers are split");
constexpr uint32_t kStepBytes = kStepKeys * kRowBytes;

template <class Job>
struct TileSmem {                           // every tile 1024-byte aligned
  uint8_t q[kQBuffers][kRows * kRowBytes];           // 2 x 16 KiB
  uint8_t k[kKStages][kStepBytes];                   // 4 x 8 KiB
  uint8_t v[kVStages][kStepBytes];                   // 3 x 8 KiB
  float4 stage[kRows][kDim / 8];                     // half of the rows' results, on their way out
  unsigned long long bar_q[kQBuffers], bar_k[kKStages];   // copies landed
  unsigned long long bar_v[kVStages];                // ... and rows no one sees cleared
  unsigned long long q_free[kQBuffers];              // read by its tile's last scores
  unsigned long long k_free[kKStages], v_free[kVStages];   // stage read by its products
  unsigned long long work_full[kWorkSlots], work_free[kWorkSlots];
  unsigned long long bar_edge;                       // V of an edge step landed
  unsigned long long bar_s, s_free;                  // S of a step computed; in registers
  unsigned long long bar_p, p_done;                  // P of a step written; multiplied
  typename Job::Work work[kWorkSlots];
  uint32_t tmem_base;
  int abort_flag;
};
template <class Job>
constexpr size_t kSmemBytes = sizeof(TileSmem<Job>) + 1024;       // + room to align the base

// What every job's parameters have.
struct TileParams {
  const int32_t* table;       // this layer's block tables [max_batch][table_stride]
  const int32_t* cu_tokens;   // [batch + 1]
  const int32_t* start_pos;   // [batch]
  float* out;                 // [total][32][64]
  int* err;
  int num_pages;
  int table_stride;
  int max_seq_len;
  int batch;
  int total_tokens;
  int window;                 // 1 .. max_seq_len
  int sinks;                  // 0 .. max_seq_len
};

// V rows that no row of the tile sees (past its last key, or between the sinks
// and the window) set to zero, so that p = 0 times them stays 0. By one warp.
template <class View>
__device__ __forceinline__ void zero_rows(uint8_t* stage, int j, const View& view, int lane) {
  #pragma unroll 4
  for (int idx = lane; idx < kStepKeys * 8; idx += 32) {
    const int row = idx >> 3;
    const int key =
        view.page((view.first_step() + j) * kStepPages + row / kPage) * kPage + row % kPage;
    if (view.dead(key))
      *reinterpret_cast<uint4*>(stage + idx * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
}

template <class Job>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) tile_attention_kernel(
    const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
    const __grid_constant__ CUtensorMap tmap_v, const typename Job::Params prm) {
  using Work = typename Job::Work;
  using View = typename Job::View;
  using Smem = TileSmem<Job>;
  static_assert(offsetof(Smem, k) % 1024 == 0 && offsetof(Smem, v) % 1024 == 0,
                "swizzled tiles start on 1024-byte boundaries");
  static_assert(kCtasPerSm * (kSmemBytes<Job> + 1024) <= 228 * 1024, "kCtasPerSm CTAs per SM");
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw + pad);

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = lane_of(tid);

  // the first sequences' lists ahead of the set-up
  typename Job::Walk walk;
  if (warp == kLoadWarp) walk.fetch(prm, lane);
  // the descriptors into the cache ahead of their first copies
  if (tid < 3)
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(
                     tid == 0 ? &tmap_q : tid == 1 ? &tmap_k : &tmap_v))
                 : "memory");
  if (warp == kLoadWarp && lane == 0) {
    for (int i = 0; i < kQBuffers; ++i) mbar_init(&sm.bar_q[i], 1);
    for (int i = 0; i < kQBuffers; ++i) mbar_init(&sm.q_free[i], 1);
    for (int i = 0; i < kKStages; ++i) mbar_init(&sm.bar_k[i], 1);
    for (int i = 0; i < kVStages; ++i) mbar_init(&sm.bar_v[i], 1);
    for (int i = 0; i < kKStages; ++i) mbar_init(&sm.k_free[i], 1);
    for (int i = 0; i < kVStages; ++i) mbar_init(&sm.v_free[i], 1);
    for (int i = 0; i < kWorkSlots; ++i) mbar_init(&sm.work_full[i], 1);
    // read by the V loader, the two issuing warps and the softmax warps
    for (int i = 0; i < kWorkSlots; ++i) mbar_init(&sm.work_free[i], 3 + kSoftmaxWarps);
    mbar_init(&sm.bar_edge, 1);
    mbar_init(&sm.bar_s, 1);
    mbar_init(&sm.s_free, kSoftmaxWarps);
    mbar_init(&sm.bar_p, kSoftmaxWarps);
    mbar_init(&sm.p_done, 1);
    sm.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0) tmem_alloc(&sm.tmem_base, kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  volatile int* abort_flag = &sm.abort_flag;
  // the kernel that joins the parts may be made ready (it waits for this one's end)
  if constexpr (Job::kParts) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // The n-th tile of this CTA, handed over by the K loader. One verdict per
  // warp: false if it never comes.
  auto wait_work = [&](int n) {
    return __all_sync(0xffffffffu,
                      mbar_wait(&sm.work_full[n % kWorkSlots], (n / kWorkSlots) & 1));
  };
  auto free_work = [&](int n) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.work_free[n % kWorkSlots]);
  };
  auto next_work = [&](int n, Work& work) {
    if (!wait_work(n)) return false;
    work = sm.work[n % kWorkSlots];
    free_work(n);
    return true;
  };
  auto give_up = [&]() {
    *abort_flag = 1;
    set_error(prm.err, PKV_DEV_ERR_TIMEOUT);
  };

  if (warp >= kLoadWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp < kScoreWarp) {
      // ---------------------------------------------------------- copy engine
      // Lanes 0..3 copy a step's 4 pages in one instruction once lane 0 saw
      // the stage free. A page that is not there is copied from past the
      // pool's end: zeros.
      // lane 4 s + e holds the e-th page of the s-th of 8 steps; the next 8
      // steps' are fetched while these are in use
      // V only: a step with rows that no one sees lands on a barrier of its
      // own; the loader clears those rows and then completes the stage.
      int edges = 0;
      // this lane's page of 8 steps from step j on: past the pool's end if there is
      // none, or an invalid one (bad)
      auto page_id = [&](const View& view, int b, int j, bool& bad) {
        int id = prm.num_pages;
        const int i = (view.first_step() + j) * kStepPages + lane;
        if (view.has_page(i)) {
          id = __ldg(prm.table + static_cast<size_t>(b) * prm.table_stride + view.page(i));
          if (id < 0 || id >= prm.num_pages) {
            id = prm.num_pages;
            bad = true;
          }
        }
        return id;
      };
      auto load_tile = [&](const View& view, const Work& work, int ids, const CUtensorMap* map,
                           uint8_t* ring, unsigned long long* full, unsigned long long* free,
                           auto& at, int& issued, int stages, bool is_v) {
        bool bad;
        int ids_next = page_id(view, work.b, 8, bad);
        for (int j = 0; j < view.n_steps; ++j) {
          if ((j & 7) == 0 && j > 0) {
            ids = ids_next;
            ids_next = page_id(view, work.b, j + 8, bad);
          }
          const int page = __shfl_sync(0xffffffffu, ids, (j & 7) * kStepPages + lane % kStepPages);
          const bool edge = is_v && view.has_dead(j);
          unsigned long long* landed = edge ? &sm.bar_edge : &full[at.stage];
          uint8_t* to = ring + at.stage * kStepBytes;
          bool good = true;
          if (lane == 0) {
            good = *abort_flag == 0;
            if (good && issued >= stages) good = mbar_wait(&free[at.stage], at.round ^ 1u);
            if (good) mbar_arrive_expect_tx(landed, kStepBytes);
          }
          if (!__shfl_sync(0xffffffffu, good ? 1 : 0, 0)) return false;
          if (lane < kStepPages)
            tma_load_3d(to + lane * kPage * kRowBytes, map, 0, work.g * kPage, page, landed);
          __syncwarp();
          if (edge) {
            if (!__all_sync(0xffffffffu, mbar_wait(&sm.bar_edge, edges & 1))) return false;
            ++edges;
            zero_rows(to, j, view, lane);
            __syncwarp();
            if (lane == 0) mbar_arrive(&full[at.stage]);
          }
          at.next();
          ++issued;
        }
        return true;
      };
      // every copy issued lands before the CTA frees its memory (bounded waits)
      auto drain = [&](unsigned long long* full, int issued, int stages) {
        if (lane == 0)
          for (int s = 0; s < stages; ++s) {
            const int uses = (issued - s + stages - 1) / stages;
            if (uses > 0) mbar_wait(&full[s], (uses - 1) & 1);
          }
      };
      bool ok = true;
      int issued = 0;
      if (warp == kLoadWarp) {
        // K, Q and the tiles themselves, in the order of the job's Walk
        RingAt<kKStages> at;
        int n = 0;                              // tiles handed over
        int q_loads = 0;
        auto hand_over = [&](const Work& work) {
          const int slot = n % kWorkSlots;
          bool good = true;
          if (lane == 0) {
            if (n >= kWorkSlots)
              good = mbar_wait(&sm.work_free[slot], (n / kWorkSlots - 1) & 1);
            if (good) {
              sm.work[slot] = work;
              mbar_arrive(&sm.work_full[slot]);
            }
          }
          return __shfl_sync(0xffffffffu, good ? 1 : 0, 0) != 0;
        };
        for (bool first = true;; first = false) {
          // Drawn: the first tile is this CTA's own (nothing to wait for); each other
          // one is taken once the last one's copies are all on their way, a
          // few steps before they are used up: any earlier, and a CTA would
          // hold a tile back from those that run out of work.
          unsigned long long index = blockIdx.x;
          if constexpr (Job::kDrawn) {
            if (!first) {
              if (lane == 0) index = gridDim.x + atomicAdd(prm.next_tile, 1ull);
              index = __shfl_sync(0xffffffffu, index, 0);
            }
          }
          Work work;
          if (!walk.next(index, prm, lane, work)) break;
          const View view(work, prm);
          const int buffer = n % kQBuffers;
          bool bad = false;
          const int ids = page_id(view, work.b, 0, bad);
          if (lane == 0) {
            if (n >= kQBuffers) ok = mbar_wait(&sm.q_free[buffer], (n / kQBuffers - 1) & 1);
            if (ok) {
              mbar_arrive_expect_tx(&sm.bar_q[buffer], kRows * kRowBytes);
              tma_load_3d(sm.q[buffer], &tmap_q, 0, work.g * kGroup, work.row, &sm.bar_q[buffer]);
            }
          }
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
          if (!ok) break;
          ++q_loads;
          // invalid ids among the pages that count
          #pragma unroll 4
          for (int j = 8; j < view.n_steps; j += 8) page_id(view, work.b, j, bad);
          work.bad_page = __any_sync(0xffffffffu, bad);
          if (work.bad_page && lane == 0) set_error(prm.err, PKV_DEV_ERR_PAGE);
          ok = hand_over(work);
          if (!ok) break;
          ++n;
          ok = load_tile(view, work, ids, &tmap_k, sm.k[0], sm.bar_k, sm.k_free, at, issued,
                         kKStages, false);
          if (!ok) break;
        }
        if (ok) {
          Work end = {};
          ok = hand_over(end);
        }
        if (!ok && lane == 0) give_up();
        drain(sm.bar_k, issued, kKStages);
        drain(sm.bar_q, q_loads, kQBuffers);
        // the last CTA to stop drawing leaves the counters at zero
        if constexpr (Job::kDrawn) {
          if (lane == 0) {
            __threadfence();
            if (atomicAdd(prm.ctas_done, 1u) == gridDim.x - 1) {
              *prm.next_tile = 0;
              *prm.ctas_done = 0;
            }
          }
        }
      } else {
        RingAt<kVStages> at;
        for (int n = 0;; ++n) {
          Work work;
          ok = next_work(n, work);
          if (!ok || work.count == 0) break;
          const View view(work, prm);
          bool bad;
          ok = load_tile(view, work, page_id(view, work.b, 0, bad), &tmap_v, sm.v[0], sm.bar_v,
                         sm.v_free, at, issued, kVStages, true);
          if (!ok) break;
        }
        if (!ok && lane == 0) give_up();
        drain(sm.bar_v, issued, kVStages);
      }
    } else {
      // ---------------------------------------------------------- tensor cores
      // One issuing warp for the scores and one for the values.
      bool ok = true;
      uint32_t steps = 0;                       // of all tiles so far
      if (warp == kScoreWarp) {
        const uint32_t idesc_s = instr_desc(kRows, kStepKeys, false);
        RingAt<kKStages> at;
        for (int n = 0; ok; ++n) {
          Work work;
          ok = next_work(n, work);
          if (!ok || work.count == 0) break;
          const View view(work, prm);
          const int buffer = n % kQBuffers;
          const uint64_t q_desc = smem_desc_sw128(smem_u32(sm.q[buffer]), 16, 1024);
          ok = __all_sync(0xffffffffu, mbar_wait(&sm.bar_q[buffer], (n / kQBuffers) & 1));
          for (int j = 0; ok && j < view.n_steps; ++j) {
            // S = Q K^T, once K landed and the last step's S is in registers
            const bool ready = *abort_flag == 0 && mbar_wait(&sm.bar_k[at.stage], at.round) &&
                               (steps == 0 || mbar_wait(&sm.s_free, (steps - 1) & 1));
            if (!__all_sync(0xffffffffu, ready)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t k_desc = smem_desc_sw128(smem_u32(sm.k[at.stage]), 16, 1024);
            if (elect_one()) {
              #pragma unroll
              for (int kk = 0; kk < kDim / 16; ++kk)
                mma_bf16(tmem, q_desc + kk * 2, k_desc + kk * 2, idesc_s, kk > 0);
              mma_commit(&sm.bar_s);
              mma_commit(&sm.k_free[at.stage]);
              if (j == view.n_steps - 1) mma_commit(&sm.q_free[buffer]);
            }
            __syncwarp();
            at.next();
            ++steps;
          }
        }
        // every product issued completes before the CTA frees its memory
        if (steps > 0) mbar_wait(&sm.bar_s, (steps - 1) & 1);
      } else {
        const uint32_t idesc_o = instr_desc(kRows, kDim, true);
        RingAt<kVStages> at;
        for (int n = 0; ok; ++n) {
          Work work;
          ok = next_work(n, work);
          if (!ok || work.count == 0) break;
          const View view(work, prm);
          for (int j = 0; j < view.n_steps; ++j) {
            // O += P V: 16 keys per product, P's three parts kPartCols columns
            // apart in each half
            if (!__all_sync(0xffffffffu, *abort_flag == 0 &&
                                             mbar_wait(&sm.bar_v[at.stage], at.round) &&
                                             mbar_wait(&sm.bar_p, steps & 1))) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t v_desc = smem_desc_sw128(smem_u32(sm.v[at.stage]), 8192, 1024);
            if (elect_one()) {
              #pragma unroll
              for (int kk = 0; kk < kStepKeys / 16; ++kk) {
                #pragma unroll
                for (int part = 0; part < 3; ++part)
                  mma_bf16_tmem_a(tmem + kTmemO,
                                  tmem + kTmemP + (3 * (kk / 2) + part) * kPartCols + (kk % 2) * 8,
                                  v_desc + kk * (16 * kRowBytes >> 4), idesc_o,
                                  (j % kSegment > 0 || kk > 0 || part > 0) ? 1u : 0u);
              }
              mma_commit(&sm.p_done);
              mma_commit(&sm.v_free[at.stage]);
            }
            __syncwarp();
            at.next();
            ++steps;
          }
        }
        if (steps > 0) mbar_wait(&sm.p_done, (steps - 1) & 1);
      }
      if (!ok && lane == 0) give_up();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ------------------------------------------------------------ softmax warps
    const int r = tid;                                  // its MMA row = tensor-memory lane
    const float c = 1.4426950408889634f * 0.125f;       // log2(e) / sqrt(64)
    const uint32_t lane_addr = static_cast<uint32_t>(warp * 32) << 16;
    bool ok = true;
    uint32_t steps = 0;                                 // of all tiles so far
    // The tile stays in its shared slot until its results are out: what only edge
    // steps and the end need of it is read there, not held in registers.
    ok = wait_work(0);
    for (int n = 0; ok && sm.work[n % kWorkSlots].count > 0; ++n) {
      const Work& work = sm.work[n % kWorkSlots];
      const View view(work, prm);
      const int n_steps = view.n_steps;
      const bool any_bad_page = work.bad_page != 0;
      float m_run = -INFINITY, l_run = 0.f;
      float m_sum = -INFINITY;                          // the max that o_sum is taken against
      float2 o_sum[kDim / 2];                           // earlier segments' O
      #pragma unroll
      for (int d = 0; d < kDim / 2; ++d) o_sum[d] = make_float2(0.f, 0.f);
      const int plain_from = any_bad_page ? n_steps : view.plain_from;
      const int plain_count = any_bad_page ? 0 : max(view.plain_to - view.plain_from, 0);
      // a warp whose rows are all past the end only keeps step with the others
      const bool idle = Job::kFewRows && warp * 8 >= work.count;
      bool s_done = false;                              // the next step's S is known to be there
      // what a step's largest score may not pass without a closer look: m_run and what p
      // may grow by, or less where m_run is huge (device_common.cuh)
      float limit = -INFINITY;
      int segment = 0;                                  // j % kSegment, kSegment before a join
      for (int j = 0; j < n_steps; ++j, ++steps) {
        if (!wait_phase_after(s_done, &sm.bar_s, steps & 1, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (idle) {
          // P's turn comes once the last step's product is done: an arrival any
          // earlier would count for that one
          tc_fence_before();
          __syncwarp();
          arrive_lane0(&sm.s_free, lane);
          if (steps > 0 && !wait_phase(&sm.p_done, (steps - 1) & 1, abort_flag)) {
            ok = false;
            break;
          }
          arrive_lane0(&sm.bar_p, lane);
          continue;
        }
        uint32_t sv[64];                                   // the row's 64 keys of the step
        tmem_ld64(tmem + lane_addr, sv);
        tc_fence_before();
        __syncwarp();
        arrive_lane0(&sm.s_free, lane);
        const bool plain =
            static_cast<unsigned>(j - plain_from) < static_cast<unsigned>(plain_count);
        if (rarely(!plain)) {
          // bit i of seen[w]: key 32 w + i of the step is visible (16 bits a
          // page; one word test and one select per key: the code of an edge step
          // is fetched anew each time, and a compare per condition and key made
          // it 1,600 cycles)
          const View view(work, prm);
          // the row's token of the tile is r / 4, its head r % 4; rows past the end
          // mirror the last one
          const typename Job::Row row(work, prm, min(r >> 2, work.count - 1));
          uint32_t seen[2] = {0u, 0u};
          #pragma unroll
          for (int e = 0; e < kStepPages; ++e) {
            const int i = (view.first_step() + j) * kStepPages + e;
            const int base = view.page(i) * kPage;
            uint32_t bits = row.seen(view, base);
            if (any_bad_page && view.has_page(i)) {
              const int id = __ldg(prm.table + static_cast<size_t>(work.b) * prm.table_stride +
                                   base / kPage);
              if (id < 0 || id >= prm.num_pages) bits = 0u;
            }
            seen[e / 2] |= (bits & 0xffffu) << (16 * (e % 2));
          }
          #pragma unroll
          for (int i = 0; i < kStepKeys; ++i)
            if (!((seen[i / 32] >> (i % 32)) & 1u)) sv[i] = __float_as_uint(-INFINITY);
        }
        float mx[4];
        #pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = max3(sv[e], sv[e + 4], sv[e + 8]);
        #pragma unroll
        for (int i = 12; i < 60; i += 8) {
          #pragma unroll
          for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], sv[i + e], sv[i + e + 4]);
        }
        #pragma unroll
        for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], __uint_as_float(sv[60 + e]));
        const float m_step = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
        // a row that grew its max rescales its O (P(j) V(j) cannot start before
        // this thread hands over P(j))
        float mu = m_run;
        if (rarely(__any_sync(0xffffffffu, m_step > limit))) {   // not while nothing was visible
          float alpha = 1.f;
          if (m_step > m_run + kRescaleLog2) {
            alpha = fast_exp2(m_run - m_step);
            m_run = m_step;
            l_run *= alpha;
            limit = is_huge(m_run) ? -FLT_MAX : m_run + kRescaleLog2;
          }
          mu = m_run;
          if (rarely(is_huge(mu))) {
            // the differences themselves, in the scores' unit (a factor that is not known
            // to the compiler, in place of c, costs every step 3 %)
            #pragma unroll
            for (int i = 0; i < kStepKeys; ++i)
              sv[i] = __float_as_uint(less(__uint_as_float(sv[i]), c, mu) * (1.f / c));
            mu = 0.f;
          }
          if (j > 0) {
            if (!wait_phase(&sm.p_done, (steps - 1) & 1, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
            #pragma unroll
            for (int dq = 0; dq < 4; ++dq) {
              uint32_t ov[16];
              tmem_ld16(tmem + lane_addr + kTmemO + dq * 16, ov);
              #pragma unroll
              for (int d = 0; d < 16; ++d)
                ov[d] = __float_as_uint(__uint_as_float(ov[d]) * alpha);
              tmem_st16(tmem + lane_addr + kTmemO + dq * 16, ov);
            }
            tmem_wait_st();
          }
        }
        // The probabilities, their sum and their three BF16 parts, 32 keys at a
        // time; into tensor memory once the last step's product has read its P.
        const bool p_free = phase_done(&sm.p_done, (steps - 1) & 1);
        const float2 c2 = make_float2(c, c);
        if (mu == -INFINITY) mu = 0.f;
        float2 acc[2];
        auto half_of_p = [&](int h, uint32_t (&hi)[16], uint32_t (&mid)[16], uint32_t (&lo)[16]) {
          const float2 nm2 = make_float2(-mu, -mu);
          #pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const int k = h * 32 + i;
            const float2 x = __ffma2_rn(
                make_float2(__uint_as_float(sv[k]), __uint_as_float(sv[k + 1])), c2, nm2);
            const float2 pp = make_float2(fast_exp2(x.x), fast_exp2(x.y));
            acc[(i >> 1) & 1] = __fadd2_rn(acc[(i >> 1) & 1], pp);
            split3(pp.x, pp.y, hi[i / 2], mid[i / 2], lo[i / 2]);
          }
        };
        auto store_half = [&](int h, const uint32_t (&hi)[16], const uint32_t (&mid)[16],
                              const uint32_t (&lo)[16]) {
          const uint32_t p_half = tmem + lane_addr + kTmemP + 3 * h * kPartCols;
          tmem_st16(p_half, hi);
          tmem_st16(p_half + kPartCols, mid);
          tmem_st16(p_half + 2 * kPartCols, lo);
        };
        {
          uint32_t hi[16], mid[16], lo[16];
          acc[0] = acc[1] = make_float2(0.f, 0.f);
          half_of_p(0, hi, mid, lo);
          if (steps > 0) {
            if (!wait_phase_after(p_free, &sm.p_done, (steps - 1) & 1, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
          }
          store_half(0, hi, mid, lo);
        }
        // after a segment O joins the sum; the next product, P(j) V(j), starts
        // from zero
        if (segment == kSegment) {
          const float beta = m_sum == -INFINITY ? 0.f : fast_exp2(m_sum - m_run);
          const float2 b2 = make_float2(beta, beta);
          #pragma unroll
          for (int dh = 0; dh < 2; ++dh) {
            uint32_t ov[32];
            tmem_ld32(tmem + lane_addr + kTmemO + dh * 32, ov);
            #pragma unroll
            for (int d = 0; d < 16; ++d)
              o_sum[dh * 16 + d] = __ffma2_rn(
                  o_sum[dh * 16 + d], b2,
                  make_float2(__uint_as_float(ov[2 * d]), __uint_as_float(ov[2 * d + 1])));
          }
          m_sum = m_run;
          segment = 0;
        }
        ++segment;
        {
          uint32_t hi[16], mid[16], lo[16];
          half_of_p(1, hi, mid, lo);
          store_half(1, hi, mid, lo);
        }
        s_done = phase_done(&sm.bar_s, (steps + 1) & 1);
        const float2 a = __fadd2_rn(acc[0], acc[1]);
        l_run += a.x + a.y;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        arrive_lane0(&sm.bar_p, lane);
      }
      // the next tile is looked up while the last product runs
      if (!ok || !wait_work(n + 1) || !wait_phase(&sm.p_done, (steps - 1) & 1, abort_flag)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const bool whole = Job::is_whole(work);
      const float inv = !whole ? 1.f : l_run > 0.f ? 1.f / l_run : 0.f;
      const float beta = m_sum == -INFINITY ? 0.f : fast_exp2(m_sum - m_run);
      // Half a row at a time through shared memory, so that 8 lanes write 128
      // contiguous bytes (a row per lane writes 32 half sectors at once: the
      // four warps' stores then took 2,000 cycles a tile). Row r's chunk c is
      // kept at c ^ (r % 8), different banks for 8 rows.
      float4* rows_out = reinterpret_cast<float4*>(
          prm.out + ((static_cast<size_t>(work.row) + warp * 8) * kHq + work.g * kGroup) * kDim);
      if constexpr (Job::kParts) {
        if (!whole) {
          if (r < work.count * kGroup) Job::put_sums(work, prm, r, m_run, l_run);
          rows_out = Job::part(work, prm) + warp * 32 * (kDim / 4);
        }
      }
      #pragma unroll
      for (int dh = 0; dh < 2; ++dh) {
        uint32_t ov[32];
        tmem_ld32(tmem + lane_addr + kTmemO + dh * 32, ov);
        #pragma unroll
        for (int d = 0; d < 8; ++d) {
          const float2 was0 = o_sum[dh * 16 + 2 * d], was1 = o_sum[dh * 16 + 2 * d + 1];
          sm.stage[r][d ^ (r & 7)] =
              make_float4(fmaf(was0.x, beta, __uint_as_float(ov[4 * d])) * inv,
                          fmaf(was0.y, beta, __uint_as_float(ov[4 * d + 1])) * inv,
                          fmaf(was1.x, beta, __uint_as_float(ov[4 * d + 2])) * inv,
                          fmaf(was1.y, beta, __uint_as_float(ov[4 * d + 3])) * inv);
        }
        __syncwarp();
        #pragma unroll
        for (int e = 0; e < 8; ++e) {           // token e of the warp's 8, its head lane / 8
          const int row = 4 * e + (lane >> 3);
          const float4 x = sm.stage[warp * 32 + row][(lane & 7) ^ (row & 7)];
          if (warp * 8 + e < work.count)
            rows_out[(e * (whole ? kHq : kGroup) + (lane >> 3)) * (kDim / 4) + dh * 8 +
                     (lane & 7)] = x;
        }
        __syncwarp();
      }
      // O is in registers before the next tile's first P is handed over
      tc_fence_before();
      free_work(n);
    }
    if (!ok) give_up();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ---------------------------------------------------------------- host
template <class Job>
bool set_smem_attribute(int device) {
  constexpr int kMaxDevices = 64;
  static std::mutex lock;
  static bool done[kMaxDevices] = {};
  if (device < 0 || device >= kMaxDevices) return false;
  std::lock_guard<std::mutex> guard(lock);
  if (!done[device]) {
    if (cudaFuncSetAttribute(tile_attention_kernel<Job>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSmemBytes<Job>)) != cudaSuccess)
      return false;
    done[device] = true;
  }
  return true;
}

}  // namespace pkv_tiles

#endif  // PKV_PREFILL_TILES_CUH
