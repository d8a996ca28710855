// Windowed prefill attention over the paged KV cache for GB300 (sm_103a): a
// chunk's tokens attend behind a sliding window, with sinks (declared in
// include/pkv_window.h).
//
// out_i = sum_t p_it V_t / sum_t p_it, p_it = 2^(q_i.K_t log2(e) / 8 - m_i), over
// the tokens visible from position p_i: one pass per 32-token query tile
// with a running maximum m_i and sum per row.
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
// What bounds it: the softmax warps, two per scheduler, and of their time less
// the arithmetic (maximum, exponentials, sums, the split into three terms: 1,200
// cycles for two warps by itself, measured alone) than what a warp waits for in
// turn: its barriers, tensor memory, votes and instructions. A step of two CTAs
// takes about 2,000 cycles, against 1,024 of the tensor pipe (16 products of 32
// cycles each); a tile's start and end cost it some 4,000 more. The products are
// never waited for: every barrier of theirs is complete when it is first looked
// at. Two 4,096-token chunks behind a 4,096-token window: 467 us (591 TFLOP/s of
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
// the last product; 467 with no tile drawn that does not exist. The second: 159
// us up to the page ids, one CTA per tile; 134 with tiles drawn by resident CTAs,
// V cleared by its loader and results written through shared memory; 122 with
// word masks and a first tile that needs no draw; 112, and 111 with the last of
// the above, at the end. Slower: two threads per row (16 softmax warps per SM, by
// 10 %), and the first half of P taken against the running maximum before the
// step's own is known, done again for a row that outgrew it (by 12 %).

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

// One tile of work, as the K loader hands it to the other warps; count 0: the end.
struct TileWork {
  int b;          // sequence
  int g;          // KV head
  int row;        // its first row of q and out
  int p_first;    // position of that row
  int count;      // rows, 1 .. 32
  int bad_page;   // some page that counts has an invalid id
};

struct WindowPrefillSmem {                           // every tile 1024-byte aligned
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
  TileWork work[kWorkSlots];
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(offsetof(WindowPrefillSmem, k) % 1024 == 0 &&
                  offsetof(WindowPrefillSmem, v) % 1024 == 0,
              "swizzled tiles start on 1024-byte boundaries");
constexpr size_t kSmemBytes = sizeof(WindowPrefillSmem) + 1024;   // + room to align the base
static_assert(kCtasPerSm * (kSmemBytes + 1024) <= 228 * 1024, "kCtasPerSm CTAs per SM");

struct WindowPrefillParams {
  const int32_t* table;       // this layer's block tables [max_batch][table_stride]
  const int32_t* cu_tokens;   // [batch + 1]
  const int32_t* start_pos;   // [batch]
  float* out;                 // [total][32][64]
  int* err;
  unsigned long long* next_tile;   // shared by the launch's CTAs; zero before and after it
  unsigned int* ctas_done;         // the same
  int num_pages;
  int table_stride;
  int max_seq_len;
  int batch;
  int tiles_max;              // tiles per sequence the launch covers
  int total_tokens;
  int window;                 // 1 .. max_seq_len
  int sinks;                  // 0 .. max_seq_len
};

// The lowest n bits of 32 (n clamped to 0 .. 32).
__device__ __forceinline__ uint32_t low_bits32(int n) {
  return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u;
}

// Whether `x` holds, which is rare: the code under it is placed out of the
// step loop's way.
__device__ __forceinline__ bool rarely(bool x) { return __builtin_expect(x, 0); }

// The rest of a bounded wait on an mbarrier phase that has not come yet; gives
// up when the CTA does.
__device__ __noinline__ bool wait_longer(unsigned long long* bar, uint32_t parity,
                                         volatile int* abort_flag) {
  const long long start = clock64();
  while (!mbar_try_wait(bar, parity))
    if (*abort_flag || clock64() - start > kWaitCycles) return false;
  return true;
}

// One verdict per warp (what follows is warp-wide).
__device__ __forceinline__ bool wait_phase(unsigned long long* bar, uint32_t parity,
                                           volatile int* abort_flag) {
  bool done = mbar_try_wait(bar, parity);
  if (!done) done = wait_longer(bar, parity, abort_flag);
  return __all_sync(0xffffffffu, done);
}

// Whether a phase is complete, without waiting for it.
__device__ __forceinline__ bool phase_done(unsigned long long* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return done != 0;
}

// wait_phase after an early look at the phase: the barrier's own latency is
// paid only where the look came too soon.
__device__ __forceinline__ bool wait_phase_after(bool done, unsigned long long* bar,
                                                 uint32_t parity, volatile int* abort_flag) {
  if (__all_sync(0xffffffffu, done)) return true;
  return wait_phase(bar, parity, abort_flag);
}

// Lane 0's arrival, predicated instead of branched around.
__device__ __forceinline__ void arrive_lane0(unsigned long long* bar, int lane) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.eq.s32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_u32(bar)), "r"(lane)
      : "memory");
}

// One lane of a converged warp, always the same. The issuing warps run their
// loops whole and only the tcgen05 instructions under this predicate, so the
// operands stay in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// The largest of three (the last two given as bits).
__device__ __forceinline__ float max3(float a, uint32_t b, uint32_t c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;"
      : "=f"(d)
      : "f"(a), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
  return d;
}
__device__ __forceinline__ float max3(uint32_t a, uint32_t b, uint32_t c) {
  return max3(__uint_as_float(a), b, c);
}

// 16 consecutive columns, complete on return.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

// 64 consecutive 32-bit columns of this thread's tensor-memory lane.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&r)[64]) {
  #pragma unroll
  for (int h = 0; h < 4; ++h)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15}, [%16];"
        : "=r"(r[16 * h]), "=r"(r[16 * h + 1]), "=r"(r[16 * h + 2]), "=r"(r[16 * h + 3]),
          "=r"(r[16 * h + 4]), "=r"(r[16 * h + 5]), "=r"(r[16 * h + 6]), "=r"(r[16 * h + 7]),
          "=r"(r[16 * h + 8]), "=r"(r[16 * h + 9]), "=r"(r[16 * h + 10]), "=r"(r[16 * h + 11]),
          "=r"(r[16 * h + 12]), "=r"(r[16 * h + 13]), "=r"(r[16 * h + 14]), "=r"(r[16 * h + 15])
        : "r"(taddr + 16 * h));
  // the registers are written once the wait returns: it takes them as operands
  #pragma unroll
  for (int h = 0; h < 4; ++h) {
    uint32_t* x = r + 16 * h;
    if (h == 0)
      asm volatile("tcgen05.wait::ld.sync.aligned;"
                   : "+r"(x[0]), "+r"(x[1]), "+r"(x[2]), "+r"(x[3]), "+r"(x[4]), "+r"(x[5]),
                     "+r"(x[6]), "+r"(x[7]), "+r"(x[8]), "+r"(x[9]), "+r"(x[10]), "+r"(x[11]),
                     "+r"(x[12]), "+r"(x[13]), "+r"(x[14]), "+r"(x[15])::"memory");
    else
      asm volatile("" : "+r"(x[0]), "+r"(x[1]), "+r"(x[2]), "+r"(x[3]), "+r"(x[4]), "+r"(x[5]),
                        "+r"(x[6]), "+r"(x[7]), "+r"(x[8]), "+r"(x[9]), "+r"(x[10]), "+r"(x[11]),
                        "+r"(x[12]), "+r"(x[13]), "+r"(x[14]), "+r"(x[15])::"memory");
  }
}

// What the tile (and each of its steps) sees of the sequence.
struct TileView {
  int p_first;           // position of the tile's first token
  int n_keys;            // position of its last token + 1
  int lo;                // first key inside some row's window
  int sinks;
  int sink_pages;        // pages of sinks before the window's
  int win_page;          // the window's first page
  int n_pages;
  int n_steps;
  int plain_from, plain_to;   // steps whose keys every row sees

  __device__ TileView(int first, int count, int window, int sinks_) {
    p_first = first;
    n_keys = first + count;
    lo = max(first - window + 1, 0);
    sinks = sinks_;
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

// V rows that no row of the tile sees (past its last key, or between the sinks
// and the window) set to zero, so that p = 0 times them stays 0. By one warp.
__device__ __forceinline__ void zero_rows(uint8_t* stage, int j, const TileView& view,
                                          int lane) {
  #pragma unroll 4
  for (int idx = lane; idx < kStepKeys * 8; idx += 32) {
    const int row = idx >> 3;
    const int key = view.page(j * kStepPages + row / kPage) * kPage + row % kPage;
    if (key >= view.n_keys || (key >= view.sinks && key < view.lo))
      *reinterpret_cast<uint4*>(stage + idx * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
}

// A step's place in a ring of stages, and how often the ring has gone round.
template <int kStages>
struct RingAt {
  int stage = 0;
  uint32_t round = 0;      // parity of the phase that the stage's barriers complete next
  __device__ void next() {
    if (++stage == kStages) {
      stage = 0;
      round ^= 1u;
    }
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
struct TileWalk {
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

__global__ void __launch_bounds__(kThreads, kCtasPerSm) window_prefill_kernel(
    const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
    const __grid_constant__ CUtensorMap tmap_v, const WindowPrefillParams prm) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t pad = (1024u - (smem_u32(smem_raw) & 1023u)) & 1023u;
  WindowPrefillSmem& sm = *reinterpret_cast<WindowPrefillSmem*>(smem_raw + pad);

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = lane_of(tid);

  // the first sequences' lists ahead of the set-up
  TileWalk walk;
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

  // The n-th tile of this CTA, handed over by the K loader. One verdict per
  // warp: false if it never comes.
  auto next_work = [&](int n, TileWork& work) {
    const int slot = n % kWorkSlots;
    if (!__all_sync(0xffffffffu, mbar_wait(&sm.work_full[slot], (n / kWorkSlots) & 1)))
      return false;
    work = sm.work[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.work_free[slot]);
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
      auto load_tile = [&](const TileView& view, const TileWork& work, const CUtensorMap* map,
                           uint8_t* ring, unsigned long long* full, unsigned long long* free,
                           auto& at, int& issued, int stages, bool is_v) {
        const int32_t* trow = prm.table + static_cast<size_t>(work.b) * prm.table_stride;
        auto page_of = [&](int j, int e) {      // the e-th page of step j, past the end if none
          int id = prm.num_pages;
          const int i = j * kStepPages + e;
          if (i < view.n_pages) {
            id = __ldg(trow + view.page(i));
            if (id < 0 || id >= prm.num_pages) id = prm.num_pages;
          }
          return id;
        };
        int ids = page_of(lane / kStepPages, lane % kStepPages);
        int ids_next = page_of(8 + lane / kStepPages, lane % kStepPages);
        for (int j = 0; j < view.n_steps; ++j) {
          if ((j & 7) == 0 && j > 0) {
            ids = ids_next;
            ids_next = page_of(j + 8 + lane / kStepPages, lane % kStepPages);
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
        // K, Q and the tiles themselves: the launch's CTAs draw them from one
        // counter, in TileWalk's order, the 8 KV heads of a tile in a row
        RingAt<kKStages> at;
        int n = 0;                              // tiles handed over
        int q_loads = 0;
        auto hand_over = [&](const TileWork& work) {
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
          // The first tile is this CTA's own (nothing to wait for); each other
          // one is drawn once the last one's copies are all on their way, a
          // few steps before they are used up: any earlier, and a CTA would
          // hold a tile back from those that run out of work.
          unsigned long long index = blockIdx.x;
          if (!first) {
            if (lane == 0) index = gridDim.x + atomicAdd(prm.next_tile, 1ull);
            index = __shfl_sync(0xffffffffu, index, 0);
          }
          const int g = static_cast<int>(index % kHkv);
          int b, tile, row0, rows, start;
          if (!walk.find(static_cast<uint32_t>(index / kHkv), prm, lane, b, tile, row0, rows,
                         start))
            break;
          TileWork work;
          work.b = b;
          work.g = g;
          work.row = row0 + tile * kTileTokens;
          work.p_first = start + tile * kTileTokens;
          work.count = min(kTileTokens, rows - tile * kTileTokens);
          const TileView view(work.p_first, work.count, prm.window, prm.sinks);
          const int32_t* trow = prm.table + static_cast<size_t>(b) * prm.table_stride;
          const int buffer = n % kQBuffers;
          if (lane == 0) {
            if (n >= kQBuffers) ok = mbar_wait(&sm.q_free[buffer], (n / kQBuffers - 1) & 1);
            if (ok) {
              mbar_arrive_expect_tx(&sm.bar_q[buffer], kRows * kRowBytes);
              tma_load_3d(sm.q[buffer], &tmap_q, 0, g * kGroup, work.row, &sm.bar_q[buffer]);
            }
          }
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
          if (!ok) break;
          ++q_loads;
          // invalid ids among the pages that count
          bool bad = false;
          for (int i = lane; i < view.n_pages; i += 32) {
            const int id = __ldg(trow + view.page(i));
            bad |= id < 0 || id >= prm.num_pages;
          }
          work.bad_page = __any_sync(0xffffffffu, bad);
          if (work.bad_page && lane == 0) set_error(prm.err, PKV_DEV_ERR_PAGE);
          ok = hand_over(work);
          if (!ok) break;
          ++n;
          ok = load_tile(view, work, &tmap_k, sm.k[0], sm.bar_k, sm.k_free, at, issued, kKStages,
                         false);
          if (!ok) break;
        }
        if (ok) {
          TileWork end = {};
          ok = hand_over(end);
        }
        if (!ok && lane == 0) give_up();
        drain(sm.bar_k, issued, kKStages);
        drain(sm.bar_q, q_loads, kQBuffers);
        // the last CTA to stop drawing leaves the counters at zero
        if (lane == 0) {
          __threadfence();
          if (atomicAdd(prm.ctas_done, 1u) == gridDim.x - 1) {
            *prm.next_tile = 0;
            *prm.ctas_done = 0;
          }
        }
      } else {
        RingAt<kVStages> at;
        for (int n = 0;; ++n) {
          TileWork work;
          ok = next_work(n, work);
          if (!ok || work.count == 0) break;
          const TileView view(work.p_first, work.count, prm.window, prm.sinks);
          ok = load_tile(view, work, &tmap_v, sm.v[0], sm.bar_v, sm.v_free, at, issued, kVStages,
                         true);
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
          TileWork work;
          ok = next_work(n, work);
          if (!ok || work.count == 0) break;
          const TileView view(work.p_first, work.count, prm.window, prm.sinks);
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
          TileWork work;
          ok = next_work(n, work);
          if (!ok || work.count == 0) break;
          const TileView view(work.p_first, work.count, prm.window, prm.sinks);
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
    const int tok = r >> 2;                             // token of the tile, head r & 3
    const float c = 1.4426950408889634f * 0.125f;       // log2(e) / sqrt(64)
    const uint32_t lane_addr = static_cast<uint32_t>(warp * 32) << 16;
    bool ok = true;
    uint32_t steps = 0;                                 // of all tiles so far
    TileWork work;
    ok = next_work(0, work);
    for (int n = 1; ok && work.count > 0; ++n) {
      const TileView view(work.p_first, work.count, prm.window, prm.sinks);
      const int n_steps = view.n_steps;
      const bool any_bad_page = work.bad_page != 0;
      const int pos = view.p_first + min(tok, work.count - 1);  // rows past the end mirror the last
      float m_run = -INFINITY, l_run = 0.f;
      float m_sum = -INFINITY;                          // the max that o_sum is taken against
      float2 o_sum[kDim / 2];                           // earlier segments' O
      #pragma unroll
      for (int d = 0; d < kDim / 2; ++d) o_sum[d] = make_float2(0.f, 0.f);
      const int plain_from = any_bad_page ? n_steps : view.plain_from;
      const int plain_count = any_bad_page ? 0 : max(view.plain_to - view.plain_from, 0);
      bool s_done = false;                              // the next step's S is known to be there
      int segment = 0;                                  // j % kSegment, kSegment before a join
      for (int j = 0; j < n_steps; ++j, ++steps) {
        if (!wait_phase_after(s_done, &sm.bar_s, steps & 1, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
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
          uint32_t seen[2] = {0u, 0u};
          #pragma unroll
          for (int e = 0; e < kStepPages; ++e) {
            const int base = view.page(j * kStepPages + e) * kPage;
            uint32_t bits =
                low_bits32(pos + 1 - base) &
                (low_bits32(view.sinks - base) | ~low_bits32(pos - prm.window + 1 - base));
            if (any_bad_page && j * kStepPages + e < view.n_pages) {
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
        const bool grow = m_step > m_run + kRescaleLog2;   // false while nothing was visible
        if (rarely(__any_sync(0xffffffffu, grow))) {
          float alpha = 1.f;
          if (grow) {
            alpha = fast_exp2(m_run - m_step);
            m_run = m_step;
            l_run *= alpha;
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
        float2 acc[2];
        auto half_of_p = [&](int h, uint32_t (&hi)[16], uint32_t (&mid)[16], uint32_t (&lo)[16]) {
          const float mu = m_run == -INFINITY ? 0.f : m_run;
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
      TileWork next;
      if (!ok || !next_work(n, next) || !wait_phase(&sm.p_done, (steps - 1) & 1, abort_flag)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const float inv = l_run > 0.f ? 1.f / l_run : 0.f;
      const float beta = m_sum == -INFINITY ? 0.f : fast_exp2(m_sum - m_run);
      // Half a row at a time through shared memory, so that 8 lanes write 128
      // contiguous bytes (a row per lane writes 32 half sectors at once: the
      // four warps' stores then took 2,000 cycles a tile). Row r's chunk c is
      // kept at c ^ (r % 8), different banks for 8 rows.
      float4* rows_out = reinterpret_cast<float4*>(
          prm.out + ((static_cast<size_t>(work.row) + warp * 8) * kHq + work.g * kGroup) * kDim);
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
            rows_out[(e * kHq + (lane >> 3)) * (kDim / 4) + dh * 8 + (lane & 7)] = x;
        }
        __syncwarp();
      }
      // O is in registers before the next tile's first P is handed over
      tc_fence_before();
      work = next;
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
      !pkv_aligned16(block_tables) || !pkv_aligned4(cu_tokens) || !pkv_aligned4(start_pos) ||
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
  prm.batch = batch;
  // every CTA of a wave takes tiles until none is left; there are at most so many
  prm.next_tile = pool->prefill_next;
  prm.ctas_done = reinterpret_cast<unsigned int*>(pool->prefill_next + 1);
  const long long tiles = std::min(static_cast<long long>(prm.tiles_max) * batch,
                                   static_cast<long long>(total_tokens) / kTileTokens + batch);
  const int ctas =
      static_cast<int>(std::min<long long>(tiles * kHkv, kCtasPerSm * pool->num_sms));
  window_prefill_kernel<<<ctas, kThreads, kSmemBytes, static_cast<cudaStream_t>(stream)>>>(
      tq, tk, tv, prm);
  return pkv_check_launch();
}
