// Windowed decode attention over the paged KV cache for GB300 (sm_103a),
// with sinks, optional fused append and rotation by several position axes,
// for contexts of up to a million tokens (declared in include/pkv_window.h).
//
// out = sum_t p_t V_t / sum_t p_t, p_t = 2^(q.K_t log2(e) / 8 - m), over the
// visible tokens: one pass with a running maximum m and sum.
//
// A sequence's visible pages are the sink pages [0, sp) and the window's
// pages [wf, n_pages); "page i" below counts through both. One block of 4
// warps per (sequence, kv head, split) serves the 4 query heads, so a page
// tile is read once; warp w takes pages w, w + 4, ... of its block's range
// through its own ring of stages, filled by the tensor copy engine. Splits
// merge inside the launch: through a thread-block cluster's shared memory,
// or through global partials and a ticket.
//
// What bounds it: the bytes of the visible pages, 4 KiB per (page, kv head).
// 4 blocks of 4 warps with 3 stages keep 192 KiB in flight per SM. Four
// sequences of 120,000 to 131,072 tokens take 155 us (6.6 TB/s, 99 % of the
// measured copy rate), 256 full 4,096-token windows 316 us (102 %), 256
// ragged ones behind 4,096 tokens with append and rotation 106.5 us (90 %; the
// last blocks' ranges are the rest). In smaller launches the latencies before
// the first page lands are what is left: 64 ragged sequences behind 1,024 tokens
// take 15.5 us, of which the block reads the lengths and finds its work for 1.7,
// its page ids for 1.2, its first page for 2.4, and merges for 1.5 to 2.3; one
// sequence behind 512 tokens 4.2 us. (Inputs larger than L2, launches in a graph.)

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "pkv.h"
#include "pkv_window.h"
#include "axes.cuh"
#include "decode_device.cuh"
#include "device_common.cuh"
#include "pool_internal.h"

using namespace pkv_dev;
using namespace pkv_decode;
using namespace pkv_axes_dev;

namespace {

constexpr int kWarps = 4;
constexpr int kStagesW = 3;
constexpr int kThreadsW = kWarps * 32;
constexpr int kTries = 8;             // range sizes tried for a one-wave launch
constexpr int kHeld = 3;              // sequences per thread whose page count is kept

struct alignas(1024) WindowSmem {
  PageRing<kStagesW> warp[kWarps];
  unsigned long long bar[kWarps][kStagesW];
  float m[kWarps][kGroup];
  float l[kWarps][kGroup];
  float acc[kWarps][kGroup][kDim];   // the warps' partial outputs (block merge)
  struct {                           // unit search
    float pages[kWarps];
    int most[kWarps];
    int full[kWarps];
    uint32_t c12[kWarps], c34[kWarps];
    int count[2][kWarps];
    int seq, split, len;
    int4 unit;
  } find;
  int last;
};
static_assert(4 * (sizeof(WindowSmem) + 1024 + 1024) <= kSmemPerSm, "4 ticket blocks per SM");
static_assert(3 * (sizeof(WindowSmem) + sizeof(AsyncInbox) + 1024 + 1024) <= kSmemPerSm,
              "3 cluster blocks per SM");
static_assert(sizeof(WindowSmem) % 16 == 0, "the cluster inbox follows 16-byte aligned");

struct WindowParams {
  const uint16_t* q;          // [B][32][64]
  const uint16_t* k_new;      // [B][8][64]   (fused only)
  const uint16_t* v_new;
  uint16_t* k_pool;           // [num_pages][8][16][64]
  uint16_t* v_pool;
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

// ---------------------------------------------------------------- page math
// As in decode_device.cuh one page's products are warp-wide mma.sync
// m16n8k16 whose 16 rows hold the 4 query heads; here all 16 rows work. A
// factor that is not exact in BF16 (a probability, a rotated query) is split
// into three BF16 terms, 24 bits in all: the high parts in rows 0..3, the
// middle ones in rows 4..7 and the low ones in rows 8..11, so one product
// covers the three (the P V products of a page take 8 instructions; two
// terms in the same rows one after the other would take 16).
__device__ __forceinline__ void mma_rows16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                           uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The queries as A fragments: lane L serves head (L / 4) % 4, dims 16 (L % 4)
// .. + 15 as 8 pairs. Without rotation both lane halves hold the same exact
// BF16 values (rows 0..3 and 4..7), so both get every score. With rotation qa
// holds the high parts (lanes 0..15) and the middle ones (16..31), ql the low
// parts (lanes 0..15; zero above). (c, s): the angle of pair `lane`.
template <bool kRope>
__device__ __forceinline__ void load_queries(const uint16_t* qrow, int lane, float c, float s,
                                             uint32_t (&qa)[8], uint32_t (&ql)[8]) {
  const int g = (lane >> 2) & 3;
  const int qq = lane & 3;
  const uint4* src = reinterpret_cast<const uint4*>(qrow + g * kDim + 16 * qq);
  const uint4 a = __ldg(src);
  const uint4 b = __ldg(src + 1);
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  #pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (!kRope) {
      qa[i] = w[i];
      ql[i] = 0u;
    } else {
      // dims < 32: x cos - y sin; dims >= 32: y cos + x sin; the partner
      // half sits in lane ^ 2
      const uint32_t pw = __shfl_xor_sync(0xffffffffu, w[i], 2);
      const float2 own = bf16x2_to_float2(w[i]);
      const float2 par = bf16x2_to_float2(pw);
      const int pair = 16 * (qq & 1) + 2 * i;
      const float c0 = __shfl_sync(0xffffffffu, c, pair);
      const float c1 = __shfl_sync(0xffffffffu, c, pair + 1);
      const float s0 = __shfl_sync(0xffffffffu, s, pair);
      const float s1 = __shfl_sync(0xffffffffu, s, pair + 1);
      const float sgn = qq < 2 ? -1.f : 1.f;
      const float r0 = __fadd_rn(__fmul_rn(own.x, c0), sgn * __fmul_rn(par.x, s0));
      const float r1 = __fadd_rn(__fmul_rn(own.y, c1), sgn * __fmul_rn(par.y, s1));
      uint32_t hi, mid, lo;
      split3(r0, r1, hi, mid, lo);
      qa[i] = lane < 16 ? hi : mid;
      ql[i] = lane < 16 ? lo : 0u;
    }
  }
}

// A warp's running softmax state: o[j] holds dims 8 j + 2 q, + 1 (q = lane % 4)
// of its row's part. A page's products start from zero and are added here: a
// tensor-core sum drops the bits below its accumulator's last one, always
// downwards, which over a long context adds up (1.8e-6 of the output after
// 131,072 tokens with the accumulator kept in the product, against 3e-7).
struct PageState {
  float o[8][2];
  float m_run;     // base-2 max the exponentials of the head are taken against
  float l_run;     // this lane's share of the head's sum
};

// One page: K tile kt and V tile vt (swizzled, in shared memory), bit t of
// `seen` = token t counts (at least one does). The scores of the others are
// dropped by select; their V rows must hold finite values. Lanes L and L + 16
// hold the same scores, maximum and sum of head (L / 4) % 4.
template <bool kRope>
__device__ __forceinline__ void attend_page(const uint8_t* kt, const uint8_t* vt, uint32_t seen,
                                            int lane, const uint32_t (&qa)[8],
                                            const uint32_t (&ql)[8], PageState& st) {
  const int g8 = lane >> 2;
  const int qq = lane & 3;
  float s[4];
  #pragma unroll
  for (int nt = 0; nt < 2; ++nt) {
    const uint8_t* row = kt + (8 * nt + g8) * kRowBytes;
    const uint4 k0 = *reinterpret_cast<const uint4*>(row + (((2 * qq) ^ g8) << 4));
    const uint4 k1 = *reinterpret_cast<const uint4*>(row + (((2 * qq + 1) ^ g8) << 4));
    const uint32_t kw[8] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w};
    float d[4] = {0.f, 0.f, 0.f, 0.f};
    #pragma unroll
    for (int sl = 0; sl < 4; ++sl)
      mma_rows16(d, qa[2 * sl], kRope ? ql[2 * sl] : 0u, qa[2 * sl + 1],
                 kRope ? ql[2 * sl + 1] : 0u, kw[2 * sl], kw[2 * sl + 1]);
    if (kRope) {   // rows g, g + 4 and g + 8: the three parts of head g's query
      d[0] = (d[0] + __shfl_xor_sync(0xffffffffu, d[0], 16)) +
             (d[2] + __shfl_xor_sync(0xffffffffu, d[2], 16));
      d[1] = (d[1] + __shfl_xor_sync(0xffffffffu, d[1], 16)) +
             (d[3] + __shfl_xor_sync(0xffffffffu, d[3], 16));
    }
    s[2 * nt] = d[0];
    s[2 * nt + 1] = d[1];
  }
  const float c = 1.4426950408889634f * 0.125f;   // log2(e) / sqrt(64)
  float x[4];
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = 8 * (i >> 1) + 2 * qq + (i & 1);
    x[i] = (seen >> t) & 1u ? s[i] * c : -INFINITY;
  }
  float pm = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
  pm = fmaxf(pm, __shfl_xor_sync(0xffffffffu, pm, 1));
  pm = fmaxf(pm, __shfl_xor_sync(0xffffffffu, pm, 2));
  // the max used moves only when the head's max grows by more than 2^8
  const bool grow = pm > st.m_run + kRescaleLog2;
  if (__any_sync(0xffffffffu, grow)) {
    const float alpha = grow ? fast_exp2(st.m_run - pm) : 1.f;   // 0 on the first page
    if (grow) st.m_run = pm;
    st.l_run *= alpha;
    #pragma unroll
    for (int j = 0; j < 8; ++j) {
      st.o[j][0] *= alpha;
      st.o[j][1] *= alpha;
    }
  }
  const float mu = st.m_run == -INFINITY ? 0.f : st.m_run;
  float p[4];
  #pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = fast_exp2(x[i] - mu);
  st.l_run += (p[0] + p[1]) + (p[2] + p[3]);
  // P as A fragments: tokens 2 q, 2 q + 1 (a0, a1) and 8 + 2 q, 9 + 2 q (a2, a3)
  uint32_t pa[2], pl[2];
  #pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t hi, mid, lo;
    split3(p[2 * h], p[2 * h + 1], hi, mid, lo);
    pa[h] = lane < 16 ? hi : mid;
    pl[h] = lane < 16 ? lo : 0u;
  }
  // lane L addresses row L % 8 of matrix L / 8 (tokens 0..7 or 8..15, dim
  // chunk 2 jj or 2 jj + 1)
  const int mrow = lane & 7;
  const int mat = lane >> 3;
  const uint32_t vrow = smem_u32(vt) + (mrow + 8 * (mat & 1)) * kRowBytes;
  #pragma unroll
  for (int jj = 0; jj < 4; ++jj) {
    uint32_t bv[4];
    ldsm_x4_trans(bv, vrow + (((2 * jj + (mat >> 1)) ^ mrow) << 4));
    #pragma unroll
    for (int h = 0; h < 2; ++h) {
      float d[4] = {0.f, 0.f, 0.f, 0.f};
      mma_rows16(d, pa[0], pl[0], pa[1], pl[1], bv[2 * h], bv[2 * h + 1]);
      // rows g (high or middle parts) and g + 8 (low parts) of the same head
      st.o[2 * jj + h][0] += d[0] + d[2];
      st.o[2 * jj + h][1] += d[1] + d[3];
    }
  }
}

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
__device__ __forceinline__ bool find_unit(int u, const WindowParams& prm, WindowSmem& sm, int& b,
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
      sm.find.pages[warp] = sum;
      sm.find.most[warp] = most;
    }
    __syncthreads();
    sum = 0.f;
    #pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      sum += sm.find.pages[w];
      most = max(most, sm.find.most[w]);
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
      sm.find.full[warp] = full;
      sm.find.c12[warp] = c12;
      sm.find.c34[warp] = c34;
    }
    __syncthreads();
    full = 0;
    c12 = c34 = 0;
    #pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      full += sm.find.full[w];
      c12 += sm.find.c12[w];
      c34 += sm.find.c34[w];
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
      if (lane == 0) sm.find.count[turn][warp] = total;
      __syncthreads();
      total = 0;
      #pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const int cw = sm.find.count[turn][w];
        excl += w < warp ? cw : 0;
        total += cw;
      }
    }
    if (u < before + total) {                // the same decision in every thread
      const bool mine = u >= excl && u < excl + units;
      const int at = cls == 0 ? u - excl : f;
      if (kBlock) {
        if (mine) {
          sm.find.seq = base + me;
          sm.find.split = at;
          sm.find.len = own_len;
        }
        __syncthreads();
        b = sm.find.seq;
        split = sm.find.split;
        len = sm.find.len;
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
template <bool kFused, bool kCluster, bool kRope>
__global__ void __launch_bounds__(kThreadsW, kCluster ? 3 : 4)
window_decode_kernel(const __grid_constant__ CUtensorMap tmap_k,
                     const __grid_constant__ CUtensorMap tmap_v, const WindowParams prm) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem_base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  WindowSmem& sm = *reinterpret_cast<WindowSmem*>(smem_base);
  AsyncInbox& inbox = *reinterpret_cast<AsyncInbox*>(smem_base + sizeof(WindowSmem));

  const bool units = !kCluster && prm.num_splits == 0;   // grid (units x kv heads)
  int split = blockIdx.x;
  const int kvh = units ? blockIdx.x % kHkv : blockIdx.y;
  int b = blockIdx.z;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  PageRing<kStagesW>& ws = sm.warp[warp];
  unsigned long long* bars = sm.bar[warp];
  if (lane == 0) {
    for (int s = 0; s < kStagesW; ++s) mbar_init(&bars[s], 1);
    fence_mbar_init();
    if (warp == 1) {          // warp 0 goes on to the unit search
      prefetch_tensormap(&tmap_k);
      prefetch_tensormap(&tmap_v);
    }
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
        found = find_unit<false>(u, prm, sm, b, split, range, len);
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
      found = find_unit<true>(u, prm, sm, b, split, range, len);
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
  const int first = page_begin + warp;        // this warp's pages: first + 4 j, j < mine
  const int mine = first < page_end ? (page_end - first + kWarps - 1) / kWarps : 0;
  const int new_slot = (len - 1) % kPage;     // slot of the appended token
  // fused: which of this warp's pages is the sequence's last one
  const int new_off = n_seen - 1 - first;
  const int j_new = new_off >= 0 && new_off % kWarps == 0 && new_off / kWarps < mine
                        ? new_off / kWarps
                        : -1;

  const int32_t* row = prm.table + static_cast<size_t>(b) * prm.table_stride;
  auto logical = [&](int j) {
    const int i = first + kWarps * j;
    return i < sink_pages ? i : i - sink_pages + win_page;
  };
  // Physical ids of 32 of this warp's pages, one per lane; the next 32 are
  // fetched while these are in use.
  auto fetch_ids = [&](int base) {
    const int j = base + lane;
    return j < mine ? __ldg(row + logical(j)) : -1;
  };
  int ids = fetch_ids(0);
  int ids_next = mine > 32 ? fetch_ids(32) : -1;
  auto good_id = [&](int phys) { return phys >= 0 && phys < prm.num_pages; };
  float ang_c = 1.f, ang_s = 0.f;                        // the angle of pair `lane`
  if (kRope && !load_pair_angle(prm.rope, rope_pos, lane, ang_c, ang_s)) {
    if (split == 0 && kvh == 0 && threadIdx.x == 0) set_error(prm.err, kErrPosition);
    leave();
    return;                                              // every block of the sequence
  }

  if (kCluster && n_splits > 1) async_inbox_setup(inbox);
  __syncwarp();

  // Copy engine: the K and V tiles of page j into `stage`, from lanes 0 and
  // 1. A page whose only token is the appended one (fused) is not copied.
  uint32_t stage_ok = 0;                      // bit s: stage s holds a valid page
  auto issue_copy = [&](int j, int stage, int phys) {
    const bool ok = good_id(phys);
    stage_ok = ok ? stage_ok | (1u << stage) : stage_ok & ~(1u << stage);
    if (lane > 1) return;
    const bool rows = !(kFused && j == j_new && new_slot == 0);
    if (!ok && lane == 0) set_error(prm.err, kErrPage);
    if (ok && rows) {
      if (lane == 0) mbar_arrive_expect_tx(&bars[stage], 2 * kTileBytes);
      __syncwarp(0x3u);   // the expected bytes are set before either copy can land
      tma_load_tile(lane == 0 ? ws.k[stage] : ws.v[stage], lane == 0 ? &tmap_k : &tmap_v,
                    kvh * kPage, phys, &bars[stage]);
    } else if (lane == 0) {
      mbar_arrive(&bars[stage]);
    }
  };
  // Fused: the appended row, one 16-byte chunk per lane (K in lanes 0..7, V
  // in 8..15). Loaded ahead of the pages; rotated, written to the pool and
  // patched into the stage at its page's turn, when the load has long arrived
  // (64 ragged sequences behind 1,024 tokens: 15.6 us; done ahead, 15.9).
  auto load_new_row = [&]() {
    uint4 val = make_uint4(0u, 0u, 0u, 0u);
    if (lane < 16)
      val = __ldg(reinterpret_cast<const uint4*>(
          (lane >= 8 ? prm.v_new : prm.k_new) +
          (static_cast<size_t>(b) * kHkv + kvh) * kDim + (lane & 7) * 8));
    return val;
  };
  auto write_new_row = [&](int phys, uint4 val) {        // returns the chunk as stored
    const int c = lane & 7;
    if (kRope) {
      const uint4 partner = shfl_xor_uint4(val, 4);
      float cs[8], sn[8];
      #pragma unroll
      for (int e = 0; e < 8; ++e) {
        cs[e] = __shfl_sync(0xffffffffu, ang_c, 8 * (c & 3) + e);
        sn[e] = __shfl_sync(0xffffffffu, ang_s, 8 * (c & 3) + e);
      }
      if (lane < 8) val = rope_key_chunk(val, partner, c >= 4, cs, sn);
    }
    if (lane < 16 && good_id(phys))
      *reinterpret_cast<uint4*>((lane >= 8 ? prm.v_pool : prm.k_pool) +
                                ((static_cast<size_t>(phys) * kHkv + kvh) * kPage + new_slot) *
                                    kDim + c * 8) = val;
    return val;
  };

  // Prefetch: the first pages' tiles in one copy instruction, lane 2 j (K)
  // and 2 j + 1 (V) serving page j. The unfused kernel defers the last page,
  // whose newest row the kernel before this one may be writing.
  const int n_prefetch = min(mine, kStagesW);
  const bool deferred = !kFused && j_new >= 0 && j_new < n_prefetch;
  {
    const int j = lane >> 1;
    const int phys = __shfl_sync(0xffffffffu, ids, j);
    const bool ok = good_id(phys);
    const bool serves = j < n_prefetch && (kFused || j != j_new);
    const bool rows = !(kFused && j == j_new && new_slot == 0);
    stage_ok = __ballot_sync(0xffffffffu, lane < n_prefetch && good_id(ids)) &
               ((1u << kStagesW) - 1u);
    if (serves && (lane & 1) == 0) {
      if (!ok) set_error(prm.err, kErrPage);
      if (ok && rows) {
        mbar_arrive_expect_tx(&bars[j], 2 * kTileBytes);
      } else {
        mbar_arrive(&bars[j]);
      }
    }
    __syncwarp();
    if (serves && ok && rows)
      tma_load_tile((lane & 1) == 0 ? ws.k[j] : ws.v[j], (lane & 1) == 0 ? &tmap_k : &tmap_v,
                    kvh * kPage, phys, &bars[j]);
  }
  pdl_wait();
  pdl_launch_dependents();
  if (deferred) issue_copy(j_new, j_new, __shfl_sync(0xffffffffu, ids, j_new));
  // the new row's load goes out before the queries', so their latencies overlap
  uint4 new_row = make_uint4(0u, 0u, 0u, 0u);
  if (kFused && j_new >= 0) new_row = load_new_row();
  int new_page = kFused && j_new >= 0 && j_new < n_prefetch ? __shfl_sync(0xffffffffu, ids, j_new)
                                                            : -1;
  uint32_t qa[8], ql[8];
  load_queries<kRope>(prm.q + (static_cast<size_t>(b) * kHq + kvh * kGroup) * kDim, lane, ang_c,
                      ang_s, qa, ql);

  PageState st;
  #pragma unroll
  for (int j = 0; j < 8; ++j) st.o[j][0] = st.o[j][1] = 0.f;
  st.m_run = -INFINITY;
  st.l_run = 0.f;
  int issued = n_prefetch;
  int consumed = 0;
  bool timed_out = false;
  int stage = 0;
  uint32_t phase = 0;
  for (int j = 0; j < mine; ++j) {
    if (!__all_sync(0xffffffffu, mbar_wait(&bars[stage], phase))) {
      timed_out = true;
      break;
    }
    consumed = j + 1;
    const int t0 = logical(j) * kPage;
    uint32_t seen = 0xffffu;
    // a page inside the window, or one of sinks alone, is seen whole
    if (t0 + kPage > len || t0 < win_lo)
      seen = low_bits(len - t0) & (low_bits(prm.sinks - t0) | (0xffffu & ~low_bits(win_lo - t0)));
    if (!((stage_ok >> stage) & 1u)) seen = 0;
    const bool with_new = kFused && j == j_new;
    if (seen != 0xffffu || with_new) {
      // V rows that do not count are zeroed (0 times what they hold must stay
      // 0), and the appended row goes over what the copy brought
      uint8_t* vt = ws.v[stage];
      for (int idx = lane; idx < kPage * 8; idx += 32)
        if (!((seen >> (idx >> 3)) & 1u))
          *reinterpret_cast<uint4*>(vt + idx * 16) = make_uint4(0u, 0u, 0u, 0u);
      __syncwarp();
      if (with_new) {
        const uint4 stored = write_new_row(new_page, new_row);
        if (seen && lane < 16) {
          uint8_t* t = lane >= 8 ? ws.v[stage] : ws.k[stage];
          *reinterpret_cast<uint4*>(t + new_slot * kRowBytes +
                                    (((lane & 7) ^ (new_slot & 7)) << 4)) = stored;
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
    }
    if (seen) attend_page<kRope>(ws.k[stage], ws.v[stage], seen, lane, qa, ql, st);
    __syncwarp();   // every lane's reads of the stage are done before it is refilled
    const int next = j + kStagesW;
    if (next < mine) {
      if ((next & 31) == 0) {
        ids = ids_next;
        ids_next = fetch_ids(next + 32);
      }
      const int phys = __shfl_sync(0xffffffffu, ids, next & 31);
      issue_copy(next, stage, phys);
      if (kFused && next == j_new) new_page = phys;
      issued = next + 1;
    }
    if (++stage == kStagesW) {
      stage = 0;
      phase ^= 1u;
    }
  }
  if (timed_out) {
    // this warp's copies in flight land before the block exits (each wait bounded)
    for (int j = consumed; j < issued; ++j) mbar_wait(&bars[j % kStagesW], (j / kStagesW) & 1);
    if (lane == 0) set_error(prm.err, kErrTimeout);
    st.m_run = -INFINITY;
    st.l_run = 0.f;
  }

  // lanes L and L + 16 hold the parts of the same head
  MmaState total;
  #pragma unroll
  for (int j = 0; j < 8; ++j) {
    #pragma unroll
    for (int e = 0; e < 2; ++e) {
      total.o[j][e] = st.o[j][e] + __shfl_xor_sync(0xffffffffu, st.o[j][e], 16);
      total.o[j][e + 2] = 0.f;
    }
  }
  total.m_run = st.m_run;
  total.l_run = st.l_run;
  float M, L;
  float2 O;
  block_merge_mma<kWarps>(sm, total, warp, lane, M, L, O);
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
constexpr size_t kTicketSmemBytes = sizeof(WindowSmem) + 1024;
constexpr size_t kClusterSmemBytes = sizeof(WindowSmem) + sizeof(AsyncInbox) + 1024;

using WindowKernel = void (*)(const CUtensorMap, const CUtensorMap, const WindowParams);

template <bool kCluster>
WindowKernel window_kernel(bool fused, bool rope) {
  return fused ? (rope ? window_decode_kernel<true, kCluster, true>
                       : window_decode_kernel<true, kCluster, false>)
               : (rope ? window_decode_kernel<false, kCluster, true>
                       : window_decode_kernel<false, kCluster, false>);
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

// Small batches take a cluster per (sequence, kv head): its merge is shorter
// than the ticket's (us, one 2,048-token sequence: cluster of 12 5.7, units
// 6.8; 4 sequences at a 1,024-token window: 6.0 and 6.9), as long as all blocks
// are resident at once (4 sequences, cluster of 16: 9.4) and either fill half
// of the slots or have few pages (one 131,072-token sequence: cluster of 12
// 120.6, units 48.0). Everything else takes units.
constexpr int kMostCluster = 12;

WindowPlan plan_window(const pkv_pool* pool, int batch, int window, int sinks, int num_splits) {
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
      static_cast<long long>(pool->window_cluster_blocks_per_sm) * pool->num_sms;
  const int s = std::min({kMostCluster, pool->max_cluster, c.max_splits,
                          (seen + kWarps - 1) / kWarps});
  if (s >= 2 && rows * s <= cluster_slots &&
      (seen <= 4 * kWarps * s || 2 * rows * s >= cluster_slots)) {
    p.num_splits = s;
    p.cluster = true;
    return p;
  }
  const int wave = std::max(1, pool->window_blocks_per_sm * pool->num_sms / kHkv);
  const int fewest = (seen + c.max_splits - 1) / c.max_splits;   // keeps to max_splits ranges
  if (batch <= std::min(wave, 32 * kHeld)) p.wave_units = wave;
  p.range_div = std::max(1, 3 * wave / 5);
  p.least_pages = std::max(2 * kWarps, fewest);
  p.units = std::max(p.wave_units, batch + p.range_div);
  return p;
}

template <bool kFused>
pkv_status launch_window(pkv_pool_t pool, int layer, const void* q, const void* k, const void* v,
                         const void* k_pool, const void* v_pool, const int32_t* block_tables,
                         const int32_t* seq_lens, float* out, int window, int sinks,
                         const pkv_axes_rope* rope, const int32_t* rope_positions,
                         int position_stride, int batch, int num_splits, void* stream) {
  if (!pool) return PKV_ERR_INVALID_ARG;
  const pkv_pool_config& c = pool->cfg;
  if (layer < 0 || layer >= c.num_layers || batch < 0 || batch > c.max_batch)
    return PKV_ERR_INVALID_ARG;
  if (num_splits < 0 || num_splits > c.max_splits || window < 1 || sinks < 0)
    return PKV_ERR_INVALID_ARG;
  if (batch == 0) return PKV_OK;
  if (!q || !k_pool || !v_pool || !block_tables || !seq_lens || !out || (kFused && (!k || !v)))
    return PKV_ERR_INVALID_ARG;
  if (!pkv_aligned16(q) || !pkv_aligned16(k) || !pkv_aligned16(v) || !pkv_aligned16(k_pool) ||
      !pkv_aligned16(v_pool) || !pkv_aligned16(block_tables) || !pkv_aligned4(seq_lens) ||
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
  prm.k_pool = const_cast<uint16_t*>(static_cast<const uint16_t*>(k_pool));
  prm.v_pool = const_cast<uint16_t*>(static_cast<const uint16_t*>(v_pool));
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
  const WindowPlan plan = plan_window(pool, batch, prm.window, prm.sinks, num_splits);
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
  cfg.dynamicSmemBytes = cluster ? kClusterSmemBytes : kTicketSmemBytes;
  cfg.stream = static_cast<cudaStream_t>(stream);
  CUtensorMap tk, tv;
  if (!pkv_pool_tensor_map(k_pool, c.num_pages, &tk) ||
      !pkv_pool_tensor_map(v_pool, c.num_pages, &tv))
    return PKV_ERR_CUDA;
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
  const WindowKernel kernel = cluster ? window_kernel<true>(kFused, rope != nullptr)
                                      : window_kernel<false>(kFused, rope != nullptr);
  if (cudaLaunchKernelEx(&cfg, kernel, tk, tv, prm) != cudaSuccess) return PKV_ERR_CUDA;
  return pkv_check_launch();
}

}  // namespace

bool pkv_window_setup(pkv_pool* pool) {
  bool ok = true;
  for (int v = 0; v < 4 && ok; ++v) {
    const WindowKernel ticket = window_kernel<false>(v & 1, v & 2);
    const WindowKernel cluster = window_kernel<true>(v & 1, v & 2);
    ok = cudaFuncSetAttribute(ticket, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(kTicketSmemBytes)) == cudaSuccess &&
         cudaFuncSetAttribute(cluster, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(kClusterSmemBytes)) == cudaSuccess &&
         cudaFuncSetAttribute(cluster, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) ==
             cudaSuccess;
  }
  ok = ok && cudaOccupancyMaxActiveBlocksPerMultiprocessor(
                 &pool->window_blocks_per_sm, window_kernel<false>(true, true), kThreadsW,
                 kTicketSmemBytes) == cudaSuccess;
  ok = ok && cudaOccupancyMaxActiveBlocksPerMultiprocessor(
                 &pool->window_cluster_blocks_per_sm, window_kernel<true>(true, true), kThreadsW,
                 kClusterSmemBytes) == cudaSuccess;
  if (pool->window_blocks_per_sm < 1) pool->window_blocks_per_sm = 1;
  if (pool->window_cluster_blocks_per_sm < 1) pool->window_cluster_blocks_per_sm = 1;
  return ok;
}

extern "C" {

pkv_status pkv_window_attention(pkv_pool_t pool, int layer, const void* q, const void* k_pool,
                                const void* v_pool, const int32_t* block_tables,
                                const int32_t* seq_lens, float* out, int window, int sinks,
                                const pkv_axes_rope* rope, const int32_t* rope_positions,
                                int position_stride, int batch, int num_splits, void* stream) {
  return launch_window<false>(pool, layer, q, nullptr, nullptr, k_pool, v_pool, block_tables,
                              seq_lens, out, window, sinks, rope, rope_positions, position_stride,
                              batch, num_splits, stream);
}

pkv_status pkv_window_append_attend(pkv_pool_t pool, int layer, const void* q, const void* k,
                                    const void* v, void* k_pool, void* v_pool,
                                    const int32_t* block_tables, const int32_t* seq_lens,
                                    float* out, int window, int sinks,
                                    const pkv_axes_rope* rope, const int32_t* rope_positions,
                                    int position_stride, int batch, int num_splits,
                                    void* stream) {
  return launch_window<true>(pool, layer, q, k, v, k_pool, v_pool, block_tables, seq_lens, out,
                             window, sinks, rope, rope_positions, position_stride, batch,
                             num_splits, stream);
}

}  // extern "C"
