// Decode attention over the 8-bit KV cache for GB300 (sm_103a), with windows,
// sinks, optional fused append and rotation by several position axes (declared
// in include/pkv_quant.h). The kernel is window_device.cuh's; here are the
// 8-bit pages' tiles and their products.
//
// A tile's codes c stand for c 2^e, e one exponent a token (K_t = c_t 2^ek_t, V_t
// = d_t 2^ev_t), so with the codes as exact FP16 operands
//   score_t = 2^ek_t (q . c_t),   out = sum_t (p_t 2^ev_t) d_t / sum_t p_t.
//
// What bounds it: the bytes of the visible tiles, 2,080 per (page, KV head), while
// a warp's instructions keep up: a tile takes half as long to arrive as a BF16 one
// and its codes have to be widened, so the arithmetic per page had to come down.
// Four sequences of 120,000 to 131,072 tokens, step by step: 131 us with one page
// at a time; 95.5 with two (one barrier, one vote and one set of unpacked exponents
// for 32 tokens, arithmetic on pairs of FP32 values); 93.7 with groups seen whole
// told by one comparison and the weights split by mixed-precision multiply-adds; 90
// with one vote per group instead of two, exponentials taken before it; 84 (6.2 TB/s,
// 93 % of the measured copy rate, 2 us more than the copies alone) with copies issued
// by one lane from uniform operands and two stages a warp instead of three. 256 ragged
// sequences behind 4,096 tokens, append and rotation included, take 68.5 us (77 %; the
// short sequences' blocks are latency), 64 of up to 2,048 tokens 11.9 us, of which the
// unit search, page ids, the first copies and the merge are 8, one of 2,048 4.6 us.
// (Inputs larger than L2 in total, launches in a graph.) Slower: five blocks an SM (by
// 7 to 20 %), scores computed ahead beside the products before them (2 % faster over
// long contexts, 3 to 6 % slower in ragged batches). Units that rise again and scores of any
// size cost the branch of each warp's first group 0.1 us apiece.

#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "pkv.h"
#include "pkv_quant.h"
#include "quant.cuh"
#include "window_device.cuh"

using namespace pkv_window;
using namespace pkv_quant_dev;

namespace {

// ---------------------------------------------------------------- page math
// A warp takes two pages at a time. Their products are warp-wide mma.sync m16n8k16
// of FP16 operands.
//   scores: S = Q K^T, rows = the 4 heads' queries, their high parts in rows 0..3
//           (again in 4..7) and with rotation their low ones in 8..11 (12..15),
//           columns = 8 tokens;
//   values: O^T += V^T P^T, rows = 16 dims, columns = the 4 heads' weights,
//           high parts in columns 0..3 and low ones in 4..7, contraction over
//           16 tokens: products that fill the instruction's whole shape.
// The scores' accumulators are then P^T's operand fragments: lane (g, q) = (L /
// 4, L % 4) holds head g % 4's tokens 2 q, 2 q + 1 of every 8 in both.
//
// FP16 has 11 bits and a narrow range: a factor that needs 24 bits (a rotated
// query, a weight) is the sum of two FP16 terms after a scaling by a power of
// two, one per head: queries so that the largest of 64 dims lies in [2^14,
// 2^15), weights p 2^ev so that the largest up to here, as it counts now, lies in
// [2^7, 2^15]. Terms lose what lies 2^-31 and more below the largest.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Two FP32 values -> FP16 pair, rounded to nearest even.
__device__ __forceinline__ uint32_t float2_to_half2(float e0, float e1) {
  uint32_t w;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(e1), "f"(e0));
  return w;
}

// x + m (an FP16 half of the pair h), m an FP16 number: with m = -1 what h, x
// rounded, leaves of x, exactly.
template <int kUpper>
__device__ __forceinline__ float plus_half(float x, uint32_t h, uint16_t m) {
  float d;
  if (kUpper)
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tfma.rn.f32.f16 %0, u, %2, %3;\n\t}"
        : "=f"(d)
        : "r"(h), "h"(m), "f"(x));
  else
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tfma.rn.f32.f16 %0, l, %2, %3;\n\t}"
        : "=f"(d)
        : "r"(h), "h"(m), "f"(x));
  return d;
}
constexpr uint16_t kMinusOne = 0xbc00;

// The high parts (m = 0) or the low ones (m = -1) of two values.
__device__ __forceinline__ uint32_t half_terms(float x0, float x1, uint16_t m) {
  const uint32_t hi = float2_to_half2(x0, x1);
  return float2_to_half2(plus_half<0>(x0, hi, m), plus_half<1>(x1, hi, m));
}

// Largest over the four lanes of a row.
__device__ __forceinline__ float row_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}

// 2^n for n <= 0, exact; 0 below 2^-126.
__device__ __forceinline__ float power_of_2(int n) {
  return scale_of(static_cast<uint32_t>(max(n + 127, 0)));
}

// -FLT_MAX, no finite score lies below it: with it as the exponent of a row that saw
// nothing yet, no test for -inf - -inf is needed.
constexpr float kNone = -0x1.fffffep127f;

// Products of scaled queries and codes reach 2^30 and exponents 2^120: a score is held
// in units of 2^16 of theirs, so that it does not pass FP32's range before the query's
// scaling is taken back out of it (with any |K| below 2^122; without the unit 2^106).
// Exact: 2^-16 2^ek is a power of two >= 2^-140.
constexpr float kScoreUnit = 0x1p-16f;

struct QuantTiles {
  // With 3, 4 sequences of 131,072 tokens take 92 us instead of 84.
  static constexpr int kStages = 2;
  static constexpr int kStagePages = 2;
  static constexpr int kParts = 1;
  static constexpr uint32_t kCopyBytes = kQuantTile;
  struct alignas(16) Ring {
    uint8_t tile[kStages][kStagePages][kQuantTile];
    // kScoreUnit 2^ek of two neighbouring tokens, then their 2^ev
    float scale[kStagePages * kPage / 2][4];
  };
  struct Source {
    uint8_t* pool;               // [num_pages][8][kQuantTile]
  };
  // Lane (g, q): head g % 4, dims 16 q .. + 15 as 8 pairs; `to_log2` takes the
  // products with the scaled query to the exponent's base-2 scores.
  struct Queries {
    uint32_t a[8], l[8];       // high parts, and with rotation low ones
    float to_log2;
  };
  struct State {
    float o[4][4];   // chunk c: dims 16 c + 2 g (0, 1) and + 1 (2, 3), columns 2 q, 2 q + 1
    float m_run;     // the base-2 exponent p is taken against: p = 2^(x - m_run) <= 1
                     // (kNone: nothing seen yet)
    float l_run;     // this lane's share of the head's sum
    float unit;      // the power of two that the weights p 2^ev are scaled by; negative
                     // where m_run is huge
    __device__ __forceinline__ void reset() {
      #pragma unroll
      for (int c = 0; c < 4; ++c) o[c][0] = o[c][1] = o[c][2] = o[c][3] = 0.f;
      m_run = kNone;
      l_run = 0.f;
      unit = 0x1p126f;
    }
    // every column's sums times its head's factor (lane (g, q) holds head g's)
    __device__ __forceinline__ void rescale(float factor, int lane) {
      const int head = 2 * (lane & 1);
      const float f0 = __shfl_sync(0xffffffffu, factor, 4 * head);
      const float f1 = __shfl_sync(0xffffffffu, factor, 4 * head + 4);
      #pragma unroll
      for (int c = 0; c < 4; ++c) {
        o[c][0] *= f0;
        o[c][1] *= f1;
        o[c][2] *= f0;
        o[c][3] *= f1;
      }
    }
  };

  static const WindowResidency& residency(const pkv_pool* pool) { return pool->quant; }
  // The largest of 16, 8 and 4 whose blocks are all resident at once. Measured (us),
  // 2,048-token sequences: one, cluster of 16 4.7, of 12 5.2, of 8 4.9; 3, of 8 5.6,
  // of 16 8.1; 6, of 8 6.4, of 4 7.0; 8, of 4 7.2, of 8 10.0; 12, of 4 8.3, units
  // 10.0; 16, units 12.3, of 4 14.4. Longer ones: one of 8,192 tokens, cluster of 16
  // 7.2, units 8.6; of 32,768, 17.8 and 12.9; 4 of 131,072, of 12 (all slots filled)
  // 89.7, units 90.
  static int cluster_size(long long rows, long long slots) {
    return rows * 16 <= slots * 9 / 16 ? 16
           : rows * 8 <= slots * 27 / 32 ? 8
           : rows * 4 <= slots * 27 / 32 ? 4
                                         : 0;
  }
  static bool fills(long long, long long) { return false; }
  static __device__ __forceinline__ void prefetch(const Source&) {}

  // One bulk copy moves the whole tile.
  static __device__ __forceinline__ void copy(Ring& ws, int stage, int e, const Source& src, int,
                                              int kvh, int phys, unsigned long long* bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
        ::"r"(smem_u32(ws.tile[stage][e])),
          "l"(src.pool + kvh * kQuantTile + static_cast<size_t>(phys) * (kHkv * kQuantTile)),
          "r"(kQuantTile),
          "r"(smem_u32(bar))
        : "memory");
  }

  // V codes and exponents of tokens that do not count: zero.
  static __device__ __forceinline__ void hide_rows(Ring& ws, int stage, uint32_t seen, int lane) {
    #pragma unroll
    for (int e = 0; e < kStagePages; ++e, seen >>= kPage) {
      uint8_t* t = ws.tile[stage][e];
      for (int idx = lane; idx < 4 * kPage; idx += 32)
        if (!((seen >> (idx & (kPage - 1))) & 1u))
          *reinterpret_cast<uint4*>(t + kCodeBytes + idx * 16) = make_uint4(0u, 0u, 0u, 0u);
      if (lane < kPage && !((seen >> lane) & 1u)) t[kVExp + lane] = 0;
    }
  }

  // The appended row (a 16-byte chunk per lane: K in lanes 0..7, V in 8..15):
  // rotated, quantised and put into the pool while the first pages are on their way
  // (256 sequences behind 4,096 tokens: 0.2 us less than at its page's turn, and three
  // registers are kept instead of seven), into the stage at its page's turn.
  struct NewRow {
    uint2 codes;
    uint32_t e;
  };
  template <bool kRope>
  static __device__ __forceinline__ NewRow make_row(const Source& src, int kvh, int slot, int phys,
                                                    bool to_pool, uint4 val, float ang_c,
                                                    float ang_s, int lane) {
    const int c = lane & 7;
    float2 x[1][4];
    unpack8(val, x[0]);
    if (kRope) {
      float2 cs[4], sn[4], partner[4];
      unpack8(shfl_xor_uint4(val, 4), partner);
      const float sign = c < 4 ? -1.f : 1.f;
      #pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int pair = 8 * (c & 3) + 2 * e;
        cs[e] = make_float2(__shfl_sync(0xffffffffu, ang_c, pair),
                            __shfl_sync(0xffffffffu, ang_c, pair + 1));
        sn[e] = make_float2(sign * __shfl_sync(0xffffffffu, ang_s, pair),
                            sign * __shfl_sync(0xffffffffu, ang_s, pair + 1));
      }
      if (lane < 8) rotate8(x[0], partner, cs, sn);
    }
    uint2 codes[1];
    uint32_t e[1];
    quantise_rows(x, codes, e);
    const NewRow made = {codes[0], e[0]};
    if (to_pool)
      store_row(src.pool + (static_cast<size_t>(phys) * kHkv + kvh) * kQuantTile, slot, made, lane);
    return made;
  }
  static __device__ __forceinline__ void store_row(uint8_t* tile, int slot, const NewRow& made,
                                                   int lane) {
    const int c = lane & 7;
    if (lane >= 16) return;
    *reinterpret_cast<uint2*>(tile + (lane < 8 ? k_at(slot, 8 * c) : v_at(slot, 8 * c))) =
        made.codes;
    if (c == 0) tile[(lane < 8 ? kKExp : kVExp) + slot] = static_cast<uint8_t>(made.e);
  }
  template <bool kRope>
  static __device__ __forceinline__ void put_row(Ring& ws, int stage, int page, const Source&, int,
                                                 int slot, int, bool, bool to_stage,
                                                 const NewRow& made, int lane) {
    if (to_stage) store_row(ws.tile[stage][page], slot, made, lane);
  }

  template <bool kRope>
  static __device__ __forceinline__ void load_queries(const uint16_t* qrow, int lane, float c,
                                                      float s, Queries& q) {
    const int g = (lane >> 2) & 3;
    const int qq = lane & 3;
    const uint4* src = reinterpret_cast<const uint4*>(qrow + g * kDim + 16 * qq);
    const uint4 w0 = __ldg(src), w1 = __ldg(src + 1);
    const uint32_t w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
    float x[16];
    #pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float2 own = bf16x2_to_float2(w[i]);
      x[2 * i] = own.x;
      x[2 * i + 1] = own.y;
      if constexpr (kRope) {
        // dims < 32: x cos - y sin; dims >= 32: y cos + x sin; the partner half
        // sits in lane ^ 2
        const float2 par = bf16x2_to_float2(__shfl_xor_sync(0xffffffffu, w[i], 2));
        const int pair = 16 * (qq & 1) + 2 * i;
        const float c0 = __shfl_sync(0xffffffffu, c, pair);
        const float c1 = __shfl_sync(0xffffffffu, c, pair + 1);
        const float s0 = __shfl_sync(0xffffffffu, s, pair);
        const float s1 = __shfl_sync(0xffffffffu, s, pair + 1);
        const float sgn = qq < 2 ? -1.f : 1.f;
        x[2 * i] = __fadd_rn(__fmul_rn(own.x, c0), sgn * __fmul_rn(par.x, s0));
        x[2 * i + 1] = __fadd_rn(__fmul_rn(own.y, c1), sgn * __fmul_rn(par.y, s1));
      }
    }
    float most = 0.f;
    #pragma unroll
    for (int i = 0; i < 16; ++i) most = fmaxf(most, fabsf(x[i]));
    most = row_max(most);
    // 2^(14 - floor(log2 most)), at most 2^125
    const uint32_t up = 268u - max(__float_as_uint(most) >> 23, 16u);
    const float scale = scale_of(up);
    // log2(e) / sqrt(64), at most 0.18 x 2^(113 + 16)
    q.to_log2 = 1.4426950408889634f * 0.125f / kScoreUnit * inverse_scale_of(up);
    #pragma unroll
    for (int i = 0; i < 8; ++i) {
      // without rotation the high parts are the queries (8 bits)
      const float x0 = x[2 * i] * scale, x1 = x[2 * i + 1] * scale;
      q.a[i] = float2_to_half2(x0, x1);
      q.l[i] = kRope ? half_terms(x0, x1, kMinusOne) : 0u;
    }
  }

  static constexpr int kTiles = 2 * kStagePages;     // of 8 tokens
  // Lane (g, q): products of head g % 4 with tokens 8 nt + 2 q, + 1.
  struct Scores {
    float2 s[kTiles];
  };
  // Their weights p 2^ev as FP16 pairs, high or low parts.
  struct Weights {
    uint32_t p[kTiles];
  };

  // A group's products with the queries, and its exponents unpacked, a token per
  // lane, for all.
  template <bool kRope>
  static __device__ __forceinline__ void scores_of(Ring& ws, int stage, int lane,
                                                   const Queries& q, Scores& out) {
    const int g8 = lane >> 2;
    const int qq = lane & 3;
    const uint8_t* own = ws.tile[stage][lane / kPage];
    const uint32_t ek = own[kKExp + lane % kPage], ev = own[kVExp + lane % kPage];
    uint4 kw[kTiles];
    #pragma unroll
    for (int nt = 0; nt < kTiles; ++nt)
      kw[nt] = *reinterpret_cast<const uint4*>(ws.tile[stage][nt / 2] +
                                               k_at(8 * (nt % 2) + g8, 16 * qq));
    ws.scale[lane / 2][lane % 2] = scale_of(ek) * kScoreUnit;
    ws.scale[lane / 2][2 + lane % 2] = scale_of(ev);
    #pragma unroll
    for (int nt = 0; nt < kTiles; ++nt) {
      const uint32_t w[4] = {kw[nt].x, kw[nt].y, kw[nt].z, kw[nt].w};
      float d[4] = {0.f, 0.f, 0.f, 0.f};
      #pragma unroll
      for (int sl = 0; sl < 4; ++sl)
        mma_f16(d, q.a[2 * sl], kRope ? q.l[2 * sl] : 0u, q.a[2 * sl + 1],
                kRope ? q.l[2 * sl + 1] : 0u, codes_to_half2<0>(w[sl]), codes_to_half2<1>(w[sl]));
      out.s[nt] = make_float2(d[0], d[1]);
      // rows g and g + 8: the two parts of head g's query
      if (kRope) out.s[nt] = __fadd2_rn(out.s[nt], make_float2(d[2], d[3]));
    }
  }

  // The group's weights; bit t of `seen` = token t counts. The scores of the
  // others are dropped by select; their V rows and exponents are zero. Lanes L and
  // L + 16 hold the same scores, maxima and sums.
  static __device__ __forceinline__ Weights weights_of(const Ring& ws, uint32_t seen, int lane,
                                                       const Queries& q, const Scores& in,
                                                       State& st) {
    const int qq = lane & 3;
    float2 s[kTiles], scale_v[kTiles], w[kTiles], sum;
    #pragma unroll
    for (int nt = 0; nt < kTiles; ++nt) {
      const float4 sc = *reinterpret_cast<const float4*>(ws.scale[4 * nt + qq]);
      s[nt] = __fmul2_rn(in.s[nt], make_float2(sc.x, sc.y));
      scale_v[nt] = make_float2(sc.z, sc.w);
    }
    if (seen != 0xffffffffu) {
      #pragma unroll
      for (int nt = 0; nt < kTiles; ++nt) {
        if (!((seen >> (8 * nt + 2 * qq)) & 1u)) s[nt].x = -INFINITY;
        if (!((seen >> (8 * nt + 2 * qq + 1)) & 1u)) s[nt].y = -INFINITY;
      }
    }
    const float2 to_log2 = make_float2(q.to_log2, q.to_log2);
    auto exponentials = [&](auto rounded) {
      const float2 minus = make_float2(-st.m_run, -st.m_run);
      sum = make_float2(0.f, 0.f);
      #pragma unroll
      for (int nt = 0; nt < kTiles; ++nt) {
        float2 x;
        if constexpr (decltype(rounded)::value) {   // where m_run is huge
          x.x = less(s[nt].x, q.to_log2, st.m_run);
          x.y = less(s[nt].y, q.to_log2, st.m_run);
        } else {
          x = __ffma2_rn(s[nt], to_log2, minus);
        }
        const float2 p = make_float2(fast_exp2(x.x), fast_exp2(x.y));
        sum = __fadd2_rn(sum, p);
        w[nt] = __fmul2_rn(p, scale_v[nt]);
      }
    };
    // Taken against the state as it is. Where a row's maximum passes the exponent
    // that p is taken against (p would pass 1), that one moves to 8 above it, by
    // whole powers of two; where that happens or the weighted rows pass 2^15 units,
    // the unit is chosen anew. Both are rare. Once a head's exponent is huge every group
    // comes by here: its unit is negative, which as an integer passes too.
    const float lane_top = largest(s) * q.to_log2;
    exponentials(std::false_type());
    const float lane_most = largest(w) * st.unit;
    if (__any_sync(0xffffffffu, lane_top > st.m_run ||
                                    __float_as_uint(lane_most) > __float_as_uint(32768.f))) {
      const float top = row_max(lane_top);
      int shift = 0;                       // the sums held shrink by 2^-shift
      if (top > st.m_run) {
        const float m = floorf(top) + kRescaleLog2;
        shift = static_cast<int>(fminf(m - st.m_run, 512.f));
        st.m_run = m;
        st.l_run *= power_of_2(-shift);    // 0 on the first page
      }
      exponentials(std::false_type());
      const bool huge = is_huge(st.m_run);
      if (__builtin_expect(huge, 0)) exponentials(std::true_type());
      const float most = row_max(largest(w));
      int by = 0;                          // what they are multiplied by: 2^by <= 1
      st.unit = fabsf(st.unit);
      if (shift > 0 || most * st.unit > 32768.f) {
        // 2^(7 - floor(log2 most)) puts the group's largest into [2^7, 2^8). The unit
        // rises as far as the sums held shrank and no further, so that of the rows that
        // they hold none passes 2^15: the largest weighted row up to here, old or new,
        // lies in [2^7, 2^15]. (A unit that did not rise again left rows of ordinary size
        // nothing behind one of 2^35 whose weight had become negligible.)
        const int was = static_cast<int>(__float_as_uint(st.unit) >> 23);
        const int byte = min(min(261 - static_cast<int>(__float_as_uint(most) >> 23), 253),
                             was + shift);
        st.unit = scale_of(static_cast<uint32_t>(byte));
        by = byte - was - shift;
      }
      st.rescale(power_of_2(by), lane);
      if (huge) st.unit = -st.unit;
    }
    st.l_run += sum.x + sum.y;
    const float2 unit = make_float2(fabsf(st.unit), fabsf(st.unit));
    const uint16_t part = lane < 16 ? 0 : kMinusOne;   // high parts in lanes 0..15
    Weights out;
    #pragma unroll
    for (int nt = 0; nt < kTiles; ++nt) {
      const float2 x = __fmul2_rn(w[nt], unit);
      out.p[nt] = half_terms(x.x, x.y, part);
    }
    return out;
  }

  // lane L addresses token L % 16 of chunk 2 j (lanes 0..15) or 2 j + 1: a
  // transposed matrix of 16-bit pairs, dims 2 g and 2 g + 1 of tokens 2 q, 2 q + 1
  static __device__ __forceinline__ void add_values(Ring& ws, int stage, int lane,
                                                    const Weights& weights, State& st) {
    #pragma unroll
    for (int j = 0; j < 2; ++j) {
      // from zero, and added up in FP32: a tensor-core sum drops the bits below
      // its accumulator's last one, always downwards
      float o[2][4] = {};
      #pragma unroll
      for (int e = 0; e < kStagePages; ++e) {
        uint32_t v[4];
        ldsm_x4_trans(v, smem_u32(ws.tile[stage][e]) + kCodeBytes + lane * 16 +
                             2 * j * kChunkBytes);
        #pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t lo = __byte_perm(v[2 * h], 0u, 0x3120);       // tokens 0..7
          const uint32_t hi = __byte_perm(v[2 * h + 1], 0u, 0x3120);   // tokens 8..15
          mma_f16(o[h], codes_to_half2<0>(lo), codes_to_half2<1>(lo), codes_to_half2<0>(hi),
                  codes_to_half2<1>(hi), weights.p[2 * e], weights.p[2 * e + 1]);
        }
      }
      #pragma unroll
      for (int h = 0; h < 2; ++h) {
        float* sum_o = st.o[2 * j + h];
        const float2 a = __fadd2_rn(make_float2(sum_o[0], sum_o[1]), make_float2(o[h][0], o[h][1]));
        const float2 b = __fadd2_rn(make_float2(sum_o[2], sum_o[3]), make_float2(o[h][2], o[h][3]));
        sum_o[0] = a.x;
        sum_o[1] = a.y;
        sum_o[2] = b.x;
        sum_o[3] = b.y;
      }
    }
  }
  // A group of pages; at least one token counts.
  template <bool kRope>
  static __device__ __forceinline__ void attend(Ring& ws, int stage, uint32_t seen, int lane,
                                                const Queries& q, State& st) {
    Scores scores;
    scores_of<kRope>(ws, stage, lane, q, scores);
    __syncwarp();
    add_values(ws, stage, lane, weights_of(ws, seen, lane, q, scores, st), st);
  }
  static __device__ __forceinline__ float largest(const float2 (&x)[kTiles]) {
    float m = fmaxf(x[0].x, x[0].y);
    #pragma unroll
    for (int i = 1; i < kTiles; ++i)
      m = max3(m, __float_as_uint(x[i].x), __float_as_uint(x[i].y));
    return m;
  }

  // The warp's part for the block merge.
  template <class Smem>
  static __device__ __forceinline__ void finish(Smem& sm, State& st, int warp, int lane) {
    const int g8 = lane >> 2;
    const int qq = lane & 3;
    st.l_run += __shfl_xor_sync(0xffffffffu, st.l_run, 1);
    st.l_run += __shfl_xor_sync(0xffffffffu, st.l_run, 2);
    st.rescale(inverse_scale_of(__float_as_uint(fabsf(st.unit)) >> 23), lane);
    if (qq == 0 && g8 < kGroup) {
      sm.m[warp][g8] = st.m_run;
      sm.l[warp][g8] = st.l_run;
    }
    #pragma unroll
    for (int c = 0; c < 4; ++c) {
      // columns 2 q, 2 q + 1 and their low parts' 2 q + 4, 2 q + 5
      #pragma unroll
      for (int e = 0; e < 4; ++e)
        st.o[c][e] += __shfl_xor_sync(0xffffffffu, st.o[c][e], 2);
      if (qq < 2) {
        #pragma unroll
        for (int e = 0; e < 2; ++e)
          *reinterpret_cast<float2*>(&sm.acc[warp][2 * qq + e][16 * c + 2 * g8]) =
              make_float2(st.o[c][e], st.o[c][e + 2]);
      }
    }
  }
};
static_assert(4 * (kTicketSmemBytes<QuantTiles> + 1024) <= kSmemPerSm, "4 ticket blocks per SM");
static_assert(3 * (kClusterSmemBytes<QuantTiles> + 1024) <= kSmemPerSm, "3 cluster blocks per SM");
static_assert(sizeof(WindowSmem<QuantTiles>) % 16 == 0,
              "the cluster inbox follows 16-byte aligned");

template <bool kFused>
pkv_status launch_quant(pkv_pool_t pool, int layer, const void* q, const void* k, const void* v,
                        const void* kv_pool, const int32_t* block_tables,
                        const int32_t* seq_lens, float* out, int window, int sinks,
                        const pkv_axes_rope* rope, const int32_t* rope_positions,
                        int position_stride, int batch, int num_splits, void* stream) {
  auto source = [&](QuantTiles::Source& src) {
    src.pool = const_cast<uint8_t*>(static_cast<const uint8_t*>(kv_pool));
    return true;
  };
  return launch_window<QuantTiles, kFused>(
      pool, layer, q, k, v, kv_pool && pkv_aligned16(kv_pool), source, block_tables, seq_lens,
      out, window, sinks, rope, rope_positions, position_stride, batch, num_splits, stream);
}

}  // namespace

bool pkv_quant_setup(pkv_pool* pool) { return setup_window<QuantTiles>(&pool->quant); }

extern "C" {

pkv_status pkv_quant_attention(pkv_pool_t pool, int layer, const void* q, const void* kv_pool,
                               const int32_t* block_tables, const int32_t* seq_lens, float* out,
                               int window, int sinks, const pkv_axes_rope* rope,
                               const int32_t* rope_positions, int position_stride, int batch,
                               int num_splits, void* stream) {
  return launch_quant<false>(pool, layer, q, nullptr, nullptr, kv_pool, block_tables, seq_lens,
                             out, window, sinks, rope, rope_positions, position_stride, batch,
                             num_splits, stream);
}

pkv_status pkv_quant_append_attend(pkv_pool_t pool, int layer, const void* q, const void* k,
                                   const void* v, void* kv_pool, const int32_t* block_tables,
                                   const int32_t* seq_lens, float* out, int window, int sinks,
                                   const pkv_axes_rope* rope, const int32_t* rope_positions,
                                   int position_stride, int batch, int num_splits, void* stream) {
  return launch_quant<true>(pool, layer, q, k, v, kv_pool, block_tables, seq_lens, out, window,
                            sinks, rope, rope_positions, position_stride, batch, num_splits,
                            stream);
}

}  // extern "C"
