// Windowed decode attention over the paged KV cache for GB300 (sm_103a),
// with sinks, optional fused append and rotation by several position axes,
// for contexts of up to a million tokens (declared in include/pkv_window.h).
//
// out = sum_t p_t V_t / sum_t p_t, p_t = 2^(q.K_t log2(e) / 8 - m), over the
// visible tokens: one pass with a running maximum m and sum.
//
// The kernel is window_device.cuh's; here are the BF16 pages' tiles and their
// products.
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

#include "pkv.h"
#include "pkv_window.h"
#include "window_device.cuh"

using namespace pkv_window;

namespace {

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
  __device__ __forceinline__ void reset() {
    #pragma unroll
    for (int j = 0; j < 8; ++j) o[j][0] = o[j][1] = 0.f;
    m_run = -INFINITY;
    l_run = 0.f;
  }
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

// ---------------------------------------------------------------- tiles
// A page of one KV head: its K and V tiles, 2 KiB each.
struct Bf16Tiles {
  static constexpr int kStages = 3;
  static constexpr int kStagePages = 1;
  static constexpr int kParts = 2;              // K and V
  static constexpr uint32_t kCopyBytes = 2 * kTileBytes;
  using Ring = PageRing<kStages>;
  using State = PageState;
  struct Source {
    CUtensorMap k, v;
    uint16_t* k_pool;           // [num_pages][8][16][64]
    uint16_t* v_pool;
  };
  struct Queries {
    uint32_t a[8], l[8];
  };

  static const WindowResidency& residency(const pkv_pool* pool) { return pool->window; }
  // Measured (us): one 2,048-token sequence, cluster of 12 5.7, units 6.8; 4
  // sequences at a 1,024-token window 6.0 and 6.9, with 16 (not all resident at
  // once) 9.4. One 131,072-token sequence, cluster of 12 120.6, units 48.0.
  static int cluster_size(long long, long long) { return 12; }
  static bool fills(long long blocks, long long slots) { return 2 * blocks >= slots; }

  static __device__ __forceinline__ void prefetch(const Source& src) {
    prefetch_tensormap(&src.k);
    prefetch_tensormap(&src.v);
  }
  static __device__ __forceinline__ void copy(Ring& ws, int stage, int, const Source& src, int part,
                                              int kvh, int phys, unsigned long long* bar) {
    tma_load_tile(part == 0 ? ws.k[stage] : ws.v[stage], part == 0 ? &src.k : &src.v,
                  kvh * kPage, phys, bar);
  }
  static __device__ __forceinline__ void hide_rows(Ring& ws, int stage, uint32_t seen, int lane) {
    uint8_t* vt = ws.v[stage];
    for (int idx = lane; idx < kPage * 8; idx += 32)
      if (!((seen >> (idx >> 3)) & 1u))
        *reinterpret_cast<uint4*>(vt + idx * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
  // The appended row, a 16-byte chunk per lane: K in lanes 0..7, V in 8..15. All is
  // done at its page's turn (64 ragged sequences behind 1,024 tokens: 15.6 us; the
  // rotation done ahead, 15.9).
  struct NewRow {
    uint4 val;
    float ang_c, ang_s;
  };
  template <bool kRope>
  static __device__ __forceinline__ NewRow make_row(const Source&, int, int, int, bool, uint4 val,
                                                    float ang_c, float ang_s, int) {
    return {val, ang_c, ang_s};
  }
  // Rotated, into its slot of the pool and of the stage.
  template <bool kRope>
  static __device__ __forceinline__ void put_row(Ring& ws, int stage, int, const Source& src,
                                                 int kvh, int slot, int phys, bool to_pool,
                                                 bool to_stage, const NewRow& made, int lane) {
    const int c = lane & 7;
    uint4 val = made.val;
    if (kRope) {
      const uint4 partner = shfl_xor_uint4(val, 4);
      float cs[8], sn[8];
      #pragma unroll
      for (int e = 0; e < 8; ++e) {
        cs[e] = __shfl_sync(0xffffffffu, made.ang_c, 8 * (c & 3) + e);
        sn[e] = __shfl_sync(0xffffffffu, made.ang_s, 8 * (c & 3) + e);
      }
      if (lane < 8) val = rope_key_chunk(val, partner, c >= 4, cs, sn);
    }
    if (lane < 16 && to_pool)
      *reinterpret_cast<uint4*>((lane >= 8 ? src.v_pool : src.k_pool) +
                                ((static_cast<size_t>(phys) * kHkv + kvh) * kPage + slot) * kDim +
                                c * 8) = val;
    if (lane < 16 && to_stage) {
      uint8_t* t = lane >= 8 ? ws.v[stage] : ws.k[stage];
      *reinterpret_cast<uint4*>(t + slot * kRowBytes + ((c ^ (slot & 7)) << 4)) = val;
    }
  }
  template <bool kRope>
  static __device__ __forceinline__ void load_queries(const uint16_t* qrow, int lane, float c,
                                                      float s, Queries& q) {
    ::load_queries<kRope>(qrow, lane, c, s, q.a, q.l);
  }
  template <bool kRope>
  static __device__ __forceinline__ void attend(Ring& ws, int stage, uint32_t seen, int lane,
                                                const Queries& q, State& st) {
    attend_page<kRope>(ws.k[stage], ws.v[stage], seen, lane, q.a, q.l, st);
  }
  // The warp's part for the block merge.
  template <class Smem>
  static __device__ __forceinline__ void finish(Smem& sm, const State& st, int warp, int lane) {
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
    block_merge_store(sm, total, warp, lane);
  }
};
static_assert(4 * (kTicketSmemBytes<Bf16Tiles> + 1024) <= kSmemPerSm, "4 ticket blocks per SM");
static_assert(3 * (kClusterSmemBytes<Bf16Tiles> + 1024) <= kSmemPerSm, "3 cluster blocks per SM");
static_assert(sizeof(WindowSmem<Bf16Tiles>) % 16 == 0,
              "the cluster inbox follows 16-byte aligned");

template <bool kFused>
pkv_status launch_bf16(pkv_pool_t pool, int layer, const void* q, const void* k, const void* v,
                       const void* k_pool, const void* v_pool, const int32_t* block_tables,
                       const int32_t* seq_lens, float* out, int window, int sinks,
                       const pkv_axes_rope* rope, const int32_t* rope_positions,
                       int position_stride, int batch, int num_splits, void* stream) {
  auto source = [&](Bf16Tiles::Source& src) {
    src.k_pool = const_cast<uint16_t*>(static_cast<const uint16_t*>(k_pool));
    src.v_pool = const_cast<uint16_t*>(static_cast<const uint16_t*>(v_pool));
    return pkv_pool_tensor_map(k_pool, pool->cfg.num_pages, &src.k) &&
           pkv_pool_tensor_map(v_pool, pool->cfg.num_pages, &src.v);
  };
  return launch_window<Bf16Tiles, kFused>(
      pool, layer, q, k, v,
      k_pool && v_pool && pkv_aligned16(k_pool) && pkv_aligned16(v_pool), source, block_tables,
      seq_lens, out, window, sinks, rope, rope_positions, position_stride, batch, num_splits,
      stream);
}

}  // namespace

bool pkv_window_setup(pkv_pool* pool) { return setup_window<Bf16Tiles>(&pool->window); }

extern "C" {

pkv_status pkv_window_attention(pkv_pool_t pool, int layer, const void* q, const void* k_pool,
                                const void* v_pool, const int32_t* block_tables,
                                const int32_t* seq_lens, float* out, int window, int sinks,
                                const pkv_axes_rope* rope, const int32_t* rope_positions,
                                int position_stride, int batch, int num_splits, void* stream) {
  return launch_bf16<false>(pool, layer, q, nullptr, nullptr, k_pool, v_pool, block_tables,
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
  return launch_bf16<true>(pool, layer, q, k, v, k_pool, v_pool, block_tables, seq_lens, out,
                             window, sinks, rope, rope_positions, position_stride, batch,
                             num_splits, stream);
}

}  // extern "C"
