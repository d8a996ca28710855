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

struct alignas(1024) WindowSmem {
  PageRing<kStagesW> warp[kWarps];
  unsigned long long bar[kWarps][kStagesW];
  float m[kWarps][kGroup];
  float l[kWarps][kGroup];
  float acc[kWarps][kGroup][kDim];   // the warps' partial outputs (block merge)
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
  int num_splits;             // ranges per sequence (and gridDim.x)
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

// x = hi + mid + lo with hi and mid truncated to BF16 (exact differences) and
// lo rounded: two values at a time, packed as BF16 pairs.
__device__ __forceinline__ void split3(float x0, float x1, uint32_t& hi, uint32_t& mid,
                                       uint32_t& lo) {
  const uint32_t b0 = __float_as_uint(x0), b1 = __float_as_uint(x1);
  hi = __byte_perm(b0, b1, 0x7632);
  const float r0 = x0 - __uint_as_float(b0 & 0xffff0000u);
  const float r1 = x1 - __uint_as_float(b1 & 0xffff0000u);
  const uint32_t c0 = __float_as_uint(r0), c1 = __float_as_uint(r1);
  mid = __byte_perm(c0, c1, 0x7632);
  lo = float2_to_bf16x2(r0 - __uint_as_float(c0 & 0xffff0000u),
                        r1 - __uint_as_float(c1 & 0xffff0000u));
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
      const float c0 = __shfl_sync(0xffffffffu, c, pair), c1 = __shfl_sync(0xffffffffu, c, pair + 1);
      const float s0 = __shfl_sync(0xffffffffu, s, pair), s1 = __shfl_sync(0xffffffffu, s, pair + 1);
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

// One page: K tile kt and V tile vt (swizzled, in shared memory), bit t of
// `seen` = token t counts (at least one does). The scores of the others are
// dropped by select; their V rows must hold finite values. Lanes L and L + 16
// hold the same scores, maximum and sum of head (L / 4) % 4.
template <bool kRope>
__device__ __forceinline__ void attend_page(const uint8_t* kt, const uint8_t* vt, uint32_t seen,
                                            int lane, const uint32_t (&qa)[8],
                                            const uint32_t (&ql)[8], MmaState& st) {
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
    // the accumulators' rows belong to the same head in every lane
    #pragma unroll
    for (int j = 0; j < 8; ++j) {
      st.o[j][0] *= alpha;
      st.o[j][1] *= alpha;
      st.o[j][2] *= alpha;
      st.o[j][3] *= alpha;
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
    mma_rows16(st.o[2 * jj], pa[0], pl[0], pa[1], pl[1], bv[0], bv[1]);
    mma_rows16(st.o[2 * jj + 1], pa[0], pl[0], pa[1], pl[1], bv[2], bv[3]);
  }
}

// The lowest n bits (n clamped to 0 .. 16).
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : n >= kPage ? 0xffffu : (1u << n) - 1u;
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

  const int split = blockIdx.x;
  const int kvh = blockIdx.y;
  const int b = blockIdx.z;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  // Before the wait (programmatic dependent launch) this block reads only
  // seq_lens, the block table, the rotary inputs and pool rows below the
  // appended position.
  const int len = prm.seq_lens[b];
  if (len == 0) return;                                  // a padding row
  if (len < 0 || len > prm.max_seq_len) {
    if (split == 0 && kvh == 0 && threadIdx.x == 0) set_error(prm.err, kErrSeqLen);
    return;
  }
  float ang_c = 1.f, ang_s = 0.f;                        // the angle of pair `lane`
  if (kRope && !load_pair_angle(prm.rope, b, lane, ang_c, ang_s)) {
    if (split == 0 && kvh == 0 && threadIdx.x == 0) set_error(prm.err, kErrPosition);
    return;                                              // every block of the sequence
  }
  const int n_pages = (len + kPage - 1) / kPage;
  const int win_lo = max(len - prm.window, 0);           // first token of the window
  const int win_page = win_lo / kPage;
  const int sink_pages = min((prm.sinks + kPage - 1) / kPage, win_page);
  const int n_seen = sink_pages + n_pages - win_page;    // visible pages, >= 1
  const int chunk = (n_seen + prm.num_splits - 1) / prm.num_splits;
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

  PageRing<kStagesW>& ws = sm.warp[warp];
  unsigned long long* bars = sm.bar[warp];
  if (lane == 0) {
    for (int s = 0; s < kStagesW; ++s) mbar_init(&bars[s], 1);
    fence_mbar_init();
    if (warp == 0) {
      prefetch_tensormap(&tmap_k);
      prefetch_tensormap(&tmap_v);
    }
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
  // in 8..15), rotated, into the pool; kept to patch into the stage.
  uint4 new_val = make_uint4(0u, 0u, 0u, 0u);
  auto write_new_row = [&](int phys) {
    const int c = lane & 7;
    uint4 val = make_uint4(0u, 0u, 0u, 0u);
    if (lane < 16)
      val = __ldg(reinterpret_cast<const uint4*>(
          (lane >= 8 ? prm.v_new : prm.k_new) +
          (static_cast<size_t>(b) * kHkv + kvh) * kDim + c * 8));
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
    new_val = val;
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
  if (kFused && j_new >= 0 && j_new < n_prefetch)
    write_new_row(__shfl_sync(0xffffffffu, ids, j_new));
  uint32_t qa[8], ql[8];
  load_queries<kRope>(prm.q + (static_cast<size_t>(b) * kHq + kvh * kGroup) * kDim, lane, ang_c,
                      ang_s, qa, ql);

  MmaState st;
  st.reset();
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
      if (with_new && seen && lane < 16) {
        uint8_t* t = lane >= 8 ? ws.v[stage] : ws.k[stage];
        *reinterpret_cast<uint4*>(t + new_slot * kRowBytes +
                                  (((lane & 7) ^ (new_slot & 7)) << 4)) = new_val;
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
      if (kFused && next == j_new) write_new_row(phys);
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

  // the three parts' accumulators of a head: rows g, g + 4 (lane + 16), g + 8
  #pragma unroll
  for (int j = 0; j < 8; ++j) {
    #pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float o = st.o[j][e] + st.o[j][e + 2];
      st.o[j][e] = o + __shfl_xor_sync(0xffffffffu, o, 16);
    }
  }
  float M, L;
  float2 O;
  block_merge_mma<kWarps>(sm, st, warp, lane, M, L, O);
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

// Splits per sequence and whether they form a cluster. Enough blocks for one
// wave of resident ones, but at least 4 pages (one per warp) per block.
void plan_window(const pkv_pool* pool, int batch, int window, int sinks, int num_splits,
                 int* splits, bool* cluster) {
  const pkv_pool_config& c = pool->cfg;
  const int max_pages = c.max_seq_len / kPage;
  const int seen = std::min(max_pages, (sinks + kPage - 1) / kPage + (window - 1) / kPage + 2);
  int s = num_splits;
  if (s == 0) {
    const int rows = batch * kHkv;
    const int fill = std::max(1, pool->window_blocks_per_sm * pool->num_sms / rows);
    s = std::max(1, std::min({fill, (seen + kWarps - 1) / kWarps, c.max_splits}));
  }
  *splits = s;
  *cluster = s >= 2 && s <= pool->max_cluster;
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
      !pkv_aligned16(v_pool) || !pkv_aligned16(block_tables) || !pkv_aligned16(seq_lens) ||
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
  bool cluster = false;
  plan_window(pool, batch, prm.window, prm.sinks, num_splits, &prm.num_splits, &cluster);

  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(prm.num_splits, kHkv, batch);
  cfg.blockDim = dim3(kThreadsW, 1, 1);
  cfg.dynamicSmemBytes = cluster ? kClusterSmemBytes : kTicketSmemBytes;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attrs[2];
  int n_attrs = 0;
  if (cluster) {
    attrs[n_attrs].id = cudaLaunchAttributeClusterDimension;
    attrs[n_attrs].val.clusterDim.x = prm.num_splits;
    attrs[n_attrs].val.clusterDim.y = 1;
    attrs[n_attrs].val.clusterDim.z = 1;
    ++n_attrs;
  }
  if (c.flags & PKV_FLAG_PDL) {
    attrs[n_attrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attrs[n_attrs].val.programmaticStreamSerializationAllowed = 1;
    ++n_attrs;
  }
  cfg.attrs = attrs;
  cfg.numAttrs = n_attrs;
  CUtensorMap tk, tv;
  if (!pkv_pool_tensor_map(k_pool, c.num_pages, &tk) ||
      !pkv_pool_tensor_map(v_pool, c.num_pages, &tv))
    return PKV_ERR_CUDA;
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
