// Attention of small drafted trees over the paged KV cache for GB300 (sm_103a):
// pkv_tree_attention's kernel where a sequence brings few drafted tokens (declared
// in include/pkv_tree.h; larger trees: tree.cu).
//
// out_i = sum_t p_it V_t / sum_t p_it, p_it = 2^(q_i.K_t log2(e) / 8 - m_i), over
// the tokens that row i sees: one pass with a running maximum m_i and sum.
//
// A tile is up to 4 or 8 drafted tokens of a sequence and KV head: 16 or 32 rows. That
// fills a quarter of a tcgen05 product's rows at most, and a CTA of that kernel takes
// 4 us before its first scores (its roles, tensor memory and first instructions). Here a
// block is four warps like the decode's: each takes every fourth page through its own
// ring of tiles and does all rows' products by warp-wide mma.sync, which needs no
// set-up. The tiles' steps (four pages, one per warp) are shared out and joined as in
// tree.cu, or, where the tiles are few and short, by a cluster of blocks per tile that
// joins its parts through shared memory, without a second launch.
//
// What bounds it: mma.sync, 64 products a page for 32 rows and 32 for up to 16 (three
// BF16 terms of the weights), 8 cycles each on a quarter of an SM: three warps there
// take a page each in about 2,000 cycles, 1,536 of them products, where the decode's
// four rows hide under the copies. So it serves few tokens: one tree of 8 over 2,000
// tokens 7.4 us (tcgen05 12.9), 128 trees of 4 over 2,000 90 us (119; the bytes alone
// 80); which calls it takes is decided in tree.cu. Many short sequences are bound by the
// start and the end of their tiles, some 5 us each for a block: 1,024 trees of 4 over
// 300 tokens 130 us (the bytes 103), 4,096 of 2 over 64 310 (98). One tree of 8 over 2,000
// tokens is latency: on the line 8.3 us, the join 2 of them, in clusters of 16 7.4;
// without the products 5.3. (Blocks of 8 warps, one an SM: 11.9, not all of their
// clusters of 16 are resident at once.)

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "pkv.h"
#include "pkv_tree.h"
#include "decode_device.cuh"
#include "device_common.cuh"
#include "pool_internal.h"
#include "tree.cuh"

using namespace pkv_tree_dev;

namespace {

// A tile of kHalves x 16 rows: 4 or 8 drafted tokens.
template <int kHalves>
constexpr int kFewTokens = 16 * kHalves / kGroup;
template <int kHalves>
constexpr int kFewRowsN = 16 * kHalves;
constexpr int kFewWarps = 4;
constexpr int kFewThreads = kFewWarps * 32;
constexpr int kFewStages = 3;
template <int kHalves>
constexpr int kFewBlocksPerSm = kHalves == 1 ? 4 : 3;   // by their registers
constexpr int kFewTileBytes = kPage * kRowBytes;     // K or V of a page: 2 KiB
constexpr int kAccStride = kDim + 4;                 // floats of a merged row: no bank conflicts
static_assert(kFewWarps == kStepPages, "a step's pages go to a warp each");

template <int kHalves>
struct alignas(1024) FewSmem {
  pkv_decode::PageRing<kFewStages> warp[kFewWarps];  // at a part's end: the warp's sums
  uint4 q[4 * kHalves][32];                          // the rows as operand fragments, by lane
  unsigned long long mask[kFewTokens<kHalves>];
  unsigned long long bar[kFewWarps][kFewStages];
  float m[kFewWarps][kFewRowsN<kHalves>];
  float l[kFewWarps][kFewRowsN<kHalves>];
  int abort;
};
template <int kHalves>
constexpr size_t kFewSmemBytes = sizeof(FewSmem<kHalves>) + 1024;   // + room to align the base
static_assert(sizeof(pkv_decode::PageRing<kFewStages>) >=
                  kFewRowsN<2> * kAccStride * sizeof(float),
              "a warp's sums fit its ring");
static_assert(kFewBlocksPerSm<1> * (kFewSmemBytes<1> + 1024) <= 228 * 1024 &&
                  kFewBlocksPerSm<2> * (kFewSmemBytes<2> + 1024) <= 228 * 1024,
              "blocks per SM");

__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Parts of a cluster's rows, each at the block that ends the row: block r % S ends row
// r, which finds part p of it in slot r / S * S + p.
struct alignas(16) RowInbox {
  float o[kFewRowsN<2>][kDim];
  float2 ml[kFewRowsN<2>];
  unsigned long long bar;
};
constexpr int kMaxParts = 16;
constexpr uint32_t kRowPartBytes = (kDim + 2) * sizeof(float);
constexpr int kPartTokens = 512;
constexpr size_t kClusterSmemBytes = kFewSmemBytes<2> + sizeof(RowInbox);
static_assert(kFewBlocksPerSm<2> * (kClusterSmemBytes + 1024) <= 228 * 1024, "blocks per SM");
static_assert(sizeof(FewSmem<2>) % 16 == 0 && kFewRowsN<2> % kMaxParts == 0, "the inbox's place");

// Asynchronous store of four floats into another block's shared memory, completing 16
// transaction bytes on that block's mbarrier `rbar`.
__device__ __forceinline__ void st_async4(uint32_t raddr, float4 v, uint32_t rbar) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];"
      ::"r"(raddr), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(rbar)
      : "memory");
}

// The rows of a tile (count of them) that this block ends, once all parts have landed
// (a bounded wait): a warp a row, two dims a lane.
__device__ __forceinline__ void end_rows(RowInbox& inbox, const TreeWork& work, float* out,
                                         int* err, int warp, int lane) {
  const int S = gridDim.x, rank = blockIdx.x;
  const int rows = work.count * kGroup;
  if (rank + warp * S >= rows) return;
  if (!__all_sync(0xffffffffu, pkv_decode::mbar_wait_cluster(&inbox.bar, 0))) {
    if (lane == 0) set_error(err, PKV_DEV_ERR_TIMEOUT);
    return;
  }
  for (int i = warp; rank + i * S < rows; i += kFewWarps) {
    const float2 part = lane < S ? inbox.ml[i * S + lane] : make_float2(-INFINITY, 0.f);
    float most = part.x;
    #pragma unroll
    for (int o = 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    const float w = part.x == -INFINITY ? 0.f : fast_exp2(part.x - most);
    float l = w * part.y;
    #pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
    float2 sum = make_float2(0.f, 0.f);
    #pragma unroll
    for (int p = 0; p < kMaxParts; ++p)
      if (p < S) {
        const float wp = __shfl_sync(0xffffffffu, w, p);
        const float2 x = *reinterpret_cast<const float2*>(&inbox.o[i * S + p][2 * lane]);
        sum.x += wp * x.x;
        sum.y += wp * x.y;
      }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const int r = rank + i * S;
    *reinterpret_cast<float2*>(
        out +
        ((static_cast<size_t>(work.row) + (r >> 2)) * kHq + work.g * kGroup + (r & 3)) * kDim +
        2 * lane) = make_float2(sum.x * inv, sum.y * inv);
  }
}

__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}

// A warp's sums over its pages. Lane (g, q) = (L / 4, L % 4) holds rows 16 t + g
// (o[t][n][0, 1]) and 16 t + 8 + g ([2, 3]), dims 8 n + 2 q, + 1; row r is drafted
// token r / 4 of the tile, head r % 4. m and l of row 16 t + 8 h + g in [2 t + h].
template <int kHalves>
struct FewState {
  float o[kHalves][8][4];
  // Base-2 exponent the row's weights are taken against, p <= 2^8. NaN where it is huge
  // (device_common.cuh): it is then kept in shared memory, and each page's scores are
  // replaced by what they differ from it, where the test that a page needs anyway leads.
  // (That costs 32 trees of 8 over 2,000 tokens 2 %; a test for each page, with a factor and a
  // maximum to choose, 7 %; a second copy of the page's arithmetic 4 %.)
  float m[2 * kHalves];
  float l[2 * kHalves];   // this lane's share of the row's sum
  __device__ __forceinline__ void reset() {
    #pragma unroll
    for (int t = 0; t < kHalves; ++t)
      #pragma unroll
      for (int n = 0; n < 8; ++n)
        #pragma unroll
        for (int e = 0; e < 4; ++e) o[t][n][e] = 0.f;
    #pragma unroll
    for (int i = 0; i < 2 * kHalves; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
    }
  }
};

// One page, K tile kt and V tile vt (swizzled). kTiles: halves that have rows. seen:
// what each of this lane's rows sees of it, 16 bits, where not `whole`; V rows that no
// row sees hold zeros. huge_m: the warp's rows' exponents where they are huge.
template <int kTiles, int kHalves>
__device__ __forceinline__ void attend_rows(const uint8_t* kt, const uint8_t* vt, bool whole,
                                            const uint32_t (&seen)[2 * kHalves],
                                            const uint4 (*q)[32], float* huge_m, int lane,
                                            FewState<kHalves>& st) {
  const int g8 = lane >> 2;
  const int qq = lane & 3;
  // scores; slice s of the contraction is dims 16 q + 4 s .. + 3 of lane q, so a
  // lane's fragments of a K row are 32 contiguous bytes (as in decode_device.cuh)
  float s[kTiles][2][4];
  {
    uint32_t kw[2][8];
    #pragma unroll
    for (int nt = 0; nt < 2; ++nt) {
      const uint8_t* row = kt + (8 * nt + g8) * kRowBytes;
      const uint4 k0 = *reinterpret_cast<const uint4*>(row + (((2 * qq) ^ g8) << 4));
      const uint4 k1 = *reinterpret_cast<const uint4*>(row + (((2 * qq + 1) ^ g8) << 4));
      kw[nt][0] = k0.x; kw[nt][1] = k0.y; kw[nt][2] = k0.z; kw[nt][3] = k0.w;
      kw[nt][4] = k1.x; kw[nt][5] = k1.y; kw[nt][6] = k1.z; kw[nt][7] = k1.w;
    }
    #pragma unroll
    for (int t = 0; t < kTiles; ++t) {
      #pragma unroll
      for (int nt = 0; nt < 2; ++nt) s[t][nt][0] = s[t][nt][1] = s[t][nt][2] = s[t][nt][3] = 0.f;
      #pragma unroll
      for (int half = 0; half < 2; ++half) {       // dims 8 half .. + 7 of each lane's 16
        const uint4 lo = q[4 * t + half][lane], hi = q[4 * t + 2 + half][lane];   // rows g, g + 8
        const uint32_t a[2][4] = {{lo.x, hi.x, lo.y, hi.y}, {lo.z, hi.z, lo.w, hi.w}};
        #pragma unroll
        for (int e = 0; e < 2; ++e)
          #pragma unroll
          for (int nt = 0; nt < 2; ++nt)
            mma_16816(s[t][nt], a[e], kw[nt][4 * half + 2 * e], kw[nt][4 * half + 2 * e + 1]);
      }
    }
  }
  if (!whole) {
    #pragma unroll
    for (int t = 0; t < kTiles; ++t)
      #pragma unroll
      for (int nt = 0; nt < 2; ++nt)
        #pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!((seen[2 * t + e / 2] >> (8 * nt + 2 * qq + e % 2)) & 1u)) s[t][nt][e] = -INFINITY;
  }
  const float c = 1.4426950408889634f * 0.125f;   // log2(e) / sqrt(64)
  float top[2 * kTiles];
  bool grow = false;
  #pragma unroll
  for (int i = 0; i < 2 * kTiles; ++i) {
    const int t = i / 2, h = 2 * (i % 2);
    top[i] = fmaxf(fmaxf(s[t][0][h], s[t][0][h + 1]), fmaxf(s[t][1][h], s[t][1][h + 1])) * c;
    grow |= !(top[i] <= st.m[i] + pkv_decode::kRescaleLog2);
  }
  // a row's exponent moves only when its maximum grows by more than 2^8
  if (__any_sync(0xffffffffu, grow)) {
    bool huge = false;
    #pragma unroll
    for (int i = 0; i < 2 * kTiles; ++i) {
      const float most = quad_max(top[i]);
      const float kept = huge_m[8 * i + g8];     // read in any case: no branch
      float m = st.m[i];
      if (m != m) m = kept;
      if (most > m + pkv_decode::kRescaleLog2) {
        const float alpha = fast_exp2(m - most);         // 0 on the first page
        st.m[i] = m = most;
        st.l[i] *= alpha;
        #pragma unroll
        for (int n = 0; n < 8; ++n) {
          st.o[i / 2][n][2 * (i % 2)] *= alpha;
          st.o[i / 2][n][2 * (i % 2) + 1] *= alpha;
        }
      }
      top[i] = m;
      huge |= is_huge(m);
    }
    if (rarely(huge)) {
      #pragma unroll
      for (int i = 0; i < 2 * kTiles; ++i) {
        const float m = top[i];
        if (!is_huge(m)) continue;
        huge_m[8 * i + g8] = m;          // the row's four lanes agree
        st.m[i] = NAN;
        #pragma unroll
        for (int nt = 0; nt < 2; ++nt)
          #pragma unroll
          for (int e = 0; e < 2; ++e) {
            float& x = s[i / 2][nt][2 * (i % 2) + e];
            x = less(x, c, m) * (1.f / c);
          }
      }
    }
  }
  // weights as three BF16 terms (24 bits): A fragments of rows g, g + 8 and tokens
  // 2 q, 2 q + 1, then 8 + 2 q, 9 + 2 q, where the scores' accumulators hold them
  uint32_t p[kTiles][3][4];
  const float2 c2 = make_float2(c, c);
  #pragma unroll
  for (int t = 0; t < kTiles; ++t)
    #pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float mu = st.m[2 * t + h] > -INFINITY ? st.m[2 * t + h] : 0.f;
      const float2 minus = make_float2(-mu, -mu);
      float2 sum = make_float2(0.f, 0.f);
      #pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        const float2 x = __ffma2_rn(make_float2(s[t][nt][2 * h], s[t][nt][2 * h + 1]), c2, minus);
        const float2 pp = make_float2(fast_exp2(x.x), fast_exp2(x.y));
        sum = __fadd2_rn(sum, pp);
        split3(pp.x, pp.y, p[t][0][2 * nt + h], p[t][1][2 * nt + h], p[t][2][2 * nt + h]);
      }
      st.l[2 * t + h] += sum.x + sum.y;
    }
  // values: a page's products start from zero and are added up in FP32
  const int mrow = lane & 7;
  const int mat = lane >> 3;
  const uint32_t vrow = smem_u32(vt) + (mrow + 8 * (mat & 1)) * kRowBytes;
  #pragma unroll
  for (int jj = 0; jj < 4; ++jj) {
    uint32_t v[4];
    pkv_decode::ldsm_x4_trans(v, vrow + (((2 * jj + (mat >> 1)) ^ mrow) << 4));
    #pragma unroll
    for (int h = 0; h < 2; ++h)
      #pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        #pragma unroll
        for (int part = 0; part < 3; ++part) mma_16816(d, p[t][part], v[2 * h], v[2 * h + 1]);
        float* o = st.o[t][2 * jj + h];
        const float2 a = __fadd2_rn(make_float2(o[0], o[1]), make_float2(d[0], d[1]));
        const float2 b = __fadd2_rn(make_float2(o[2], o[3]), make_float2(d[2], d[3]));
        o[0] = a.x;
        o[1] = a.y;
        o[2] = b.x;
        o[3] = b.y;
      }
  }
}

// kCluster: grid (parts, KV heads, tiles), a tile's parts in a cluster; otherwise the
// blocks share the line.
template <int kHalves, bool kCluster>
__global__ void __launch_bounds__(kFewThreads, kFewBlocksPerSm<kHalves>) tree_few_kernel(
    const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
    const uint16_t* __restrict__ q, const TreeParams prm) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  constexpr int kTokens = kFewTokens<kHalves>, kRowsN = kFewRowsN<kHalves>;
  using Smem = FewSmem<kHalves>;
  Smem& sm = *reinterpret_cast<Smem*>(
      smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u));
  RowInbox& inbox = *reinterpret_cast<RowInbox*>(&sm + 1);     // kCluster
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int g8 = lane >> 2;
  const int qq = lane & 3;
  const int kvh = kCluster ? blockIdx.y : blockIdx.x % kHkv;
  pkv_decode::PageRing<kFewStages>& ring = sm.warp[warp];
  unsigned long long* bars = sm.bar[warp];
  // the kernel that joins the parts may be made ready (it waits for this one's end)
  if (!kCluster) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // every warp walks the line for itself
  TreeWalk<kTokens> walk;
  TreeLane<kTokens> lists;
  if constexpr (kCluster)
    lists.load(prm, lane, blockIdx.x + blockIdx.y + blockIdx.z == 0);
  else
    walk.fetch(prm, lane);
  if (lane == 0) {
    for (int s = 0; s < kFewStages; ++s) mbar_init(&bars[s], 1);
    fence_mbar_init();
    if (warp == 0) {
      pkv_decode::prefetch_tensormap(&tmap_k);
      pkv_decode::prefetch_tensormap(&tmap_v);
      sm.abort = 0;
    }
  }
  __syncwarp();

  uint32_t used = 0;                  // pages that went through the ring
  TreeWork work;
  auto next = [&]() {
    if constexpr (!kCluster) return walk.next(0, prm, lane, work);
    work.g = kvh;
    // the same decision in every block of the cluster; returns after its one part
    return part_of_tile<kTokens>(prm, lists, blockIdx.z, blockIdx.x, gridDim.x, lane, work);
  };
  while (next()) {
    if constexpr (kCluster) {
      const int S = gridDim.x, rank = blockIdx.x;
      const int ends = max(work.count * kGroup - rank + S - 1, 0) / S;     // rows
      if (threadIdx.x == 0 && ends > 0) {
        mbar_init(&inbox.bar, 1);
        fence_mbar_init();
        mbar_arrive_expect_tx(&inbox.bar, ends * S * kRowPartBytes);
      }
      __syncwarp();
      pkv_decode::cluster_arrive_release();
    }
    const TreeView view(work, prm);
    const int mine = work.steps;      // this warp's pages: one of every step
    const int32_t* row = prm.table + static_cast<size_t>(work.b) * prm.table_stride;
    auto list_at = [&](int j) { return (work.step + j) * kStepPages + warp; };
    // physical ids of 32 of this warp's pages, one per lane (the next 32 on their
    // way): -1 invalid, -2 no such page or no token that counts
    auto fetch_ids = [&](int base) {
      int id = -2;
      if (base + lane < mine && view.has_page(list_at(base + lane))) {
        id = __ldg(row + view.page(list_at(base + lane)));
        if (id < 0 || id >= prm.num_pages) id = -1;
      }
      return id;
    };
    int ids = fetch_ids(0);
    int ids_next = fetch_ids(32);
    // the rows and what they see, for all warps: fragment c of lane (g, q) holds dims
    // 16 q + 8 (c % 2) .. + 7 of row 16 (c / 4) + 8 (c / 2 % 2) + g
    #pragma unroll
    for (int e = 0; e < kHalves; ++e) {
      const int c = kHalves * warp + e;
      const int r = 16 * (c >> 2) + 8 * (c >> 1 & 1) + g8;
      const int token = work.row + min(r >> 2, work.count - 1);   // past the end: the last one's
      sm.q[c][lane] = __ldg(reinterpret_cast<const uint4*>(
          q + (static_cast<size_t>(token) * kHq + kvh * kGroup + (r & 3)) * kDim + 16 * qq +
          8 * (c & 1)));
    }
    if (threadIdx.x < kTokens)
      sm.mask[threadIdx.x] = prm.tree[work.row + min(static_cast<int>(threadIdx.x),
                                                     work.count - 1)];
    // Copy engine: K and V of page j into its stage, by one lane from operands that the
    // warp shares (those of a lane's own take a loop over the lanes).
    auto issue = [&](int j) {
      const int stage = (used + j) % kFewStages;
      const int id = __shfl_sync(0xffffffffu, ids, j & 31);
      if (elect_one()) {
        if (id >= 0) {
          mbar_arrive_expect_tx(&bars[stage], 2 * kFewTileBytes);
          pkv_decode::tma_load_tile(ring.k[stage], &tmap_k, kvh * kPage, id, &bars[stage]);
          pkv_decode::tma_load_tile(ring.v[stage], &tmap_v, kvh * kPage, id, &bars[stage]);
        } else {
          if (id == -1) set_error(prm.err, PKV_DEV_ERR_PAGE);
          mbar_arrive(&bars[stage]);
        }
      }
      __syncwarp();
    };
    int issued = min(mine, kFewStages);
    uint32_t good = __ballot_sync(0xffffffffu, ids >= 0);   // of the 32 pages in `ids`
    uint32_t good_now = good;                               // ... of the 32 being attended
    for (int j = 0; j < issued; ++j) issue(j);
    __syncthreads();

    FewState<kHalves> st;
    st.reset();
    int landed = 0;
    bool timed_out = sm.abort != 0;
    for (int j = 0; j < mine && !timed_out; ++j) {
      const uint32_t at = used + j;
      const int stage = at % kFewStages;
      if (!__all_sync(0xffffffffu, mbar_wait(&bars[stage], at / kFewStages & 1u))) {
        timed_out = true;
        break;
      }
      landed = j + 1;
      if ((j & 31) == 0) good_now = good;
      if (good_now >> (j & 31) & 1u) {
        const int i = list_at(j);
        const bool whole = i >= view.whole_from && i < view.whole_to;
        uint32_t seen[2 * kHalves];
        if (!whole) {
          const int base = view.page(i) * kPage;
          uint8_t* vt = ring.v[stage];
          bool cleared = false;
          for (int idx = lane; idx < kPage * 8; idx += 32)
            if (view.dead(base + (idx >> 3))) {
              *reinterpret_cast<uint4*>(vt + idx * 16) = make_uint4(0u, 0u, 0u, 0u);
              cleared = true;
            }
          if (cleared) pkv_prefill_dev::fence_proxy_async_smem();
          #pragma unroll
          for (int r = 0; r < 2 * kHalves; ++r) {
            const int token = 4 * (r >> 1) + 2 * (r & 1) + (g8 >> 2);
            seen[r] = TreeRow(work, prm, sm.mask[token]).seen(view, base);
          }
          __syncwarp();
        }
        if (kHalves == 2 && work.count > kTokens / 2)
          attend_rows<kHalves>(ring.k[stage], ring.v[stage], whole, seen, sm.q, sm.m[warp], lane,
                               st);
        else
          attend_rows<1>(ring.k[stage], ring.v[stage], whole, seen, sm.q, sm.m[warp], lane, st);
      }
      __syncwarp();   // every lane's reads of the stage are done before it is refilled
      const int next = j + kFewStages;
      if (next < mine) {
        if ((next & 31) == 0) {
          ids = ids_next;
          good = __ballot_sync(0xffffffffu, ids >= 0);
          ids_next = fetch_ids(next + 32);
        }
        issue(next);
        issued = next + 1;
      }
    }
    if (timed_out) {
      // this warp's copies in flight land before the block goes on (each wait bounded)
      for (int j = landed; j < issued; ++j)
        mbar_wait(&bars[(used + j) % kFewStages], (used + j) / kFewStages & 1u);
      if (lane == 0) {
        set_error(prm.err, PKV_DEV_ERR_TIMEOUT);
        sm.abort = 1;
      }
    }
    used += mine;

    // the warps' sums, each in its own ring (whose copies have all landed)
    float* acc = reinterpret_cast<float*>(&ring);
    #pragma unroll
    for (int i = 0; i < 2 * kHalves; ++i) {
      const int r = 8 * i + g8;
      float l = st.l[i];
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      if (qq == 0) {
        if (st.m[i] == st.m[i]) sm.m[warp][r] = st.m[i];
        sm.l[warp][r] = l;
      }
      #pragma unroll
      for (int n = 0; n < 8; ++n)
        *reinterpret_cast<float2*>(acc + r * kAccStride + 8 * n + 2 * qq) =
            make_float2(st.o[i / 2][n][2 * (i % 2)], st.o[i / 2][n][2 * (i % 2) + 1]);
    }
    __syncthreads();
    // the same decision in every warp; a cluster's other blocks expect their parts
    if (!kCluster && sm.abort) return;
    // every block's inbox is ready
    if constexpr (kCluster) pkv_decode::cluster_wait_acquire();
    // 8 threads a row, two float4 each, 16 rows at a time
    #pragma unroll
    for (int pass = 0; pass < kHalves; ++pass) {
      const int r = 16 * pass + (threadIdx.x >> 3), at = threadIdx.x & 7;
      if (r < work.count * kGroup) {
        float M = -INFINITY, L = 0.f;
        #pragma unroll
        for (int w = 0; w < kFewWarps; ++w) M = fmaxf(M, sm.m[w][r]);
        float4 sum[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
        #pragma unroll
        for (int w = 0; w < kFewWarps; ++w) {
          const float f = M == -INFINITY ? 0.f : fast_exp2(sm.m[w][r] - M);
          L += f * sm.l[w][r];
          const float4* o = reinterpret_cast<const float4*>(
              reinterpret_cast<const float*>(&sm.warp[w]) + r * kAccStride) + at;
          #pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float4 x = o[8 * h];
            sum[h].x += f * x.x;
            sum[h].y += f * x.y;
            sum[h].z += f * x.z;
            sum[h].w += f * x.w;
          }
        }
        if constexpr (kCluster) {
          const int S = gridDim.x;
          const uint32_t end = r % S;
          const int slot = r / S * S + blockIdx.x;
          const uint32_t rbar = pkv_decode::cluster_addr(&inbox.bar, end);
          #pragma unroll
          for (int h = 0; h < 2; ++h)
            st_async4(pkv_decode::cluster_addr(&inbox.o[slot][4 * at + 32 * h], end), sum[h], rbar);
          if (at == 0)
            pkv_decode::st_async2(pkv_decode::cluster_addr(&inbox.ml[slot], end),
                                  make_float2(M, L), rbar);
          continue;
        }
        float4* to;
        if (work.slot < 0) {
          const float inv = L > 0.f ? 1.f / L : 0.f;
          #pragma unroll
          for (int h = 0; h < 2; ++h)
            sum[h] = make_float4(sum[h].x * inv, sum[h].y * inv, sum[h].z * inv, sum[h].w * inv);
          to = reinterpret_cast<float4*>(
              prm.out + ((static_cast<size_t>(work.row) + (r >> 2)) * kHq + kvh * kGroup +
                         (r & 3)) * kDim);
        } else {
          const size_t at_row = static_cast<size_t>(work.slot) * kRowsN + r;
          to = reinterpret_cast<float4*>(prm.part_o + at_row * kDim);
          if (at == 0) prm.part_ml[at_row] = make_float2(M, L);
        }
        to[at] = sum[0];
        to[at + 8] = sum[1];
      }
    }
    if constexpr (kCluster) {
      end_rows(inbox, work, prm.out, prm.err, warp, lane);
      return;
    }
    // the rings are copied into again
    pkv_prefill_dev::fence_proxy_async_smem();
    __syncthreads();
  }
}

}  // namespace

bool pkv_tree_few_setup() {
  return cudaFuncSetAttribute(tree_few_kernel<1, false>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(kFewSmemBytes<1>)) == cudaSuccess &&
         cudaFuncSetAttribute(tree_few_kernel<2, false>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(kFewSmemBytes<2>)) == cudaSuccess &&
         cudaFuncSetAttribute(tree_few_kernel<2, true>,
                              cudaFuncAttributeMaxDynamicSharedMemorySize,
                              static_cast<int>(kClusterSmemBytes)) == cudaSuccess &&
         cudaFuncSetAttribute(tree_few_kernel<2, true>,
                              cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
}

template <int kHalves>
static pkv_status launch_line(pkv_pool_t pool, const void* q, const CUtensorMap& tk,
                              const CUtensorMap& tv, TreeParams prm, cudaStream_t st) {
  set_wave(&prm, kFewBlocksPerSm<kHalves> * pool->num_sms);
  tree_few_kernel<kHalves, false><<<prm.wave * kHkv, kFewThreads, kFewSmemBytes<kHalves>, st>>>(
      tk, tv, static_cast<const uint16_t*>(q), prm);
  if (cudaGetLastError() != cudaSuccess) return PKV_ERR_CUDA;
  return launch_join<kFewTokens<kHalves>>(prm, st);
}

static pkv_status launch_cluster(const void* q, const CUtensorMap& tk, const CUtensorMap& tv,
                                 const TreeParams& prm, int parts, cudaStream_t st) {
  // no sequences of so many tokens have more tiles
  const int sequences = std::min(prm.batch, prm.total_tokens);
  const int tiles = (prm.total_tokens + (kFewTokens<2> - 1) * sequences) / kFewTokens<2>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(parts, kHkv, tiles);
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = kClusterSmemBytes;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = parts;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, tree_few_kernel<2, true>, tk, tv, static_cast<const uint16_t*>(q),
                         prm) != cudaSuccess)
    return PKV_ERR_CUDA;
  return pkv_check_launch();
}

// The blocks of a tile's cluster: the largest of 16, 8 and 4 whose blocks are all
// resident at once if the sequences bring equally many tokens, while it leaves a block
// no more than 512 committed tokens; 0: the line. Measured (us, clusters and the line;
// sequences x drafted tokens over committed ones): of 16 1 x 8 over 2,000 7.4 and 8.3, 1
// x 4 over 8,000 10.8 and 12.8, over 16,000 16.6 and 15.9; of 8 4 x 8 over 2,000 9.7 and
// 12.3, 6 x 8 11.6 and 14.2; of 4 8 x 8 over 2,000 14.6 and 15.6, 12 x 4 14.4 and 16.3, 8
// x 4 over 300 6.2 and 7.2. Too large ones: of 16 3 x 8 over 2,000 11.6 (of 8 9.7).
int pkv_tree_cluster(const pkv_pool* pool, int batch, int total_tokens, int seen_tokens) {
  const long long sequences = std::min(batch, total_tokens);
  const long long each = sequences * kFewTokens<2>;
  const long long blocks = sequences * ((total_tokens + each - 1) / each) * kHkv;
  const long long slots = static_cast<long long>(kFewBlocksPerSm<2>) * pool->num_sms;
  const int parts = batch > 32                          ? 0
                    : blocks * 16 <= slots * 9 / 16     ? 16
                    : blocks * 8 <= slots * 27 / 32     ? 8
                    : blocks * 4 <= slots * 27 / 32     ? 4
                                                        : 0;
  return parts <= pool->max_cluster && seen_tokens <= kPartTokens * parts ? parts : 0;
}

pkv_status pkv_tree_few(pkv_pool_t pool, const void* q, const CUtensorMap& tk,
                        const CUtensorMap& tv, TreeParams prm, int parts, cudaStream_t st) {
  if (parts > 0) return launch_cluster(q, tk, tv, prm, parts, st);
  // Tiles of 4 tokens, and a block more per SM, where sequences bring no more on
  // average and there are several for each block (us, with tiles of 4 and of 8: 4,096
  // sequences x 2 over 64 committed tokens 321 and 392, 1,024 x 4 over 300 136 and 158,
  // 256 x 4 over 1,000 94.7 and 99.6; 128 x 4 over 2,000 94.1 and 93.2, 8 x 4 13.7 and
  // 13.0).
  const int wave = kFewBlocksPerSm<1> * pool->num_sms / kHkv;
  return prm.total_tokens <= 4ll * prm.batch && prm.batch >= 2 * wave
             ? launch_line<1>(pool, q, tk, tv, prm, st)
             : launch_line<2>(pool, q, tk, tv, prm, st);
}
