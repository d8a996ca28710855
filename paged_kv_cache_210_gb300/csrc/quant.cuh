// Internal to libpkv: the 8-bit cache's tiles (include/pkv_quant.h) and the
// quantisation of a row, shared by the fill (quant_store.cu) and the fused
// decode (quant.cu).
#ifndef PKV_QUANT_CUH
#define PKV_QUANT_CUH

#include <cuda_runtime.h>
#include <stdint.h>

#include "pkv_quant.h"
#include "device_common.cuh"

namespace pkv_quant_dev {

using namespace pkv_dev;

constexpr int kQuantTile = PKV_QUANT_TILE_BYTES;
constexpr int kCodeBytes = kPage * kDim;             // of K, and of V
constexpr int kChunkDims = 16;                       // dims of a V chunk
constexpr int kChunkBytes = kPage * kChunkDims;      // 256
constexpr int kKExp = 2 * kCodeBytes;                // exponent bytes of K ...
constexpr int kVExp = kKExp + kPage;                 // ... and of V
static_assert(kVExp + kPage == kQuantTile && kQuantTile % 16 == 0, "the documented tile");

// Where dims d .. of token t start in a tile (of V: d a multiple of 8).
__host__ __device__ constexpr int k_at(int t, int d) { return t * kDim + d; }
__host__ __device__ constexpr int v_at(int t, int d) {
  return kCodeBytes + d / kChunkDims * kChunkBytes + t * kChunkDims + d % kChunkDims;
}

constexpr float kLargest = 0x1.ep127f;               // 240 x 2^120, the largest value stored

// The exponent byte of a row whose largest magnitude is `most` (clamped): the
// least e >= -124 with most <= 448 x 2^e = 1.75 x 2^(e + 8), plus 127. Adding
// 0x1fffff carries into the exponent where the fraction is above 1.75.
__device__ __forceinline__ uint32_t exponent_byte(float most) {
  const int e = static_cast<int>((__float_as_uint(most) + 0x1fffffu) >> 23) - 8;
  return static_cast<uint32_t>(max(e, 3));
}

// 2^(byte - 127) and its inverse, exact for 1 <= byte <= 253.
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }
__device__ __forceinline__ float inverse_scale_of(uint32_t byte) {
  return __uint_as_float((254u - byte) << 23);
}

// Two values -> their e4m3 codes, the first in the low byte; rounded to
// nearest, ties to even.
__device__ __forceinline__ uint32_t codes_of(float x0, float x1) {
  uint16_t c;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(x1), "f"(x0));
  return c;
}

// Two codes (the low or the high half of w) -> FP16 pair, exact.
template <int kUpper>
__device__ __forceinline__ uint32_t codes_to_half2(uint32_t w) {
  uint32_t h;
  if (kUpper)
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, u;\n\t}"
        : "=r"(h)
        : "r"(w));
  else
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}"
        : "=r"(h)
        : "r"(w));
  return h;
}

// Rows of 64 values, each held by 8 neighbouring lanes, 8 values each (four rows a
// warp): exponent bytes and this lane's 8 codes of each. Called by a whole warp.
// Arithmetic on pairs where the hardware has it, and one branch for all rows: each
// lane's instructions, and how many rows are under way at once, bound the fill.
__device__ __forceinline__ float row_most(const float2 (&x)[4]) {
  float most = 0.f;                                            // a NaN does not count
  #pragma unroll
  for (int i = 0; i < 4; ++i)
    most = max3(most, __float_as_uint(fabsf(x[i].x)), __float_as_uint(fabsf(x[i].y)));
  #pragma unroll
  for (int o = 1; o < 8; o <<= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
  return most;
}
__device__ __forceinline__ uint32_t row_codes(float2 (&x)[4], float most, uint2& codes) {
  const uint32_t e = exponent_byte(most);
  const float2 inv = make_float2(inverse_scale_of(e), inverse_scale_of(e));
  #pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = __fmul2_rn(x[i], inv);
  codes.x = codes_of(x[0].x, x[0].y) | codes_of(x[1].x, x[1].y) << 16;
  codes.y = codes_of(x[2].x, x[2].y) | codes_of(x[3].x, x[3].y) << 16;
  return e;
}
template <int kRows>
__device__ __forceinline__ void quantise_rows(float2 (&x)[kRows][4], uint2 (&codes)[kRows],
                                              uint32_t (&exps)[kRows]) {
  float most[kRows], top = 0.f;
  #pragma unroll
  for (int r = 0; r < kRows; ++r) {
    most[r] = row_most(x[r]);
    top = fmaxf(top, most[r]);
  }
  if (__any_sync(0xffffffffu, top > kLargest)) {
    // values beyond the largest are taken as that; NaN stays
    #pragma unroll
    for (int r = 0; r < kRows; ++r) {
      #pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (fabsf(x[r][i].x) > kLargest) x[r][i].x = copysignf(kLargest, x[r][i].x);
        if (fabsf(x[r][i].y) > kLargest) x[r][i].y = copysignf(kLargest, x[r][i].y);
      }
      most[r] = fminf(most[r], kLargest);
    }
  }
  #pragma unroll
  for (int r = 0; r < kRows; ++r) exps[r] = row_codes(x[r], most[r], codes[r]);
}

// BF16 chunk -> 8 FP32 values, exact.
__device__ __forceinline__ void unpack8(uint4 v, float2 (&x)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  #pragma unroll
  for (int i = 0; i < 4; ++i)
    x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}

// 8 dims of a row rotated: own = dims 8 c .., partner = the other half's (c ^ 4),
// cs and sn the angles of pairs 8 (c % 4) .., sn negated for the lower half (c <
// 4: x cos - y sin); products and sum each rounded in FP32: the scalar _rn
// intrinsics are never contracted, those on pairs were (one code in four million
// came out different).
__device__ __forceinline__ void rotate8(float2 (&x)[4], const float2 (&partner)[4],
                                        const float2 (&cs)[4], const float2 (&sn)[4]) {
  #pragma unroll
  for (int i = 0; i < 4; ++i)
    x[i] = make_float2(__fadd_rn(__fmul_rn(x[i].x, cs[i].x), __fmul_rn(partner[i].x, sn[i].x)),
                       __fadd_rn(__fmul_rn(x[i].y, cs[i].y), __fmul_rn(partner[i].y, sn[i].y)));
}

// 8 dims of a row rotated, the 4 in x[0], x[1] being the partners of those in x[2],
// x[3]; cs and sn the angles of their 4 pairs; rounded as above.
__device__ __forceinline__ void rotate_halves(float2 (&x)[4], const float2 (&cs)[2],
                                              const float2 (&sn)[2]) {
  #pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 a = x[i], b = x[i + 2];
    x[i] = make_float2(__fsub_rn(__fmul_rn(a.x, cs[i].x), __fmul_rn(b.x, sn[i].x)),
                       __fsub_rn(__fmul_rn(a.y, cs[i].y), __fmul_rn(b.y, sn[i].y)));
    x[i + 2] = make_float2(__fadd_rn(__fmul_rn(b.x, cs[i].x), __fmul_rn(a.x, sn[i].x)),
                           __fadd_rn(__fmul_rn(b.y, cs[i].y), __fmul_rn(a.y, sn[i].y)));
  }
}

}  // namespace pkv_quant_dev

#endif  // PKV_QUANT_CUH
