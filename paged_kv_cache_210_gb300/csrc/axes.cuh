// Internal to libpkv: rotation by several position axes (include/pkv_axes.h),
// shared by the prefill fill (axes.cu) and the windowed decode (window.cu).
#ifndef PKV_AXES_CUH
#define PKV_AXES_CUH

#include <cuda_runtime.h>
#include <stdint.h>

#include "pkv_axes.h"
#include "device_common.cuh"
#include "pool_internal.h"

namespace pkv_axes_dev {

using namespace pkv_dev;

constexpr int kPairs = kDim / 2;
static_assert(kPairs == 32, "a warp's lanes hold one rotary pair each");

// The kernels' copy of a pkv_axes_rope and its positions.
struct AxesArgs {
  const float* cos;
  const float* sin;
  const int32_t* positions;       // [num_axes][stride]
  long long stride;
  int rows;
  unsigned long long axes;        // 2 bits per pair: its axis
};

// INVALID_ARG unless the rotation can be used for `tokens` tokens.
inline pkv_status make_axes_args(const pkv_axes_rope* rope, const int32_t* positions, int stride,
                                 int tokens, AxesArgs* out) {
  if (!rope || !rope->cos || !rope->sin || !positions || rope->rows < 1 || rope->num_axes < 1 ||
      rope->num_axes > PKV_MAX_AXES || stride < tokens)
    return PKV_ERR_INVALID_ARG;
  if (!pkv_aligned16(rope->cos) || !pkv_aligned16(rope->sin) || !pkv_aligned4(positions))
    return PKV_ERR_INVALID_ARG;
  unsigned long long axes = 0;
  for (int i = 0; i < kPairs; ++i) {
    if (rope->axis_of_pair[i] >= rope->num_axes) return PKV_ERR_INVALID_ARG;
    axes |= static_cast<unsigned long long>(rope->axis_of_pair[i]) << (2 * i);
  }
  *out = AxesArgs{rope->cos, rope->sin, positions, stride, rope->rows, axes};
  return PKV_OK;
}

// Lane i's position for pair i of token `token` (to be checked by its user).
__device__ __forceinline__ int pair_position(const AxesArgs& rope, long long token, int lane) {
  const int axis = static_cast<int>(rope.axes >> (2 * lane)) & 3;
  return __ldg(rope.positions + axis * rope.stride + token);
}

// Lane i's angle of pair i at its position p; false (in every lane) if a lane's
// position is outside the tables. Called by a whole warp.
__device__ __forceinline__ bool load_pair_angle(const AxesArgs& rope, int p, int lane, float& c,
                                                float& s) {
  if (!__all_sync(0xffffffffu, p >= 0 && p < rope.rows)) return false;
  const size_t at = static_cast<size_t>(p) * kPairs + lane;
  c = __ldg(rope.cos + at);
  s = __ldg(rope.sin + at);
  return true;
}

// BF16 pair -> two FP32 values, exact.
__device__ __forceinline__ float2 pair_to_float2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// Two 16-byte chunks of one head, dims 8 c .. + 7 (lo) and 32 + 8 c .. + 7
// (hi), rotated in place: products and sum each rounded in FP32 (no fused
// multiply-add), then to BF16. cs, sn: the angles of pairs 8 c .. + 7.
__device__ __forceinline__ void rotate_chunks(uint4& lo, uint4& hi, const float (&cs)[8],
                                              const float (&sn)[8]) {
  uint32_t a[4] = {lo.x, lo.y, lo.z, lo.w};
  uint32_t b[4] = {hi.x, hi.y, hi.z, hi.w};
  #pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = pair_to_float2(a[j]), y = pair_to_float2(b[j]);
    const float c0 = cs[2 * j], c1 = cs[2 * j + 1], s0 = sn[2 * j], s1 = sn[2 * j + 1];
    a[j] = float2_to_bf16x2(__fsub_rn(__fmul_rn(x.x, c0), __fmul_rn(y.x, s0)),
                            __fsub_rn(__fmul_rn(x.y, c1), __fmul_rn(y.y, s1)));
    b[j] = float2_to_bf16x2(__fadd_rn(__fmul_rn(y.x, c0), __fmul_rn(x.x, s0)),
                            __fadd_rn(__fmul_rn(y.y, c1), __fmul_rn(x.y, s1)));
  }
  lo = make_uint4(a[0], a[1], a[2], a[3]);
  hi = make_uint4(b[0], b[1], b[2], b[3]);
}

}  // namespace pkv_axes_dev

#endif  // PKV_AXES_CUH
