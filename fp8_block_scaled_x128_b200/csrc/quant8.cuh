// quant8.cuh -- quantisation of 8 values of a 1x128 group whose largest
// magnitude is known: for finite values the codes and scale of quant_impl.cuh's
// definition, bit for bit, at fewer instructions (a group with an infinite value
// gets a NaN scale here, an infinite one there; its codes are NaN in both).
//
//   scale = fl(amax / 448) (1 where that is zero), code = e4m3(fl(x / scale))
//
// quant_impl.cuh divides amax by 448 in IEEE arithmetic and multiplies every
// value by a power of two that is 1 for all but tiny groups.  Here both
// quotients come from quotient_rn, the first with the constant fl(1 / 448),
// and a warp that holds a tiny group (amax below 2^-80, far above the point
// where the corrections would leave the normal range) takes the general path.
#pragma once

#include "quant_impl.cuh"
#include "rows.cuh"

namespace fp8g {
namespace quant {

constexpr float kTinyAmax = 8.27180613e-25f;  // 2^-80
constexpr float kInv448 = 1.0f / kE4M3Max;    // rounded to nearest

// The scale of a group whose amax is 0 or at least kTinyAmax.
__device__ __forceinline__ float normal_scale(float amax) { return amax > 0.f ? quotient_rn(amax, kE4M3Max, kInv448) : 1.f; }

// Codes of 8 values, packed 4 per word, with scale s and y = fl(1 / s), given
// the values' negatives.  The quotients are quotient_rn's, two at a time in
// packed FP32x2 instructions (each half rounds like its scalar form), with the
// residual taken as q s - x: then a zero quotient keeps its sign through both
// corrections (q s - x = +0 for either zero, and q - (+0) y = q), so no value's
// sign has to be restored.
__device__ __forceinline__ void normal_codes(const rows::Pair8& neg, float s, float y, uint32_t (&c)[2]) {
  using namespace rows;
  const uint64_t ss = both(s), ny = both(-y);
  float q[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint64_t r = mul2(neg.v[i], ny);
    r = fma2(fma2(r, ss, neg.v[i]), ny, r);
    r = fma2(fma2(r, ss, neg.v[i]), ny, r);
    split2(r, q[2 * i], q[2 * i + 1]);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) c[i] = e4m3x2(q[4 * i], q[4 * i + 1]) | (e4m3x2(q[4 * i + 2], q[4 * i + 3]) << 16);
}

// The general path, for groups of any magnitude: quant_impl.cuh's scale_of, and its codes.
__device__ __forceinline__ void any_codes(const rows::Pair8& neg, float s, uint32_t (&c)[2]) {
  float v[8];
  rows::values_of(neg, v);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = -v[i];
  encode_group(v, s, c);
}

// Scale and codes of a lane's 8 values of a group with largest magnitude amax,
// given the values' negatives.  All 32 lanes call it.
__device__ __forceinline__ void quantize8(const rows::Pair8& neg, float amax, float& s, uint32_t (&c)[2]) {
  if (__any_sync(0xffffffffu, amax > 0.f && amax < kTinyAmax)) {
    s = scale_of(amax);
    any_codes(neg, s, c);
  } else {
    s = normal_scale(amax);
    normal_codes(neg, s, __frcp_rn(s), c);
  }
}

}  // namespace quant
}  // namespace fp8g
