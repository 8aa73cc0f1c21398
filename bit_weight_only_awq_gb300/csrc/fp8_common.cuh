// Scales and codes of e4m3 activations, for the quantization by itself and inside the product.
#pragma once

#include "awq_types.cuh"

namespace awq {
namespace {

// Two fp32 values rounded to e4m3 (to nearest even, saturating), the first in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// RN(x / s) for |x / s| <= 449 from inv = RN(1 / s), s >= 2^-100, wherever it is at least 2^-10 (smaller quotients have code 0
// either way): a product, its remainder in one fma, and the correction, which is the correctly rounded quotient as long as
// the remainder is exact (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor", 1990).
// Eight divisions and the scale's took 16 us for 4096 x 4096 codes, these 13.6.
__device__ __forceinline__ float quotient(float x, float s, float inv) {
  const float q = x * inv, r = fmaf(fmaf(-q, s, x), inv, q);
  return __uint_as_float((__float_as_uint(r) & 0x7FFFFFFFu) | (__float_as_uint(x) & 0x80000000u));  // -0 stays
}

// Eight of a token's 128 channels, the other fifteen lanes of the half warp having the rest: their codes and the scale.
template <bool BF16>
__device__ __forceinline__ uint2 quantize8(const uint4& v, float& scale) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float f[8], top = 0.f;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const float2 a = unpack2<BF16>(w[p]);
    f[2 * p] = a.x;
    f[2 * p + 1] = a.y;
    top = max_nan(top, fabsf(a.x), fabsf(a.y));
  }
#pragma unroll
  for (int d = 8; d > 0; d /= 2) top = max_nan(top, top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
  scale = __fdiv_rn(top, 448.f);
  const bool finite = top - top == 0.f;
  if (!finite) scale = __uint_as_float(0x7FFFFFFFu);
  uint32_t q[2] = {0u, 0u};
  if (finite && scale >= 0x1p-100f) {
    const float inv = __frcp_rn(scale);
#pragma unroll
    for (int p = 0; p < 8; ++p) f[p] = quotient(f[p], scale, inv);
#pragma unroll
    for (int p = 0; p < 2; ++p)
      q[p] = e4m3x2(f[4 * p], f[4 * p + 1]) | e4m3x2(f[4 * p + 2], f[4 * p + 3]) << 16;
  } else if (finite && scale > 0.f) {
#pragma unroll
    for (int p = 0; p < 2; ++p)
      q[p] = e4m3x2(__fdiv_rn(f[4 * p], scale), __fdiv_rn(f[4 * p + 1], scale)) |
             e4m3x2(__fdiv_rn(f[4 * p + 2], scale), __fdiv_rn(f[4 * p + 3], scale)) << 16;
  }
  return make_uint2(q[0], q[1]);
}

}  // namespace
}  // namespace awq
