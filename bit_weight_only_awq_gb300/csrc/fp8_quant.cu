// Activations in e4m3 with a scale for each token and 128 channels.
#include "awq_internal.h"
#include "awq_types.cuh"

namespace awq {
namespace {

// Two fp32 values rounded to e4m3 (to nearest even, saturating), the first in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// A half warp has one token's 128 channels, a lane eight of them.  Groups of a token are neighbours.
template <bool BF16>
__global__ void __launch_bounds__(256) fp8_quant_kernel(const uint16_t* __restrict__ x, int64_t x_stride,
                                                        uint8_t* __restrict__ xq, float* __restrict__ s_x, int64_t M, int K,
                                                        int groups) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) / 16;
  const int lane = threadIdx.x % 16;
  const int64_t m = i / groups;
  const int g = (int)(i - m * groups), k = g * 128 + lane * 8;
  const bool in = m < M && k < K;
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (in) v = *reinterpret_cast<const uint4*>(x + m * x_stride + k);
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
  float scale = __fdiv_rn(top, 448.f);
  const bool finite = top - top == 0.f;
  if (!finite) scale = __uint_as_float(0x7FFFFFFFu);
  const bool codes = finite && scale > 0.f;
  uint32_t q[2] = {0u, 0u};
  if (codes) {
#pragma unroll
    for (int p = 0; p < 2; ++p)
      q[p] = e4m3x2(__fdiv_rn(f[4 * p], scale), __fdiv_rn(f[4 * p + 1], scale)) |
             e4m3x2(__fdiv_rn(f[4 * p + 2], scale), __fdiv_rn(f[4 * p + 3], scale)) << 16;
  }
  if (in) *reinterpret_cast<uint2*>(xq + m * K + k) = make_uint2(q[0], q[1]);
  if (m < M && lane == 0) s_x[(int64_t)g * M + m] = scale;
}

}  // namespace

cudaError_t launch_fp8_quant(const uint16_t* x, int64_t x_stride, uint8_t* xq, float* s_x, int64_t M, int64_t K, bool bf16,
                             cudaStream_t s) {
  const int groups = (int)((K + 127) / 128);
  const int64_t blocks = (M * groups * 16 + 255) / 256;
  (bf16 ? fp8_quant_kernel<true> : fp8_quant_kernel<false>)<<<(unsigned)blocks, 256, 0, s>>>(x, x_stride, xq, s_x, M, (int)K,
                                                                                            groups);
  return cudaGetLastError();
}

}  // namespace awq
