// Activations in e4m3 with a scale for each token and 128 channels.
#include "awq_internal.h"
#include "awq_host.h"
#include "awq_ptx.cuh"
#include "fp8_common.cuh"

namespace awq {
namespace {

// A half warp has one token's 128 channels, a lane eight of them.  Groups of a token are neighbours.  4096 x 4096: 13.6 us, 3.7 TB/s;
// bound by the instructions of the quotients (issue slots 76 % busy).  Two or four pieces a half warp and 32-bit divisions took 12.8 to
// 13.1: 0.2 % of the layer of 28672 outputs that it was timed in, so the plain form stays.
template <bool BF16>
__global__ void __launch_bounds__(256) fp8_quant_kernel(const uint16_t* __restrict__ x, int64_t x_stride,
                                                        uint8_t* __restrict__ xq, float* __restrict__ s_x, int64_t M, int K,
                                                        int groups) {
  wait_then_release_dependents();
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) / 16;
  const int lane = threadIdx.x % 16;
  const int64_t m = i / groups;
  const int g = (int)(i - m * groups), k = g * 128 + lane * 8;
  const bool in = m < M && k < K;
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (in) v = *reinterpret_cast<const uint4*>(x + m * x_stride + k);
  float scale;
  const uint2 codes = quantize8<BF16>(v, scale);
  if (in) *reinterpret_cast<uint2*>(xq + m * K + k) = codes;
  if (m < M && lane == 0) s_x[(int64_t)g * M + m] = scale;
}

}  // namespace

cudaError_t launch_fp8_quant(const uint16_t* x, int64_t x_stride, uint8_t* xq, float* s_x, int64_t M, int64_t K, bool bf16,
                             cudaStream_t s) {
  const int groups = (int)((K + 127) / 128);
  const int64_t blocks = (M * groups * 16 + 255) / 256;
  return launch_dependent(bf16 ? fp8_quant_kernel<true> : fp8_quant_kernel<false>, dim3((unsigned)blocks), 256, 0, s, x,
                          x_stride, xq, s_x, M, (int)K, groups);
}

}  // namespace awq
