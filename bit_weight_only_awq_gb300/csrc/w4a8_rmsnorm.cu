// Root-mean-square norm with the residual's addition and per-token int8 codes.
//
//   h = x + residual,  y = h w / sqrt(mean(h^2) + eps),  s = max|y| / 127,  code = rint(y / s)
//
// The factor 1 / sqrt(...) divides out of y / s, so the codes come from t = h w alone: with d = max|t| / 127,
// code = rint(t / d) and s = d / sqrt(mean(h^2) + eps).
#include <cmath>

#include "awq_host.h"
#include "awq_internal.h"
#include "awq_types.cuh"

namespace awq {
namespace {

constexpr int kNThreads = 256;

// The 8 values of one 16-byte vector of the row: h = x + residual in fp32.
template <bool BF16>
__device__ __forceinline__ void load_h(const uint4* x, const uint4* res, int i, float (&h)[8]) {
  const uint4 a = x[i];
  const uint32_t aw[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const float2 f = unpack2<BF16>(aw[p]);
    h[2 * p] = f.x;
    h[2 * p + 1] = f.y;
  }
  if (res) {
    const uint4 b = res[i];
    const uint32_t bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const float2 f = unpack2<BF16>(bw[p]);
      h[2 * p] = __fadd_rn(h[2 * p], f.x);
      h[2 * p + 1] = __fadd_rn(h[2 * p + 1], f.y);
    }
  }
}

// One CTA per row; the second pass reads the row again.
template <bool BF16>
__global__ void __launch_bounds__(kNThreads)
rmsnorm_kernel(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, uint16_t* res_out, uint16_t* y,
               int8_t* xq, float* s_tok, int K, int64_t x_stride, int64_t res_stride, float eps) {
  __shared__ float part[2][kNThreads / 32];
  const int64_t r = blockIdx.x;
  const uint4* xr = reinterpret_cast<const uint4*>(x + r * x_stride);
  const uint4* rr = residual ? reinterpret_cast<const uint4*>(residual + r * res_stride) : nullptr;
  const uint4* wr = reinterpret_cast<const uint4*>(weight);
  const int nvec = K / 8;
  float sum = 0.f, top = 0.f;
  for (int i = threadIdx.x; i < nvec; i += kNThreads) {
    float h[8], w[8];
    load_h<BF16>(xr, rr, i, h);
    load_h<BF16>(wr, nullptr, i, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sum = fmaf(h[j], h[j], sum);
      top = fmaxf(top, fabsf(__fmul_rn(h[j], w[j])));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  }
  if ((threadIdx.x & 31) == 0) {
    part[0][threadIdx.x >> 5] = sum;
    part[1][threadIdx.x >> 5] = top;
  }
  __syncthreads();
  sum = 0.f;
  top = 0.f;
  for (int w = 0; w < kNThreads / 32; ++w) {
    sum += part[0][w];
    top = fmaxf(top, part[1][w]);
  }
  const float rstd = 1.0f / sqrtf(sum / (float)K + eps);
  // fmaxf drops a NaN, but the sum of squares keeps it, and an infinity too
  const bool finite = sum - sum == 0.f && top - top == 0.f;
  const float step = __fdiv_rn(top, 127.0f);
  if (s_tok && threadIdx.x == 0) s_tok[r] = finite ? step * rstd : __uint_as_float(0x7FC00000u);
  for (int i = threadIdx.x; i < nvec; i += kNThreads) {
    float h[8], w[8];
    load_h<BF16>(xr, rr, i, h);
    load_h<BF16>(wr, nullptr, i, w);
    if (xq) {
      uint32_t out[2] = {0, 0};
      if (finite && step > 0.f) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float q = rintf(__fdiv_rn(__fmul_rn(h[j], w[j]), step));
          out[j >> 2] |= ((uint32_t)(int)fminf(fmaxf(q, -128.f), 127.f) & 0xFFu) << (8 * (j & 3));
        }
      }
      reinterpret_cast<uint2*>(xq + r * (int64_t)K)[i] = make_uint2(out[0], out[1]);
    }
    if (y) {
      uint32_t o[4];
#pragma unroll
      for (int p = 0; p < 4; ++p)
        o[p] = pack2<BF16>(h[2 * p] * rstd * w[2 * p], h[2 * p + 1] * rstd * w[2 * p + 1]);
      reinterpret_cast<uint4*>(y + r * (int64_t)K)[i] = make_uint4(o[0], o[1], o[2], o[3]);
    }
    if (res_out) {
      uint32_t o[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) o[p] = pack2<BF16>(h[2 * p], h[2 * p + 1]);
      reinterpret_cast<uint4*>(res_out + r * (int64_t)K)[i] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

}  // namespace

cudaError_t launch_rmsnorm(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, uint16_t* res_out,
                           uint16_t* y, int8_t* xq, float* s_tok, int64_t M, int64_t K, int64_t x_stride,
                           int64_t res_stride, float eps, bool bf16, cudaStream_t s) {
  const auto fn = bf16 ? rmsnorm_kernel<true> : rmsnorm_kernel<false>;
  fn<<<(unsigned)M, kNThreads, 0, s>>>(x, residual, weight, res_out, y, xq, s_tok, (int)K, x_stride, res_stride, eps);
  return cudaGetLastError();
}

}  // namespace awq
