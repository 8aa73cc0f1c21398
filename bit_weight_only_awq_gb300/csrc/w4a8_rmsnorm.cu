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

// The eight values of a 16-byte vector in fp32.
template <bool BF16>
__device__ __forceinline__ void widen8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const float2 d = unpack2<BF16>(w[p]);
    f[2 * p] = d.x;
    f[2 * p + 1] = d.y;
  }
}
template <bool BF16>
__device__ __forceinline__ uint4 narrow8(const float (&f)[8]) {
  return make_uint4(pack2<BF16>(f[0], f[1]), pack2<BF16>(f[2], f[3]), pack2<BF16>(f[4], f[5]), pack2<BF16>(f[6], f[7]));
}

// Four codes rint(t / step) in the bytes of a word.  t * inv is within 127 * 2^-23 of the correctly rounded
// quotient, so the integer differs from the quotient's only where it lies next to a half-integer; there the
// division is made exactly.  Adding 1.5 * 2^23 rounds to the nearest integer, ties to even, and leaves it in the
// low bits of the sum.
__device__ __forceinline__ uint32_t codes4(const float* t, float step, float inv) {
  constexpr float kMagic = 12582912.f;
  uint32_t b[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float r = t[j] * inv;
    float m = r + kMagic;
    if (!(fabsf(r - (m - kMagic)) < 0.4999f)) m = __fdiv_rn(t[j], step) + kMagic;
    b[j] = __float_as_uint(m);
  }
  return __byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410);
}

// One CTA per row, which is read once: each thread keeps t = h w of its V vectors in registers between the
// reduction and the codes.  The CTA's threads cover the row's K / 8 vectors V times.
template <bool BF16, int V, int T>
__global__ void __launch_bounds__(T)
rmsnorm_kernel(const uint16_t* x, const uint16_t* residual, const uint16_t* __restrict__ weight, uint16_t* res_out,
               uint16_t* y, int8_t* __restrict__ xq, float* __restrict__ s_tok, int K, int64_t x_stride,
               int64_t res_stride, float eps) {
  // a dependent launched early waits for this grid before it reads what is written here
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ float2 part[T / 32];
  const int64_t r = blockIdx.x;
  const int tid = threadIdx.x, threads = blockDim.x, nvec = K / 8;
  const uint4* xr = reinterpret_cast<const uint4*>(x + r * x_stride);
  const uint4* rr = reinterpret_cast<const uint4*>(residual + r * res_stride);
  const uint4* wr = reinterpret_cast<const uint4*>(weight);
  uint4 xv[V], rv[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = tid + v * threads;
    xv[v] = i < nvec ? xr[i] : make_uint4(0u, 0u, 0u, 0u);
    rv[v] = residual && i < nvec ? rr[i] : make_uint4(0u, 0u, 0u, 0u);
  }
  float t[V][8];
  float sum = 0.f, top = 0.f;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int i = tid + v * threads;
    float h[8], w[8];
    widen8<BF16>(xv[v], h);
    widen8<BF16>(i < nvec ? __ldg(wr + i) : make_uint4(0u, 0u, 0u, 0u), w);
    if (residual) {
      float d[8];
      widen8<BF16>(rv[v], d);
#pragma unroll
      for (int j = 0; j < 8; ++j) h[j] = __fadd_rn(h[j], d[j]);
    }
    if (res_out && i < nvec) reinterpret_cast<uint4*>(res_out + r * (int64_t)K)[i] = narrow8<BF16>(h);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      sum = fmaf(h[j], h[j], sum);
      t[v][j] = __fmul_rn(h[j], w[j]);
      top = fmaxf(top, fabsf(t[v][j]));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  }
  if ((tid & 31) == 0) part[tid >> 5] = make_float2(sum, top);
  __syncthreads();
  {
    const int lane = tid & 31, warps = threads >> 5;
    const float2 p = lane < warps ? part[lane] : make_float2(0.f, 0.f);
    sum = p.x;
    top = p.y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
      top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    }
  }
  const float rstd = 1.0f / sqrtf(sum / (float)K + eps);
  if (xq) {
    // fmaxf drops a NaN, but the sum of squares keeps it, and an infinity too
    const bool finite = sum - sum == 0.f && top - top == 0.f;
    const float step = __fdiv_rn(top, 127.0f);
    const float inv = 1.0f / step;  // infinite for a step below the smallest normal number: exact division then
    if (tid == 0) s_tok[r] = finite ? step * rstd : __uint_as_float(0x7FC00000u);
    const bool codes = finite && step > 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = tid + v * threads;
      if (i < nvec)
        reinterpret_cast<uint2*>(xq + r * (int64_t)K)[i] =
            codes ? make_uint2(codes4(t[v], step, inv), codes4(t[v] + 4, step, inv)) : make_uint2(0u, 0u);
    }
  }
  if (y) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = tid + v * threads;
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = t[v][j] * rstd;
      if (i < nvec) reinterpret_cast<uint4*>(y + r * (int64_t)K)[i] = narrow8<BF16>(f);
    }
  }
}

template <bool BF16>
cudaError_t launch(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, uint16_t* res_out, uint16_t* y,
                   int8_t* xq, float* s_tok, int64_t M, int64_t K, int64_t x_stride, int64_t res_stride, float eps,
                   cudaStream_t s) {
  const int nvec = (int)(K / 8);
  // Rows that do not fill the GPU get as many threads as they have vectors, up to 1024, so that a row's loads are
  // all in flight at once; many rows get 2 or 4 vectors a thread, and more rows on an SM.
  const bool few = M <= 2 * (int64_t)device_sm_count();
  const int v = few ? (nvec <= 1024 ? 1 : nvec <= 2048 ? 2 : nvec <= 4096 ? 4 : 8)
                    : (nvec <= 256 ? 1 : nvec <= 512 ? 2 : nvec <= 4096 ? 4 : 8);
  const int threads = ((nvec + v - 1) / v + 31) / 32 * 32;
  const auto fn = v == 1   ? rmsnorm_kernel<BF16, 1, 1024>
                  : v == 2 ? rmsnorm_kernel<BF16, 2, 1024>
                  : v == 8 ? rmsnorm_kernel<BF16, 8, 1024>
                  : threads <= 512 ? rmsnorm_kernel<BF16, 4, 512>
                                   : rmsnorm_kernel<BF16, 4, 1024>;
  fn<<<(unsigned)M, threads, 0, s>>>(x, residual, weight, res_out, y, xq, s_tok, (int)K, x_stride, res_stride, eps);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rmsnorm(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, uint16_t* res_out,
                           uint16_t* y, int8_t* xq, float* s_tok, int64_t M, int64_t K, int64_t x_stride,
                           int64_t res_stride, float eps, bool bf16, cudaStream_t s) {
  return bf16 ? launch<true>(x, residual, weight, res_out, y, xq, s_tok, M, K, x_stride, res_stride, eps, s)
              : launch<false>(x, residual, weight, res_out, y, xq, s_tok, M, K, x_stride, res_stride, eps, s);
}

}  // namespace awq
