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

// Eight codes rint(t / step).  t * inv is within 127 * 2^-22 of the correctly rounded quotient, so the integer differs
// from the quotient's only where it lies next to a half-integer; there the division is made exactly.  Adding 1.5 * 2^23
// rounds to the nearest integer, ties to even, and leaves it in the low bits of the sum.
__device__ __forceinline__ uint2 codes8(const F2 (&t)[4], float step, float inv) {
  constexpr float kMagic = 12582912.f;
  const F2 inv2(inv, inv), magic(kMagic, kMagic), minus(-1.f, -1.f);
  uint32_t b[8];
  float far = 0.f;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const F2 m = fma2(t[p], inv2, magic);
    const float2 e = fma2(t[p], inv2, fma2(m, minus, magic)).get(), w = m.get();
    far = fmaxf(far, fmaxf(fabsf(e.x), fabsf(e.y)));
    b[2 * p] = __float_as_uint(w.x);
    b[2 * p + 1] = __float_as_uint(w.y);
  }
  if (!(far < 0.49996f && inv < INFINITY)) {  // an infinite reciprocal makes NaN, which the maximum drops
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const float2 v = t[p].get();
      b[2 * p] = __float_as_uint(__fdiv_rn(v.x, step) + kMagic);
      b[2 * p + 1] = __float_as_uint(__fdiv_rn(v.y, step) + kMagic);
    }
  }
  return make_uint2(__byte_perm(__byte_perm(b[0], b[1], 0x0040), __byte_perm(b[2], b[3], 0x0040), 0x5410),
                    __byte_perm(__byte_perm(b[4], b[5], 0x0040), __byte_perm(b[6], b[7], 0x0040), 0x5410));
}

// A CTA takes rows in turn and reads each once: a thread keeps t = h w of its V vectors in registers between the
// reduction and the codes, and has the next row's vectors on the way meanwhile.  The CTA's threads cover the row's K / 8
// vectors V times.  HBM bound: 8192 x 8192 with the residual moves 470 MB in 72 us, 6.5 TB/s; 4096 x 4096 takes 19.7 us
// (6.0 TB/s), 8 rows 2.5 us.  7001 x 11016 in bf16 without residual takes 58 us (4.0 TB/s): in a capture 62 % of the issue
// slots are busy and DRAM 42 %, with dependences between instructions the first stall (1.8 of an issue's), and a row
// of 1377 vectors fills eleven warps with a ragged fourth vector.  Registers: V = 4 spills 40 to 64 bytes at two CTAs (none
// in threads of 384 without a residual, none at one CTA of 512), 52 to 440 at 1024 threads, V = 8 532 to 1004; rows wider
// than 16384 have only those two (1024 x 28672 with a residual 58 us, 4.0 TB/s).
template <bool BF16, bool RES, int V, int T, int CTAS>
__global__ void __launch_bounds__(T, CTAS)
rmsnorm_kernel(const uint16_t* x, const uint16_t* residual, const uint16_t* __restrict__ weight, uint16_t* res_out,
               uint16_t* y, int8_t* __restrict__ xq, float* __restrict__ s_tok, int M, int K, int64_t x_stride,
               int64_t res_stride, float eps) {
  // a dependent launched early waits for this grid before it reads what is written here
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ float2 part[2][T / 32];
  const int tid = threadIdx.x, threads = blockDim.x, nvec = K / 8;
  const uint4* wr = reinterpret_cast<const uint4*>(weight);
  const uint4 none = make_uint4(0u, 0u, 0u, 0u);
  uint4 xv[V], rv[RES ? V : 1];
  auto read = [&](int64_t r) {
    const uint4* xr = reinterpret_cast<const uint4*>(x + r * x_stride);
    const uint4* rr = reinterpret_cast<const uint4*>(residual + (RES ? r * res_stride : 0));
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = tid + v * threads;
      xv[v] = i < nvec ? xr[i] : none;
      if constexpr (RES) rv[v] = i < nvec ? rr[i] : none;
    }
  };
  read(blockIdx.x);
  int turn = 0;
  for (int64_t r = blockIdx.x; r < M; r += gridDim.x, turn ^= 1) {
    F2 t[V][4], sum2(0.f, 0.f);
    float top = 0.f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int i = tid + v * threads;
      float h[8], w[8];
      widen8<BF16>(xv[v], h);
      widen8<BF16>(i < nvec ? __ldg(wr + i) : none, w);
      if constexpr (RES) {
        float d[8];
        widen8<BF16>(rv[v], d);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = __fadd_rn(h[j], d[j]);
      }
      if (res_out && i < nvec) reinterpret_cast<uint4*>(res_out + r * (int64_t)K)[i] = narrow8<BF16>(h);
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const F2 h2(h[2 * p], h[2 * p + 1]);
        sum2 = fma2(h2, h2, sum2);
        t[v][p] = mul2(h2, F2(w[2 * p], w[2 * p + 1]));
        const float2 a = t[v][p].get();
        top = max_nan(top, fabsf(a.x), fabsf(a.y));
      }
    }
    float sum = sum2.get().x + sum2.get().y;
    if (r + gridDim.x < M) read(r + gridDim.x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
      const float other = __shfl_xor_sync(0xFFFFFFFFu, top, o);
      top = max_nan(top, other, other);
    }
    if ((tid & 31) == 0) part[turn][tid >> 5] = make_float2(sum, top);
    __syncthreads();  // one a row: the other half of `part` is still read by nobody two rows on
    {
      const int lane = tid & 31, warps = threads >> 5;
      const float2 p = lane < warps ? part[turn][lane] : make_float2(0.f, 0.f);
      sum = p.x;
      top = p.y;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
        const float other = __shfl_xor_sync(0xFFFFFFFFu, top, o);
        top = max_nan(top, other, other);
      }
    }
    const float rstd = 1.0f / sqrtf(sum / (float)K + eps);  // infinite for a row of zeros when eps = 0
    if (xq) {
      // a row, or a weight, that is not finite shows in the sum of squares, or in the largest product
      const bool finite = sum - sum == 0.f && top - top == 0.f;
      // top / 127 rounded once: a quotient next to the right one, corrected by its exact remainder (Markstein 1990)
      const float near = top * (1.f / 127.f), step = fmaf(fmaf(-127.f, near, top), 1.f / 127.f, near);
      const float inv = 1.0f / step;  // infinite for a step below the smallest normal number: exact division then
      const bool codes = finite && step > 0.f;
      if (tid == 0) s_tok[r] = codes ? step * rstd : finite ? 0.f : __uint_as_float(0x7FC00000u);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int i = tid + v * threads;
        if (i < nvec)
          reinterpret_cast<uint2*>(xq + r * (int64_t)K)[i] =
              codes ? codes8(t[v], step, inv) : make_uint2(0u, 0u);
      }
    }
    if (y) {
      const float by = top == 0.f && sum - sum == 0.f ? 0.f : rstd;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int i = tid + v * threads;
        float f[8];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const float2 a = t[v][p].get();
          f[2 * p] = a.x * by;
          f[2 * p + 1] = a.y * by;
        }
        if (i < nvec) reinterpret_cast<uint4*>(y + r * (int64_t)K)[i] = narrow8<BF16>(f);
      }
    }
  }
}

template <bool BF16, bool RES>
cudaError_t launch(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, uint16_t* res_out, uint16_t* y,
                   int8_t* xq, float* s_tok, int64_t M, int64_t K, int64_t x_stride, int64_t res_stride, float eps,
                   cudaStream_t s) {
  const int nvec = (int)(K / 8), sms = device_sm_count();
  // Rows that do not fill the GPU get as many threads as they have vectors, up to 1024, so that a row's loads are
  // all in flight at once; many rows get 2 or 4 vectors a thread, and a few CTAs on each SM go through them (a CTA for
  // each row instead: 4096 x 4096 24.4 us).  With 4 vectors two CTAs of 512 threads an SM need 64 registers, which only
  // the form without a residual has (7001 x 11016: 76 us at one, 64 at two; with a residual 62 against 75); two of up to
  // 384 threads have 80 (7001 x 11016 62 -> 58 us, 4096 x 11008 with a residual 60 -> 52).
  const bool few = M <= 2 * (int64_t)sms;
  const int v = few ? (nvec <= 1024 ? 1 : nvec <= 2048 ? 2 : nvec <= 4096 ? 4 : 8)
                    : (nvec <= 256 ? 1 : nvec <= 1024 ? 2 : nvec <= 4096 ? 4 : 8);
  const int threads = ((nvec + v - 1) / v + 31) / 32 * 32;
  const auto fn = v == 1   ? rmsnorm_kernel<BF16, RES, 1, 1024, 1>
                  : v == 2 ? (threads <= 512 ? rmsnorm_kernel<BF16, RES, 2, 512, 2> : rmsnorm_kernel<BF16, RES, 2, 1024, 1>)
                  : v == 8 ? rmsnorm_kernel<BF16, RES, 8, 1024, 1>
                  : threads <= 384 ? rmsnorm_kernel<BF16, RES, 4, 384, 2>
                  : threads <= 512 ? rmsnorm_kernel<BF16, RES, 4, 512, RES ? 1 : 2>
                                   : rmsnorm_kernel<BF16, RES, 4, 1024, 1>;
  const int64_t grid = few ? M : (int64_t)sms * 2048 / threads;
  fn<<<(unsigned)(grid < M ? grid : M), threads, 0, s>>>(x, residual, weight, res_out, y, xq, s_tok, (int)M, (int)K,
                                                         x_stride, res_stride, eps);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rmsnorm(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, uint16_t* res_out,
                           uint16_t* y, int8_t* xq, float* s_tok, int64_t M, int64_t K, int64_t x_stride,
                           int64_t res_stride, float eps, bool bf16, cudaStream_t s) {
  const auto fn = bf16 ? (residual ? launch<true, true> : launch<true, false>)
                       : (residual ? launch<false, true> : launch<false, false>);
  return fn(x, residual, weight, res_out, y, xq, s_tok, M, K, x_stride, res_stride, eps, s);
}

}  // namespace awq
