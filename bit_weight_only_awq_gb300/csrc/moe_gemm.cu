// Products grouped by expert on prepared 4-bit weights (layout: include/awq.h).
//
// y[r, n] = sum_k x[src(r), k] RN16((q[k, n] - z) s) over an expert's rows; gated: silu(gate) * up.
// A CTA has 256 columns and 8 rows of one expert; a thread has one column of each half.
#include "awq_internal.h"
#include "awq_types.cuh"

namespace awq {
namespace {

constexpr int kRows = 8;

template <bool BF16>
__device__ __forceinline__ float round16(float v) {
  return unpack2<BF16>(pack2<BF16>(v, 0.f)).x;
}
template <bool BF16>
__device__ __forceinline__ float widen(uint16_t v) {
  return unpack2<BF16>((uint32_t)v).x;
}

template <bool BF16, bool GATED>
__global__ void __launch_bounds__(128) moe_gemm_simple(const MoeGemmArgs a) {
  __shared__ float xs[kRows][128];
  __shared__ int where[3];  // expert, first row, rows
  const int tid = threadIdx.x;
  if (tid == 0) {
    int item = blockIdx.y, end = 0;
    where[0] = -1;
    for (int e = 0; e < a.experts; ++e) {
      const int begin = max(end, min(a.offsets[e], (int)a.R));
      end = max(begin, min(a.offsets[e + 1], (int)a.R));
      const int items = (end - begin + kRows - 1) / kRows;
      if (item < items) {
        where[0] = e;
        where[1] = begin + item * kRows;
        where[2] = min(kRows, end - where[1]);
        break;
      }
      item -= items;
    }
  }
  __syncthreads();
  const int e = where[0], r0 = where[1], rows = where[2];
  if (e < 0) return;
  const int groups = (int)(a.K / 128), tile = blockIdx.x;
  float acc[2][kRows] = {};
  for (int g = 0; g < groups; ++g) {
    __syncthreads();
    for (int r = 0; r < kRows; ++r) {
      int64_t src = r < rows ? (a.order ? (a.order[r0 + r] < 0 ? -1 : a.order[r0 + r] / a.top_k) : r0 + r) : -1;
      if (src >= a.x_rows) src = -1;
      xs[r][tid] = src >= 0 ? widen<BF16>(a.x[src * a.x_stride + g * 128 + tid]) : 0.f;
    }
    __syncthreads();
    const uint8_t* unit = a.packed + (((int64_t)e * a.tiles + tile) * groups + g) * kMoeUnitBytes;
    for (int b = 0; b < 2; ++b) {
      const int n = b * 128 + tid;
      const float z = (float)(unit[kMoeZeroOffset + n / 2] >> (4 * (n & 1)) & 15);
      const float s = widen<BF16>(*reinterpret_cast<const uint16_t*>(unit + kMoeScaleOffset + 2 * n));
      for (int c = 0; c < 4; ++c) {
        const uint4 v = *reinterpret_cast<const uint4*>(unit + moe_code_offset(n, c));
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        for (int q = 0; q < 4; ++q)
          for (int i = 0; i < 8; ++i) {
            const float weight = round16<BF16>(((float)(w[q] >> (4 * i) & 15u) - z) * s);
            const int k = 32 * c + 8 * q + order_map(i);
#pragma unroll
            for (int r = 0; r < kRows; ++r) acc[b][r] = fmaf(weight, xs[r][k], acc[b][r]);
          }
      }
    }
  }
  const int64_t out = GATED ? a.N / 2 : a.N;
  for (int r = 0; r < rows; ++r) {
    if (GATED) {
      const int64_t n = (int64_t)tile * 128 + tid;
      const float v = acc[0][r] / (1.f + expf(-acc[0][r])) * acc[1][r];
      if (n < out) a.y[(int64_t)(r0 + r) * out + n] = (uint16_t)pack2<BF16>(v, 0.f);
    } else {
      for (int b = 0; b < 2; ++b) {
        const int64_t n = (int64_t)tile * 256 + b * 128 + tid;
        if (n < out) a.y[(int64_t)(r0 + r) * out + n] = (uint16_t)pack2<BF16>(acc[b][r], 0.f);
      }
    }
  }
}

}  // namespace

size_t moe_gemm_workspace(int64_t, int, int64_t, int64_t, bool) { return 0; }

cudaError_t launch_moe_gemm(const MoeGemmArgs& a, bool gated, bool bf16, void*, int*, cudaStream_t s) {
  const int64_t items = a.R / kRows + (a.experts < a.R ? a.experts : a.R);
  const dim3 grid((unsigned)a.tiles, (unsigned)items);
  const auto fn = bf16 ? (gated ? moe_gemm_simple<true, true> : moe_gemm_simple<true, false>)
                       : (gated ? moe_gemm_simple<false, true> : moe_gemm_simple<false, false>);
  fn<<<grid, 128, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace awq
