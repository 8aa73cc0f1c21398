// Attention over the 4-bit paged cache.
//
//   S_j = scale q . k_j,  out = sum_j exp(S_j - m) v_j / sum_j exp(S_j - m),  m the running maximum of S
//
// with keys and values zero + u * scale for each token and head (unit layout: include/awq.h).
#include <cmath>

#include "awq_host.h"
#include "awq_internal.h"
#include "awq_types.cuh"

namespace awq {
namespace {

constexpr int kSThreads = 128;  // keys of one step, and channels at most

template <int D, bool BF16>
__global__ void __launch_bounds__(kSThreads) kv4_attention_simple_kernel(Kv4AttnArgs a) {
  __shared__ float qs[D];
  __shared__ float red[4];
  __shared__ float prob[kSThreads];
  const int tid = threadIdx.x;
  const int h = blockIdx.y, b = blockIdx.z;
  const int begin = a.q_start ? min(max(a.q_start[b], 0), (int)a.T) : b;
  const int end = a.q_start ? min(max(a.q_start[b + 1], begin), (int)a.T) : b + 1;
  const int n = min(end - begin, a.max_q), i = blockIdx.x;
  if (i >= n) return;
  const int len = min(max(a.kv_len[b], 0), a.max_pages * a.page_size);
  const int pos = len - n + i;
  const int lo = a.window > 0 ? max(0, pos - a.window + 1) : 0;
  const int64_t row = (int64_t)(begin + i) * a.heads + h;
  if (tid < D / 2) {
    const float2 f = unpack2<BF16>(
        reinterpret_cast<const uint32_t*>(a.q + (begin + i) * a.q_stride + h * D)[tid]);
    qs[2 * tid] = f.x;
    qs[2 * tid + 1] = f.y;
  }
  const int kvh = h / (a.heads / a.kv_heads), units = a.page_size / kKv4Unit;
  const int* table = a.block_table + b * a.table_stride;
  auto unit = [&](int j) {
    int page = table[j / a.page_size];
    if (page < 0 || page >= a.num_pages) page = 0;
    return a.cache + (((int64_t)page * a.kv_heads + kvh) * units + j % a.page_size / kKv4Unit) * kv4_unit_bytes(D);
  };
  float m = -INFINITY, l = 0.f, acc = 0.f;
  __syncthreads();
  for (int j0 = lo / kSThreads * kSThreads; j0 <= pos; j0 += kSThreads) {
    const int j = j0 + tid;
    float s = -INFINITY;
    if (j >= lo && j <= pos) {
      const uint8_t* u = unit(j);
      const float2 sz = unpack2<false>(*reinterpret_cast<const uint32_t*>(u + kv4_meta_offset(D, j % 16)));
      const uint32_t* w = reinterpret_cast<const uint32_t*>(u + kv4_key_offset(D, j % 16));
      float dot = 0.f, sum = 0.f;
      for (int c = 0; c < D; ++c) {
        dot = fmaf(qs[c], (float)(w[c / 8] >> (4 * slot_of_col(c % 8)) & 15u), dot);
        sum += qs[c];
      }
      s = a.scale * (sz.y * sum + sz.x * dot);
    }
    float top = s;
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    if (tid % 32 == 0) red[tid / 32] = top;
    __syncthreads();
    top = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), m);
    const float base = top == -INFINITY ? 0.f : top, old = expf(m - base);
    prob[tid] = expf(s - base);
    m = top;
    __syncthreads();
    l *= old;
    acc *= old;
    for (int t = 0; t < kSThreads; ++t) {
      if (j0 + t < lo || j0 + t > pos) continue;  // the cache may hold anything there
      l += prob[t];
      if (tid < D) {
        const uint8_t* u = unit(j0 + t);
        const float2 sz = unpack2<false>(*reinterpret_cast<const uint32_t*>(u + kv4_meta_offset(D, (j0 + t) % 16) + 4));
        const uint32_t half = *reinterpret_cast<const uint16_t*>(u + kv4_value_offset(D, (j0 + t) % 16, tid));
        acc += prob[t] * (sz.y + sz.x * (float)(half >> (4 * (tid % 4)) & 15u));
      }
    }
    __syncthreads();
  }
  if (tid < D) {
    const uint32_t o = pack2<BF16>(l > 0.f || l != l ? acc / l : 0.f, 0.f);
    a.out[row * D + tid] = (uint16_t)o;
  }
  if (a.lse && tid == 0) a.lse[row] = l > 0.f || l != l ? m + logf(l) : -INFINITY;
}

}  // namespace

size_t kv4_attention_workspace(int64_t, int64_t, int, int, int, int) { return 0; }

cudaError_t launch_kv4_attention(const Kv4AttnArgs& a, int dim, bool bf16, void*, int*, cudaStream_t s) {
  const auto fn = dim == 128 ? (bf16 ? kv4_attention_simple_kernel<128, true> : kv4_attention_simple_kernel<128, false>)
                             : (bf16 ? kv4_attention_simple_kernel<64, true> : kv4_attention_simple_kernel<64, false>);
  const int64_t most = a.max_q < a.T ? a.max_q : a.T;
  fn<<<dim3((unsigned)most, (unsigned)a.heads, (unsigned)a.B), kSThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace awq
