// The router of a layer with experts: softmax and top_k of each token, the plan that puts the chosen rows in the experts'
// order, and the weighted sum of a token's rows.
//
// 8191 tokens' fp32 logits over 128 experts are 4 MB and take 9.5 us, about half of it instructions (issue slots 63 % busy), the rest
// the launch and the first loads.  A warp has a token; its lanes hold the logits
// in registers, as keys whose order as whole numbers is the logits' order, and every choice is one reduction of keys and
// one ballot for the lowest expert among equals.
#include <type_traits>

#include "awq_host.h"
#include "awq_internal.h"
#include "awq_ptx.cuh"
#include "awq_types.cuh"

namespace awq {
namespace {

constexpr uint32_t kAll = 0xFFFFFFFFu;

// A float as a key: larger for a larger value, equal for 0 and -0, above all others for a NaN.  0 is no value's key.
__device__ __forceinline__ uint32_t key_of(float v) {
  if (v != v) return 0xFFFFFFFFu;
  const uint32_t u = __float_as_uint(v + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t key) {
  if (key == 0xFFFFFFFFu) return __uint_as_float(0x7FFFFFFFu);
  return __uint_as_float(key & 0x80000000u ? key & 0x7FFFFFFFu : ~key);
}

template <int TYPE>
__device__ __forceinline__ float read_logit(const void* p, int64_t i) {
  if constexpr (TYPE == 2) return static_cast<const float*>(p)[i];
  else if constexpr (TYPE == 1) return __uint_as_float((uint32_t)static_cast<const uint16_t*>(p)[i] << 16);
  else return __half2float(static_cast<const __half*>(p)[i]);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(kAll, v, d);
  return v;
}

// One token, by one warp: choice j's expert and weight end up in lane j.
template <int TYPE, int L>
__device__ __forceinline__ void route_token(const void* logits, int64_t at, int experts, int top_k, bool normalize, int lane,
                                            int& id, float& weight) {
  uint32_t key[L];
#pragma unroll
  for (int l = 0; l < L; ++l) {
    const int e = lane + 32 * l;
    key[l] = e < experts ? key_of(read_logit<TYPE>(logits, at + e)) : 0u;
  }
  uint32_t most = 0u;
#pragma unroll
  for (int l = 0; l < L; ++l) most = max(most, key[l]);
  const float top = value_of(__reduce_max_sync(kAll, most));
  float sum = 0.f;
  if (!normalize) {
#pragma unroll
    for (int l = 0; l < L; ++l)
      if (key[l] != 0u) sum += expf(value_of(key[l]) - top);
    sum = warp_sum(sum);
  }
  id = 0;
  float mine = 0.f;
  for (int j = 0; j < top_k; ++j) {
    uint32_t best = 0u;
    int where = 0;
#pragma unroll
    for (int l = 0; l < L; ++l)
      if (key[l] > best) {
        best = key[l];
        where = l;
      }
    const uint32_t k = __reduce_max_sync(kAll, best);
    const int e = (int)__reduce_min_sync(kAll, best == k ? (uint32_t)(lane + 32 * where) : kAll);
#pragma unroll
    for (int l = 0; l < L; ++l)
      if (lane + 32 * l == e) key[l] = 0u;
    if (lane == j) {
      id = e;
      mine = expf(value_of(k) - top);
    }
  }
  if (normalize) sum = warp_sum(mine);
  // a row of nothing but -inf has no weights; a NaN or +inf makes `top - top` NaN, and every weight with it
  weight = top == -INFINITY ? 0.f : mine / sum;
  if (!(top - top == 0.f) && top != -INFINITY) weight = __uint_as_float(0x7FFFFFFFu);
}

// Class of a position: its expert, or `experts` for an id that is none.
__device__ __forceinline__ int class_of(int id, int experts) { return (unsigned)id < (unsigned)experts ? id : experts; }

// Four ids from position i on; `none` beyond the end.
__device__ __forceinline__ void read4(const int32_t* ids, int i, int end, bool aligned, int experts, int (&c)[4]) {
  constexpr int kBeyond = 0x7FFFFFFF;
  if (aligned && i + 4 <= end) {
    const int4 v = *reinterpret_cast<const int4*>(ids + i);
    c[0] = class_of(v.x, experts), c[1] = class_of(v.y, experts), c[2] = class_of(v.z, experts), c[3] = class_of(v.w, experts);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) c[j] = i + j < end ? class_of(ids[i + j], experts) : kBeyond;
  }
}
// The warp's positions [begin, end): how many are of a class below e, and of class e.  A lane reads four neighbours.
__device__ __forceinline__ void count_class(const int32_t* ids, int begin, int end, bool aligned, int e, int experts, int lane,
                                            int& below, int& equal) {
  int b = 0, q = 0;
#pragma unroll 4
  for (int i = begin + 4 * lane; i < end; i += 128) {
    int c[4];
    read4(ids, i, end, aligned, experts, c);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      b += c[j] < e;
      q += c[j] == e;
    }
  }
  below = __reduce_add_sync(kAll, b);
  equal = __reduce_add_sync(kAll, q);
}
// Writes the rows of class e among them, from row `row` on.
__device__ __forceinline__ void place_class(const int32_t* ids, int begin, int end, bool aligned, int e, int experts, int lane,
                                            int row, int32_t* order, int32_t* place) {
  const uint32_t before = (1u << lane) - 1u;
#pragma unroll 4
  for (int i0 = begin; i0 < end; i0 += 128) {
    const int i = i0 + 4 * lane;
    int c[4];
    read4(ids, i, end, aligned, experts, c);
    uint32_t votes[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) votes[j] = __ballot_sync(kAll, c[j] == e);
    int r = row;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      r += __popc(votes[j] & before);
      row += __popc(votes[j]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c[j] == e) {
        order[r] = e < experts ? i + j : -1;
        place[i + j] = e < experts ? r : -1;
        ++r;
      }
  }
}

// A CTA for each class (expert, and "none"): counts what comes before its rows, then writes them.  Every CTA
// looks at all ids twice (8192 of 128 experts: 4.9 us, where the form for many rows takes 8.0).
__global__ void __launch_bounds__(1024) plan_kernel(const int32_t* __restrict__ ids, int R, int experts,
                                                    int32_t* __restrict__ offsets, int32_t* __restrict__ order,
                                                    int32_t* __restrict__ place) {
  __shared__ int s_below[32], s_equal[32];
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, e = blockIdx.x;
  wait_then_release_dependents();
  const int share = (int)(((int64_t)R + 4095) / 4096 * 128);
  const bool aligned = (reinterpret_cast<uintptr_t>(ids) & 15u) == 0;
  const int begin = (int)min((int64_t)R, (int64_t)warp * share), end = (int)min((int64_t)R, (int64_t)(warp + 1) * share);
  int below, equal;
  count_class(ids, begin, end, aligned, e, experts, lane, below, equal);
  if (lane == 0) {
    s_below[warp] = below;
    s_equal[warp] = equal;
  }
  __syncthreads();
  int row = s_below[lane], before = lane < warp ? s_equal[lane] : 0;
#pragma unroll
  for (int d = 16; d > 0; d /= 2) {
    row += __shfl_xor_sync(kAll, row, d);
    before += __shfl_xor_sync(kAll, before, d);
  }
  if (threadIdx.x == 0) offsets[e] = row;
  place_class(ids, begin, end, aligned, e, experts, lane, row + before, order, place);
}

// Many rows: one cluster of CTAs, each warp with a stretch of positions of its own.  The warps count their classes in shared memory, sums
// over the warps of a CTA, the CTAs (through distributed shared memory) and the lower classes give each warp the first row of each
// class, and the warps go over their stretch again, 32 positions at once in order.  Every id is read twice, not twice a class; bound by
// the steps' latency (5 us without any rows to speak of) and 8 SMs.
constexpr int kPlanCtas = 8, kPlanWarps = 32;
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__global__ void __cluster_dims__(kPlanCtas, 1, 1) __launch_bounds__(kPlanWarps * 32)
plan_many_kernel(const int32_t* __restrict__ ids, int R, int experts, int32_t* __restrict__ offsets, int32_t* __restrict__ order,
                 int32_t* __restrict__ place) {
  extern __shared__ int s_counts[];  // [warp][class] | this CTA's sums of classes | first rows
  __shared__ int s_warp[kPlanWarps];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, rank = blockIdx.x, classes = experts + 1;
  int* mine = s_counts + warp * classes;
  int* sums = s_counts + kPlanWarps * classes;
  int* first = sums + classes;
  wait_then_release_dependents();
  for (int c = lane; c < classes; c += 32) mine[c] = 0;
  __syncwarp();
  constexpr int kStretches = kPlanCtas * kPlanWarps;
  const int64_t share = ((int64_t)R + kStretches * 128 - 1) / (kStretches * 128) * 128, at = (int64_t)(rank * kPlanWarps + warp) * share;
  const int begin = (int)min((int64_t)R, at), end = (int)min((int64_t)R, at + share);
  const bool aligned = (reinterpret_cast<uintptr_t>(ids) & 15u) == 0;
#pragma unroll 2
  for (int i = begin + 4 * lane; i < end; i += 128) {
    int c[4];
    read4(ids, i, end, aligned, experts, c);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (c[j] < classes) atomicAdd(mine + c[j], 1);
  }
  __syncthreads();
  if (tid < classes) {
    int sum = 0;
#pragma unroll 8
    for (int w = 0; w < kPlanWarps; ++w) {
      const int n = s_counts[w * classes + tid];
      s_counts[w * classes + tid] = sum;
      sum += n;
    }
    sums[tid] = sum;
  }
  cluster_sync();
  int before = 0, all = 0;  // of class `tid`: in the CTAs before this one, in all
  if (tid < classes) {
    const uint32_t own = smem_u32(sums + tid);
#pragma unroll
    for (int r = 0; r < kPlanCtas; ++r) {
      uint32_t there;
      int n;
      asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(own), "r"(r));
      asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(n) : "r"(there) : "memory");
      before += r < rank ? n : 0;
      all += n;
    }
  }
  int row = all;  // sums of the classes up to this one, of the warp's
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const int o = __shfl_up_sync(kAll, row, d);
    if (lane >= d) row += o;
  }
  if (lane == 31) s_warp[warp] = row;
  __syncthreads();
  int lower = lane < warp ? s_warp[lane] : 0;
#pragma unroll
  for (int d = 16; d > 0; d /= 2) lower += __shfl_xor_sync(kAll, lower, d);
  row += lower - all;
  if (tid < classes) {
    first[tid] = row + before;
    if (rank == 0) offsets[tid] = row;
  }
  __syncthreads();
  const uint32_t left = (1u << lane) - 1u;
  const int bits = 32 - __clz(classes);
  int id = begin + lane < end ? ids[begin + lane] : 0;
  for (int i0 = begin; i0 < end; i0 += 32) {
    const int i = i0 + lane, c = i < end ? class_of(id, experts) : classes;
    if (i + 32 < end) id = ids[i + 32];
    uint32_t same = kAll;  // lanes of the same class, bit by bit (__match_any_sync takes the
    // longer the more there are: 14.6 us against 11.1 for 65528 ids of 128 experts)
#pragma unroll 4
    for (int b = 0; b < bits; ++b) {
      const uint32_t set = __ballot_sync(kAll, c >> b & 1);
      same &= c >> b & 1 ? set : ~set;
    }
    int r = 0;
    if (c < classes) r = first[c] + mine[c] + __popc(same & left);
    __syncwarp();
    if (c < classes) {
      if ((same & left) == 0u) mine[c] += __popc(same);
      order[r] = c < experts ? i : -1;
      place[i] = c < experts ? r : -1;
    }
    __syncwarp();
  }
  cluster_sync();  // the others may still read this CTA's sums
}

template <int TYPE, int L>
__global__ void __launch_bounds__(256) route_kernel(const void* __restrict__ logits, int64_t stride, int T, int experts,
                                                    int top_k, int normalize, int32_t* __restrict__ ids,
                                                    float* __restrict__ weights) {
  const int lane = threadIdx.x % 32;
  const int64_t t = (int64_t)blockIdx.x * 8 + threadIdx.x / 32;
  wait_then_release_dependents();
  if (t >= T) return;
  int id;
  float weight;
  route_token<TYPE, L>(logits, t * stride, experts, top_k, normalize != 0, lane, id, weight);
  if (lane < top_k) {
    ids[t * top_k + lane] = id;
    weights[t * top_k + lane] = weight;
  }
}

// Few tokens: one CTA routes them, a token a warp, and makes the plan from ids in shared memory: one launch instead of two (8 tokens
// over 64 experts, 8 each: 4.4 us against 5.4; 32 over 8, 2 each: 3.9 against 4.9; 32 over 128, 8 each, would be 8.5 against 5.9; 64 over
// 8, 5.4 against 4.9).
constexpr int kFewTokens = 32, kFewRows = 128;
template <int TYPE, int L>
__global__ void __launch_bounds__(1024) route_few_kernel(const void* __restrict__ logits, int64_t stride, int T, int experts,
                                                         int top_k, int normalize, int32_t* __restrict__ ids,
                                                         float* __restrict__ weights, int32_t* __restrict__ offsets,
                                                         int32_t* __restrict__ order, int32_t* __restrict__ place) {
  __shared__ int32_t s_ids[kFewRows];
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, R = T * top_k;
  wait_then_release_dependents();
  if (warp < T) {
    int id;
    float weight;
    route_token<TYPE, L>(logits, warp * stride, experts, top_k, normalize != 0, lane, id, weight);
    if (lane < top_k) {
      ids[warp * top_k + lane] = id;
      weights[warp * top_k + lane] = weight;
      s_ids[warp * top_k + lane] = id;
    }
  }
  __syncthreads();
  // a row's place is the number of rows that come before it, an expert's offset the number of rows of lower ones
  if (tid < R) {
    const int id = s_ids[tid];
    int before = 0;
    for (int q = 0; q < R; ++q) {
      const int other = s_ids[q];
      before += other < id || (other == id && q < tid);
    }
    order[before] = tid;
    place[tid] = before;
  } else if (tid >= kFewRows && tid - kFewRows <= experts) {
    int below = 0;
    for (int q = 0; q < R; ++q) below += s_ids[q] < tid - kFewRows;
    offsets[tid - kFewRows] = below;
  }
}

// WIDE: y in fp32.
template <bool BF16, bool WIDE>
__global__ void __launch_bounds__(256) combine_kernel(const void* __restrict__ y, const int32_t* __restrict__ place,
                                                      const float* __restrict__ weights, const uint16_t* residual,
                                                      int64_t res_stride, uint16_t* out, int64_t T, int top_k, int64_t H,
                                                      int64_t R) {
  const int64_t vec = H / 8, i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  wait_then_release_dependents();
  if (i >= T * vec) return;
  const int64_t t = i / vec, c = (i - t * vec) * 8;
  float sum[8];
#pragma unroll
  for (int p = 0; p < 8; ++p) sum[p] = 0.f;
  if (residual) {
    const uint4 v = *reinterpret_cast<const uint4*>(residual + t * res_stride + c);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const float2 f = unpack2<BF16>(w[p]);
      sum[2 * p] = f.x;
      sum[2 * p + 1] = f.y;
    }
  }
#pragma unroll 4
  for (int j = 0; j < top_k; ++j) {
    const int r = place[t * top_k + j];
    if (r < 0 || r >= R) continue;
    const float weight = weights[t * top_k + j];
    float f[8];
    if constexpr (WIDE) {
      const float4* v = reinterpret_cast<const float4*>(static_cast<const float*>(y) + r * H + c);
      const float4 lo = v[0], hi = v[1];
      f[0] = lo.x, f[1] = lo.y, f[2] = lo.z, f[3] = lo.w;
      f[4] = hi.x, f[5] = hi.y, f[6] = hi.z, f[7] = hi.w;
    } else {
      const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(y) + r * H + c);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const float2 u = unpack2<BF16>(w[p]);
        f[2 * p] = u.x;
        f[2 * p + 1] = u.y;
      }
    }
#pragma unroll
    for (int p = 0; p < 8; ++p) sum[p] = fmaf(weight, f[p], sum[p]);
  }
  *reinterpret_cast<uint4*>(out + t * H + c) = make_uint4(pack2<BF16>(sum[0], sum[1]), pack2<BF16>(sum[2], sum[3]),
                                                          pack2<BF16>(sum[4], sum[5]), pack2<BF16>(sum[6], sum[7]));
}

}  // namespace

// us of a CTA a class and of one cluster: 16384 ids of 128 experts 5.9 and 8.0, all of one expert 12.3 and 6.9; 32768 of 512 experts
// 19.2 and 9.0; 65528 of 128 15.2 and 11.1, of one 41.3 and 10.0; 2^20 of 256 experts 258 and 104.
constexpr int64_t kPlanFewRows = 16384;
cudaError_t launch_moe_plan(const int32_t* ids, int64_t R, int experts, int32_t* offsets, int32_t* order, int32_t* place,
                            cudaStream_t s) {
  if (R > kPlanFewRows) {
    const int smem = (kPlanWarps + 2) * (experts + 1) * (int)sizeof(int);
    const cudaError_t e = set_smem_once(reinterpret_cast<const void*>(plan_many_kernel),
                                        (kPlanWarps + 2) * (kMoeMaxExperts + 1) * (int)sizeof(int));
    if (e != cudaSuccess) return e;
    return launch_dependent(plan_many_kernel, dim3(kPlanCtas), kPlanWarps * 32, smem, s, ids, (int)R, experts, offsets, order, place);
  }
  return launch_dependent(plan_kernel, dim3(experts + 1), 1024, 0, s, ids, (int)R, experts, offsets, order, place);
}

cudaError_t launch_moe_route(const void* logits, int64_t stride, int64_t T, int experts, int top_k, bool normalize, int type,
                             int32_t* ids, float* weights, int32_t* offsets, int32_t* order, int32_t* place,
                             cudaStream_t s) {
  const bool few = offsets && T <= kFewTokens && T * top_k <= kFewRows;
  auto by_size = [&](auto kType, auto kL) {
    constexpr int TYPE = decltype(kType)::value, L = decltype(kL)::value;
    if (few)
      return launch_dependent(route_few_kernel<TYPE, L>, dim3(1), 1024, 0, s, logits, stride, (int)T, experts, top_k,
                              (int)normalize, ids, weights, offsets, order, place);
    return launch_dependent(route_kernel<TYPE, L>, dim3((unsigned)((T + 7) / 8)), 256, 0, s, logits, stride, (int)T, experts,
                            top_k, (int)normalize, ids, weights);
  };
  auto by_type = [&](auto t) {
    return experts <= 32    ? by_size(t, std::integral_constant<int, 1>{})
           : experts <= 64  ? by_size(t, std::integral_constant<int, 2>{})
           : experts <= 128 ? by_size(t, std::integral_constant<int, 4>{})
           : experts <= 256 ? by_size(t, std::integral_constant<int, 8>{})
                            : by_size(t, std::integral_constant<int, 16>{});
  };
  if (T > 0) {
    const cudaError_t e = type == 0   ? by_type(std::integral_constant<int, 0>{})
                          : type == 1 ? by_type(std::integral_constant<int, 1>{})
                                      : by_type(std::integral_constant<int, 2>{});
    if (e != cudaSuccess || few) return e;
  }
  return offsets ? launch_moe_plan(ids, T * top_k, experts, offsets, order, place, s) : cudaSuccess;
}

cudaError_t launch_moe_combine(const void* y, bool wide, const int32_t* place, const float* weights, const uint16_t* residual,
                               int64_t res_stride, uint16_t* out, int64_t T, int top_k, int64_t H, int64_t R, bool bf16,
                               cudaStream_t s) {
  const int64_t threads = T * (H / 8);
  const auto fn = bf16 ? (wide ? combine_kernel<true, true> : combine_kernel<true, false>)
                       : (wide ? combine_kernel<false, true> : combine_kernel<false, false>);
  return launch_dependent(fn, dim3((unsigned)((threads + 255) / 256)), 256, 0, s, y, place, weights, residual, res_stride, out,
                          T, top_k, H, R);
}

}  // namespace awq
