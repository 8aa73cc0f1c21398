// The 4-bit paged cache: rotary append and read-back.  Layout of a unit: include/awq.h.
#include <cfloat>

#include "awq_host.h"
#include "awq_internal.h"
#include "awq_types.cuh"

namespace awq {
namespace {

constexpr int kAThreads = 256;

// (t, head) items are handled by D / 4 lanes each, four channels a lane.
template <int D, bool BF16>
__device__ __forceinline__ void load4(const uint16_t* row, int lane, float (&x)[4]) {
  const uint2 v = *reinterpret_cast<const uint2*>(row + 4 * lane);
  const float2 a = unpack2<BF16>(v.x), b = unpack2<BF16>(v.y);
  x[0] = a.x;
  x[1] = a.y;
  x[2] = b.x;
  x[3] = b.y;
}

// Rotates the four channels of this lane.  Every product and sum is rounded by itself (no fused multiply-add),
// so the codes made from the result are a function of the inputs alone.
template <int LANES>
__device__ __forceinline__ void rotate4(float (&x)[4], const float* row, int rot, bool interleaved, int lane) {
  const int half = rot / 2;
  if (interleaved) {
    if (4 * lane < rot) {
      const float2 c = *reinterpret_cast<const float2*>(row + 2 * lane);
      const float2 s = *reinterpret_cast<const float2*>(row + half + 2 * lane);
      const float a0 = x[0], b0 = x[1], a1 = x[2], b1 = x[3];
      x[0] = __fsub_rn(__fmul_rn(a0, c.x), __fmul_rn(b0, s.x));
      x[1] = __fadd_rn(__fmul_rn(b0, c.x), __fmul_rn(a0, s.x));
      x[2] = __fsub_rn(__fmul_rn(a1, c.y), __fmul_rn(b1, s.y));
      x[3] = __fadd_rn(__fmul_rn(b1, c.y), __fmul_rn(a1, s.y));
    }
    return;
  }
  // pairs (i, i + half): the partner's four channels are rot / 8 lanes away
  const int off = rot / 8;
  const bool first = lane < off, in = 4 * lane < rot;
  const int src = !in ? lane : first ? lane + off : lane - off;
  float other[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) other[j] = __shfl_sync(0xFFFFFFFFu, x[j], src, LANES);
  if (in) {
    const int i = 4 * (first ? lane : lane - off);
    const float4 c = *reinterpret_cast<const float4*>(row + i);
    const float4 s = *reinterpret_cast<const float4*>(row + half + i);
    const float cv[4] = {c.x, c.y, c.z, c.w}, sv[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float p = __fmul_rn(x[j], cv[j]), q = __fmul_rn(other[j], sv[j]);
      x[j] = first ? __fsub_rn(p, q) : __fadd_rn(p, q);
    }
  }
}

// Scale and zero of a head and this lane's four codes.
template <int LANES>
__device__ __forceinline__ void quantize4(const float (&x)[4], uint32_t (&u)[4], __half& scale, __half& zero) {
  float low = FLT_MAX, high = -FLT_MAX;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const bool finite = x[j] - x[j] == 0.f;
    low = fminf(low, x[j]);
    high = finite ? fmaxf(high, x[j]) : INFINITY;
  }
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) {
    low = fminf(low, __shfl_xor_sync(0xFFFFFFFFu, low, o, LANES));
    high = fmaxf(high, __shfl_xor_sync(0xFFFFFFFFu, high, o, LANES));
  }
  zero = __float2half_rn(fminf(fmaxf(low, -65504.f), 65504.f));
  scale = __float2half_rn(fminf(__fdiv_rn(__fsub_rn(high, low), 15.0f), 65504.f));
  const float s = __half2float(scale), z = __half2float(zero);
  const bool poison = high > FLT_MAX;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    u[j] = !poison && s > 0.f ? (uint32_t)fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(x[j], z), s)), 0.f), 15.f) : 0u;
  if (poison) {
    scale = __ushort_as_half((unsigned short)0x7E00);
    zero = __ushort_as_half((unsigned short)0);
  }
}

struct AppendArgs {
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  const int64_t* slots;
  Kv4Rope rope;
  uint16_t* q_out;
  int64_t q_out_stride;
  uint8_t* cache;
  Kv4Shape c;
  int64_t T;
  int heads;
};

// The unit of `slot`'s token and head, nullptr for a slot outside the cache.
__device__ __forceinline__ uint8_t* unit_of(uint8_t* cache, const Kv4Shape& c, int dim, int64_t slot, int head) {
  if (slot < 0 || slot >= c.num_pages * c.page_size) return nullptr;
  const int64_t page = slot / c.page_size;
  const int in_page = (int)(slot - page * c.page_size);
  const int units = c.page_size / kKv4Unit;
  return cache + ((page * c.kv_heads + head) * units + in_page / kKv4Unit) * kv4_unit_bytes(dim);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kAThreads) kv4_append_kernel(AppendArgs a) {
  constexpr int LANES = D / 4;
  const int lane = threadIdx.x % LANES;
  const int per = a.heads + 2 * a.c.kv_heads;
  const int64_t item = (blockIdx.x * (int64_t)kAThreads + threadIdx.x) / LANES;
  // lanes past the end stay for the shuffles and touch no memory
  const bool in = item < a.T * per;
  const int64_t t = in ? item / per : 0;
  const int head = in ? (int)(item - t * per) : 0;
  const bool is_q = head < a.heads, is_k = !is_q && head < a.heads + a.c.kv_heads;
  const int h = is_q ? head : is_k ? head - a.heads : head - a.heads - a.c.kv_heads;
  float x[4] = {0.f, 0.f, 0.f, 0.f};
  if (in) {
    const uint16_t* row = is_q ? a.q + t * a.q_stride : is_k ? a.k + t * a.k_stride : a.v + t * a.v_stride;
    load4<D, BF16>(row + h * D, lane, x);
  }
  const int64_t pos = a.rope.rot && in ? a.rope.positions[t] : 0;
  const bool pos_ok = !a.rope.rot || (pos >= 0 && pos < a.rope.max_pos);
  const bool turns = in && a.rope.rot && pos_ok && (is_q || is_k);
  // a lane outside the table takes part in the shuffles with a rotation of nothing
  rotate4<LANES>(x, a.rope.table + (turns ? pos * a.rope.rot : 0), turns ? a.rope.rot : 0, a.rope.interleaved, lane);
  uint32_t u[4];
  __half scale, zero;
  quantize4<LANES>(x, u, scale, zero);
  const uint32_t part = u[0] | u[2] << 4 | u[1] << 16 | u[3] << 20;  // AWQ order: 0, 2, 4, 6, 1, 3, 5, 7
  const uint32_t next = __shfl_down_sync(0xFFFFFFFFu, part, 1, LANES);
  if (!in) return;
  if (is_q) {
    const uint2 o = pos_ok ? make_uint2(pack2<BF16>(x[0], x[1]), pack2<BF16>(x[2], x[3])) : make_uint2(0u, 0u);
    *reinterpret_cast<uint2*>(a.q_out + t * a.q_out_stride + h * D + 4 * lane) = o;
    return;
  }
  const int64_t slot = a.slots[t];
  uint8_t* unit = pos_ok ? unit_of(a.cache, a.c, D, slot, h) : nullptr;
  if (!unit) return;
  const int token = (int)(slot % kKv4Unit);
  if (is_k) {
    if (lane % 2 == 0)
      *reinterpret_cast<uint32_t*>(unit + kv4_key_offset(D, token) + 2 * lane) = part | next << 8;
  } else {
    *reinterpret_cast<uint16_t*>(unit + kv4_value_offset(D, token, 4 * lane)) =
        (uint16_t)(u[0] | u[1] << 4 | u[2] << 8 | u[3] << 12);
  }
  if (lane == 0)
    *reinterpret_cast<uint32_t*>(unit + kv4_meta_offset(D, token) + (is_k ? 0 : 4)) =
        (uint32_t)__half_as_ushort(scale) | (uint32_t)__half_as_ushort(zero) << 16;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kAThreads)
kv4_gather_kernel(const uint8_t* cache, const int64_t* slots, uint16_t* k, uint16_t* v, Kv4Shape c, int64_t T) {
  constexpr int LANES = D / 4;
  const int lane = threadIdx.x % LANES;
  const int64_t item = (blockIdx.x * (int64_t)kAThreads + threadIdx.x) / LANES;
  if (item >= T * c.kv_heads) return;
  const int64_t t = item / c.kv_heads;
  const int h = (int)(item - t * c.kv_heads);
  const int64_t slot = slots[t];
  const uint8_t* unit = unit_of(const_cast<uint8_t*>(cache), c, D, slot, h);
  const int token = unit ? (int)(slot % kKv4Unit) : 0;
  const int64_t at = (t * c.kv_heads + h) * D + 4 * lane;
  const uint2 m = unit ? *reinterpret_cast<const uint2*>(unit + kv4_meta_offset(D, token)) : make_uint2(0u, 0u);
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    uint16_t* out = kv ? v : k;
    if (!out) continue;
    const float2 sz = unpack2<false>(kv ? m.y : m.x);
    float f[4] = {0.f, 0.f, 0.f, 0.f};
    if (unit) {
      uint32_t codes;  // the four codes in 4-bit fields 0, 4, 8, 12
      if (kv) {
        codes = *reinterpret_cast<const uint16_t*>(unit + kv4_value_offset(D, token, 4 * lane));
      } else {
        const uint32_t w = *reinterpret_cast<const uint32_t*>(unit + kv4_key_offset(D, token) + (lane / 2) * 4) >> (8 * (lane % 2));
        codes = (w & 15u) | (w >> 16 & 15u) << 4 | (w >> 4 & 15u) << 8 | (w >> 20 & 15u) << 12;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = __fadd_rn(sz.y, __fmul_rn((float)(codes >> (4 * j) & 15u), sz.x));
    }
    *reinterpret_cast<uint2*>(out + at) = make_uint2(pack2<BF16>(f[0], f[1]), pack2<BF16>(f[2], f[3]));
  }
}

}  // namespace

cudaError_t launch_kv4_append(const uint16_t* q, const uint16_t* k, const uint16_t* v, int64_t q_stride,
                              int64_t k_stride, int64_t v_stride, const int64_t* slots, const Kv4Rope& rope,
                              uint16_t* q_out, int64_t q_out_stride, uint8_t* cache, const Kv4Shape& c, int64_t T,
                              int heads, bool bf16, cudaStream_t s) {
  const AppendArgs a{q, k, v, q_stride, k_stride, v_stride, slots, rope, q_out, q_out_stride, cache, c, T, heads};
  const int64_t blocks = (T * (heads + 2 * c.kv_heads) * (c.dim / 4) + kAThreads - 1) / kAThreads;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  const auto fn = c.dim == 128 ? (bf16 ? kv4_append_kernel<128, true> : kv4_append_kernel<128, false>)
                               : (bf16 ? kv4_append_kernel<64, true> : kv4_append_kernel<64, false>);
  fn<<<(unsigned)blocks, kAThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv4_gather(const uint8_t* cache, const int64_t* slots, uint16_t* k, uint16_t* v, const Kv4Shape& c,
                              int64_t T, bool bf16, cudaStream_t s) {
  const int64_t blocks = (T * c.kv_heads * (c.dim / 4) + kAThreads - 1) / kAThreads;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  const auto fn = c.dim == 128 ? (bf16 ? kv4_gather_kernel<128, true> : kv4_gather_kernel<128, false>)
                               : (bf16 ? kv4_gather_kernel<64, true> : kv4_gather_kernel<64, false>);
  fn<<<(unsigned)blocks, kAThreads, 0, s>>>(cache, slots, k, v, c, T);
  return cudaGetLastError();
}

}  // namespace awq
