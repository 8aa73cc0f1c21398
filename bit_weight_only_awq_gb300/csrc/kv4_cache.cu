// The 4-bit paged cache: rotary append and read-back.  Layout of a unit: include/awq.h.
#include <cfloat>

#include "awq_host.h"
#include "awq_internal.h"
#include "awq_types.cuh"

namespace awq {
namespace {

// Both kernels: a CTA for each token, D / 8 lanes for each of its heads, eight channels a lane: one 16-byte
// access, one AWQ word of the keys, two halves of the values.  HBM bound where there are many tokens; what the
// SMs have to do for each byte comes close to it (rotation and codes are about nine operations a channel, the
// reductions over a head four shuffles each for two or four heads at once).
constexpr int kAThreads = 256;
constexpr int kAWarps = kAThreads / 32;
constexpr int kTeamWarps = 256;  // warps that each SM should get

template <bool BF16>
__device__ __forceinline__ void widen8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const float2 f = unpack2<BF16>(w[p]);
    x[2 * p] = f.x;
    x[2 * p + 1] = f.y;
  }
}
template <bool BF16>
__device__ __forceinline__ uint4 narrow8(const float (&f)[8]) {
  return make_uint4(pack2<BF16>(f[0], f[1]), pack2<BF16>(f[2], f[3]), pack2<BF16>(f[4], f[5]), pack2<BF16>(f[6], f[7]));
}

// The rotation of a lane's eight channels, the same for every head of a token.  Every product and sum is rounded
// by itself (no fused multiply-add), so the codes made from the result are a function of the inputs alone.
template <int LANES>
struct Turn {
  float c[8], s[8];  // cosines and sines; interleaved: four of each
  int src[2];        // pairs (i, i + rot / 2): the lane that holds the partners of each four channels
  bool in[2], first[2];
  int rot, odd;
  bool interleaved;

  __device__ __forceinline__ void load(const float* row, int rot_dim, bool inter, int lane) {
    rot = rot_dim;
    interleaved = inter;
    const int half = rot / 2;
    odd = half / 4 % 2;
    if (interleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool on = 8 * lane < rot;
        c[i] = on ? row[4 * lane + i] : 0.f;
        s[i] = on ? row[half + 4 * lane + i] : 0.f;
      }
      return;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = 8 * lane + 4 * h;
      in[h] = at < rot;
      first[h] = at < half;
      const int partner = !in[h] ? at : first[h] ? at + half : at - half;
      src[h] = partner / 8;
      const int i = first[h] ? at : partner;
      const float4 cv = in[h] ? *reinterpret_cast<const float4*>(row + i) : make_float4(0.f, 0.f, 0.f, 0.f);
      const float4 sv = in[h] ? *reinterpret_cast<const float4*>(row + half + i) : make_float4(0.f, 0.f, 0.f, 0.f);
      c[4 * h] = cv.x, c[4 * h + 1] = cv.y, c[4 * h + 2] = cv.z, c[4 * h + 3] = cv.w;
      // a first half turns by - b s, a second one by + a s
      const float sg = first[h] ? -1.f : 1.f;  // a c + (-b s) rounds as a c - b s
      s[4 * h] = sg * sv.x, s[4 * h + 1] = sg * sv.y, s[4 * h + 2] = sg * sv.z, s[4 * h + 3] = sg * sv.w;
    }
  }
  // every lane of the warp takes part
  __device__ __forceinline__ void apply(float (&x)[8], int lane) const {
    if (rot == 0) return;
    if (interleaved) {
      if (8 * lane < rot) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = x[2 * i], b = x[2 * i + 1];
          x[2 * i] = __fsub_rn(__fmul_rn(a, c[i]), __fmul_rn(b, s[i]));
          x[2 * i + 1] = __fadd_rn(__fmul_rn(b, c[i]), __fmul_rn(a, s[i]));
        }
      }
      return;
    }
    float other[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) other[j] = x[j];
    if (odd) {  // with an odd number of fours in a half, the partners are the other four of their lane
#pragma unroll
      for (int j = 0; j < 8; ++j) other[j] = x[j ^ 4];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) other[j] = __shfl_sync(0xFFFFFFFFu, other[j], src[j / 4], LANES);
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (in[h]) {
#pragma unroll
        for (int j = 4 * h; j < 4 * h + 4; ++j) x[j] = __fadd_rn(__fmul_rn(x[j], c[j]), __fmul_rn(other[j], s[j]));
      }
  }
};

// Minimum and maximum that keep a NaN.
__device__ __forceinline__ float min_nan(float a, float b) {
  float r;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Scale and zero of a head (returned, fp16 each) and this lane's eight codes: u[j] is a float 1.5 * 2^23 + code, so
// that the code stands in its low bits.
constexpr float kMagic = 12582912.f;
template <int LANES>
__device__ __forceinline__ uint32_t quantize8(const float (&x)[8], uint32_t (&u)[8]) {
  float low = x[0], high = x[0];
#pragma unroll
  for (int j = 1; j < 8; ++j) {
    low = min_nan(low, x[j]);
    high = max_nan(high, x[j]);
  }
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) {
    low = min_nan(low, __shfl_xor_sync(0xFFFFFFFFu, low, o, LANES));
    high = max_nan(high, __shfl_xor_sync(0xFFFFFFFFu, high, o, LANES));
  }
  const __half zero = __float2half_rn(fminf(fmaxf(low, -65504.f), 65504.f));
  const __half scale = __float2half_rn(fminf(__fdiv_rn(__fsub_rn(high, low), 15.0f), 65504.f));
  const float s = __half2float(scale), z = __half2float(zero);
  float inv;  // a reciprocal to a few units in the last place is enough
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  if (s == 0.f) inv = 0.f;
  // (x - z) * inv is within 2^-17 of the correctly rounded quotient, so only next to a half-integer can its integer
  // differ; there, and where the rounding of zero and scale puts a code outside 0..15, the slow way is taken.
  // Adding 1.5 * 2^23 rounds to the nearest integer, ties to even.
  float far = fmaxf(-(low - z) * inv, (high - z) * inv - 15.f);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float d = __fsub_rn(x[j], z), m = fmaf(d, inv, kMagic);
    far = fmaxf(far, fabsf(fmaf(d, inv, kMagic - m)));
    u[j] = __float_as_uint(m);
  }
  const bool finite = low >= -FLT_MAX && high <= FLT_MAX;
  if (!(far < 0.4999f && finite)) {
    if (!finite) {
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] = __float_as_uint(kMagic);
      return 0x00007E00u;  // scale NaN, zero 0
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      u[j] = __float_as_uint(kMagic + (s > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(x[j], z), s)), 0.f), 15.f) : 0.f));
  }
  return (uint32_t)__half_as_ushort(scale) | (uint32_t)__half_as_ushort(zero) << 16;
}

// The page of a slot and the token's place in it (divided in 32 bits where that is enough).
__device__ __forceinline__ int64_t page_of(int64_t slot, int page_size, int& in_page) {
  const int64_t page = (slot >> 32) == 0 ? (int64_t)((uint32_t)slot / (uint32_t)page_size) : slot / page_size;
  in_page = (int)(slot - page * page_size);
  return page;
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
  int team;  // warps that share a token
};

template <int D, bool BF16>
__global__ void __launch_bounds__(kAThreads, 4) kv4_append_kernel(const AppendArgs a) {
  // a dependent launched early waits for this grid before it reads what is written here
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int LANES = D / 8, HEADS = 32 / LANES;  // lanes of a head, heads of a warp
  const int warp = threadIdx.x / 32, sub = threadIdx.x % 32 / LANES, lane = threadIdx.x % LANES;
  // `team` warps share a token
  const int team = a.team;
  const int64_t t = blockIdx.x * (int64_t)(kAWarps / team) + warp / team;
  if (t >= a.T) return;
  // rounds of HEADS heads: queries, then keys, then values
  const int q_rounds = (a.heads + HEADS - 1) / HEADS, kv_rounds = (a.c.kv_heads + HEADS - 1) / HEADS;
  const int rounds = q_rounds + 2 * kv_rounds, stride = team * gridDim.y;
  int r = blockIdx.y * team + warp % team;
  if (r >= rounds) return;
  const int own = sub * D + 8 * lane;  // this lane's place in a round
  const uint16_t* q_row = a.q + t * a.q_stride + own;
  const uint16_t* k_row = a.k + t * a.k_stride + own;
  const uint16_t* v_row = a.v + t * a.v_stride + own;
  auto read = [&](int i) {
    const int kr = i - q_rounds, vr = kr - kv_rounds;
    const uint16_t* at = kr < 0 ? q_row + i * (HEADS * D) : vr < 0 ? k_row + kr * (HEADS * D) : v_row + vr * (HEADS * D);
    const int h = (kr < 0 ? i : vr < 0 ? kr : vr) * HEADS + sub;
    return i < rounds && h < (kr < 0 ? a.heads : a.c.kv_heads) ? *reinterpret_cast<const uint4*>(at)
                                                               : make_uint4(0u, 0u, 0u, 0u);
  };
  uint4 next = read(r);
  const int64_t pos = a.rope.rot ? a.rope.positions[t] : 0;
  const bool pos_ok = !a.rope.rot || (pos >= 0 && pos < a.rope.max_pos);
  const int64_t slot = a.c.kv_heads ? a.slots[t] : -1;
  Turn<LANES> turn;
  turn.load(a.rope.table + (pos_ok ? pos * a.rope.rot : 0), pos_ok ? a.rope.rot : 0, a.rope.interleaved, lane);
  const bool keep = pos_ok && slot >= 0 && slot < a.c.num_pages * a.c.page_size;
  int in_page;
  const int64_t page = page_of(keep ? slot : 0, a.c.page_size, in_page);
  const int units = a.c.page_size / kKv4Unit, token = in_page % kKv4Unit;
  const int head_bytes = units * kv4_unit_bytes(D);
  uint8_t* unit0 = a.cache + (page * a.c.kv_heads * units + in_page / kKv4Unit) * kv4_unit_bytes(D);
  const int key_at = kv4_key_offset(D, token) + 4 * lane, value_at = kv4_value_offset(D, token, 8 * lane);
  const int meta_at = kv4_meta_offset(D, token);
  for (; r < rounds; r += stride) {
    float x[8];
    widen8<BF16>(next, x);
    next = read(r + stride);
    const int kr = r - q_rounds, vr = kr - kv_rounds;
    if (kr < 0) {
      turn.apply(x, lane);
      if (r * HEADS + sub < a.heads)
        *reinterpret_cast<uint4*>(a.q_out + t * a.q_out_stride + r * (HEADS * D) + own) =
            pos_ok ? narrow8<BF16>(x) : make_uint4(0u, 0u, 0u, 0u);
      continue;
    }
    if (vr < 0) turn.apply(x, lane);
    uint32_t u[8];
    const uint32_t meta = quantize8<LANES>(x, u);
    const int h = (vr < 0 ? kr : vr) * HEADS + sub;
    if (!keep || h >= a.c.kv_heads) continue;  // after the last shuffle of the round
    uint8_t* unit = unit0 + (int64_t)h * head_bytes;
    if (vr < 0) {  // AWQ order: 0, 2, 4, 6, 1, 3, 5, 7; the upper bits of the floats are taken off the sum
      constexpr uint32_t kOff = 0x4B400000u * 0x11111111u;
      *reinterpret_cast<uint32_t*>(unit + key_at) = u[0] + (u[2] << 4) + (u[4] << 8) + (u[6] << 12) + (u[1] << 16) +
                                                    (u[3] << 20) + (u[5] << 24) + (u[7] << 28) - kOff;
    } else {  // the channels of a lane are two halves, four bytes apart
#pragma unroll
      for (int p = 0; p < 2; ++p)
        *reinterpret_cast<uint16_t*>(unit + value_at + 4 * p) =
            (uint16_t)(u[4 * p] + (u[4 * p + 1] << 4) + (u[4 * p + 2] << 8) + (u[4 * p + 3] << 12));
    }
    if (lane == 0) *reinterpret_cast<uint32_t*>(unit + meta_at + (vr < 0 ? 0 : 4)) = meta;
  }
}

// zero + u * scale of eight codes, given as pairs in bits 0-3 and 16-19 of w >> shift: exact halves 1024 + u first.
template <bool BF16>
__device__ __forceinline__ uint32_t two_values(uint32_t pair, float2 sz) {
  const uint32_t w = (pair & 0x000F000Fu) | 0x64006400u;
  const float2 f = __half22float2(__hsub2(*reinterpret_cast<const __half2*>(&w), __float2half2_rn(1024.f)));
  return pack2<BF16>(__fadd_rn(sz.y, __fmul_rn(f.x, sz.x)), __fadd_rn(sz.y, __fmul_rn(f.y, sz.x)));
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kAThreads)
kv4_gather_kernel(const uint8_t* __restrict__ cache, const int64_t* __restrict__ slots, uint16_t* __restrict__ k,
                  uint16_t* __restrict__ v, const Kv4Shape c) {
  constexpr int LANES = D / 8, HEADS = kAThreads / LANES;
  const int lane = threadIdx.x % LANES;
  const int64_t t = blockIdx.x;
  const int64_t slot = slots[t];
  const bool in = slot >= 0 && slot < c.num_pages * c.page_size;
  int in_page;
  const int64_t page = page_of(in ? slot : 0, c.page_size, in_page);
  const int units = c.page_size / kKv4Unit, token = in_page % kKv4Unit;
  for (int h = threadIdx.x / LANES; h < c.kv_heads; h += HEADS) {
    uint4 ko = make_uint4(0u, 0u, 0u, 0u), vo = ko;
    if (in) {
      const uint8_t* unit = cache + ((page * c.kv_heads + h) * units + in_page / kKv4Unit) * kv4_unit_bytes(D);
      const uint2 m = *reinterpret_cast<const uint2*>(unit + kv4_meta_offset(D, token));
      const uint32_t w = *reinterpret_cast<const uint32_t*>(unit + kv4_key_offset(D, token) + 4 * lane);
      const uint32_t a = *reinterpret_cast<const uint16_t*>(unit + kv4_value_offset(D, token, 8 * lane));
      const uint32_t b = *reinterpret_cast<const uint16_t*>(unit + kv4_value_offset(D, token, 8 * lane + 4));
      const float2 ks = unpack2<false>(m.x), vs = unpack2<false>(m.y);
      ko = make_uint4(two_values<BF16>(w, ks), two_values<BF16>(w >> 4, ks), two_values<BF16>(w >> 8, ks),
                      two_values<BF16>(w >> 12, ks));
      // a half holds its four codes side by side: nibbles 0, 1 and 2, 3 become pairs
      vo = make_uint4(two_values<BF16>(a | a << 12, vs), two_values<BF16>(a >> 8 | a << 4, vs),
                      two_values<BF16>(b | b << 12, vs), two_values<BF16>(b >> 8 | b << 4, vs));
    }
    const int64_t at = (t * c.kv_heads + h) * D + 8 * lane;
    if (k) *reinterpret_cast<uint4*>(k + at) = ko;
    if (v) *reinterpret_cast<uint4*>(v + at) = vo;
  }
}

}  // namespace

cudaError_t launch_kv4_append(const uint16_t* q, const uint16_t* k, const uint16_t* v, int64_t q_stride,
                              int64_t k_stride, int64_t v_stride, const int64_t* slots, const Kv4Rope& rope,
                              uint16_t* q_out, int64_t q_out_stride, uint8_t* cache, const Kv4Shape& c, int64_t T,
                              int heads, bool bf16, cudaStream_t s) {
  // One warp goes through a token's heads when the tokens alone fill the GPU (what it finds out about the token,
  // its page and rotation, then serves all of them); fewer tokens get more warps, down to one round of heads each.
  const int at_once = 256 / c.dim, rounds = (heads + at_once - 1) / at_once + 2 * ((c.kv_heads + at_once - 1) / at_once);
  const int64_t room = kTeamWarps * (int64_t)device_sm_count() / T;
  const int team = room >= 8 ? 8 : room >= 4 ? 4 : room >= 2 ? 2 : 1;
  const int64_t most = (rounds + team - 1) / team;
  const unsigned split = (unsigned)(team < 8 ? 1 : room / 8 < most ? room / 8 : most);
  const int64_t blocks = (T * team + kAWarps - 1) / kAWarps;
  const AppendArgs a{q, k, v, q_stride, k_stride, v_stride, slots, rope, q_out, q_out_stride, cache, c, T, heads, team};
  const auto fn = c.dim == 128 ? (bf16 ? kv4_append_kernel<128, true> : kv4_append_kernel<128, false>)
                               : (bf16 ? kv4_append_kernel<64, true> : kv4_append_kernel<64, false>);
  fn<<<dim3((unsigned)blocks, split), kAThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_kv4_gather(const uint8_t* cache, const int64_t* slots, uint16_t* k, uint16_t* v, const Kv4Shape& c,
                              int64_t T, bool bf16, cudaStream_t s) {
  const auto fn = c.dim == 128 ? (bf16 ? kv4_gather_kernel<128, true> : kv4_gather_kernel<128, false>)
                               : (bf16 ? kv4_gather_kernel<64, true> : kv4_gather_kernel<64, false>);
  fn<<<(unsigned)T, kAThreads, 0, s>>>(cache, slots, k, v, c);
  return cudaGetLastError();
}

}  // namespace awq
