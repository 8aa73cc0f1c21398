// The 4-bit paged cache: rotary append and read-back.  Layout of a unit: include/awq.h.
#include <cfloat>

#include "awq_host.h"
#include "awq_internal.h"
#include "awq_types.cuh"

namespace awq {
namespace {

// Both kernels: D / 8 lanes for each head of a token, eight channels a lane: one 16-byte access, one AWQ word of the keys,
// two halves of the values.  The floor is HBM's: 8165 tokens of 32 + 32 + 32 heads move 305 MB in 77 us, 3.9 TB/s
// (74 us when all channels turn, in halves).  In a capture the warps wait for memory first (long scoreboard 4.4 of an
// issue's stalls) with 66 % of the issue slots busy; without any one of the rotation, the stores or the check for ties it
// still takes 70 to 73, and reading further ahead changed nothing.  64 registers, for four CTAs an SM, spill 56 to 60 bytes
// in the general rotation, 20 to 24 with halves, none with neighbours.  Reading back moves 169 MB in 34 us, 5.0 TB/s,
// with the same first stall (5.2): a lane's value halves are two bytes each, so a token uses a quarter of the sectors that it
// touches.  64 tokens of 32 + 8 + 8 heads take 4 us.
constexpr int kAThreads = 256;
constexpr int kAWarps = kAThreads / 32;
constexpr int kACtas = 4;  // resident on an SM

template <bool BF16>
__device__ __forceinline__ void widen8(const uint4& v, F2 (&x)[4]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const float2 f = unpack2<BF16>(w[p]);
    x[p] = F2(f.x, f.y);
  }
}
template <bool BF16>
__device__ __forceinline__ uint32_t narrow2(F2 x) {
  const float2 f = x.get();
  return pack2<BF16>(f.x, f.y);
}

// How the channels turn: all of them, in pairs (i, i + D / 2) or (2i, 2i + 1), or any other way.  With the first two known
// the loops over the heads have no choices left: 74 and 71 us instead of 79 and 77 for 8165 tokens of 32 + 32 + 32
// heads of 128 channels.
enum Rotation { kHalves, kNeighbours, kAnyRotation };

// The rotation of a lane's eight channels, the same for every head of a token: x c + partner s, with the sine's sign
// that of the channel's half (a c + b (-s) rounds as a c - b s).  Every product and sum is rounded by itself, so the codes
// made from the result are a function of the inputs alone.  The products are fused multiply-adds of -0, a value that the
// compiler does not know (mul.rn.f32x2 with add.rn.f32x2 would not do: the pair was seen to come out as one fused
// operation).
template <int LANES, bool BF16, Rotation HOW>
struct Turn {
  F2 c[4], s[4], minus_zero;
  int src[2];   // pairs (i, i + rot / 2): the lane that holds the partners of each four channels
  bool in[2];   // of each four channels: whether they turn
  int rot, odd;
  bool interleaved;

  __device__ __forceinline__ void load(const float* row, const Kv4Rope& rope, bool ok, float zero, int lane) {
    minus_zero = F2(zero, zero);
    rot = !ok ? 0 : HOW == kAnyRotation ? rope.rot : LANES * 8;
    interleaved = HOW == kAnyRotation ? rope.interleaved : HOW == kNeighbours;
    const int half = rot / 2;
    odd = half / 4 % 2;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int at = 8 * lane + 4 * h;
      in[h] = at < rot;
      src[h] = lane;
      if (interleaved) {
        const float2 cv = in[h] ? *reinterpret_cast<const float2*>(row + at / 2) : make_float2(0.f, 0.f);
        const float2 sv = in[h] ? *reinterpret_cast<const float2*>(row + half + at / 2) : make_float2(0.f, 0.f);
        c[2 * h] = F2(cv.x, cv.x);
        c[2 * h + 1] = F2(cv.y, cv.y);
        s[2 * h] = F2(-sv.x, sv.x);
        s[2 * h + 1] = F2(-sv.y, sv.y);
      } else {
        const bool first = at < half;
        const int partner = !in[h] ? at : first ? at + half : at - half;
        src[h] = partner / 8;
        const int i = first ? at : partner;
        const float4 cv = in[h] ? *reinterpret_cast<const float4*>(row + i) : make_float4(0.f, 0.f, 0.f, 0.f);
        const float4 sv = in[h] ? *reinterpret_cast<const float4*>(row + half + i) : make_float4(0.f, 0.f, 0.f, 0.f);
        const float sg = first ? -1.f : 1.f;
        c[2 * h] = F2(cv.x, cv.y);
        c[2 * h + 1] = F2(cv.z, cv.w);
        s[2 * h] = F2(sg * sv.x, sg * sv.y);
        s[2 * h + 1] = F2(sg * sv.z, sg * sv.w);
      }
    }
  }
  __device__ __forceinline__ F2 one(F2 x, F2 other, int p) const {
    return add2(fma2(x, c[p], minus_zero), fma2(other, s[p], minus_zero));
  }
  // The turned channels of raw; every lane of the warp takes part.
  __device__ __forceinline__ void apply(const uint4& raw, F2 (&x)[4]) const {
    widen8<BF16>(raw, x);
    if (HOW == kAnyRotation && rot == 0) return;
    F2 other[4];
    if (interleaved) {
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const float2 f = x[p].get();
        other[p] = F2(f.y, f.x);
      }
    } else {
      uint4 w = raw;
      if (HOW == kHalves) {
        constexpr int kFar = LANES / 2;
        w = make_uint4(__shfl_xor_sync(0xFFFFFFFFu, raw.x, kFar, LANES), __shfl_xor_sync(0xFFFFFFFFu, raw.y, kFar, LANES),
                       __shfl_xor_sync(0xFFFFFFFFu, raw.z, kFar, LANES), __shfl_xor_sync(0xFFFFFFFFu, raw.w, kFar, LANES));
      } else {
        if (odd) w = make_uint4(raw.z, raw.w, raw.x, raw.y);  // with an odd number of fours in a half, the other four of their lane
        w = make_uint4(__shfl_sync(0xFFFFFFFFu, w.x, src[0], LANES), __shfl_sync(0xFFFFFFFFu, w.y, src[0], LANES),
                       __shfl_sync(0xFFFFFFFFu, w.z, src[1], LANES), __shfl_sync(0xFFFFFFFFu, w.w, src[1], LANES));
      }
      widen8<BF16>(w, other);
    }
#pragma unroll
    for (int p = 0; p < 4; ++p)
      if (HOW != kAnyRotation || in[p / 2]) x[p] = one(x[p], other[p], p);
  }
};

// d / 15 rounded once: a quotient next to the right one, corrected by its exact remainder times the rounded reciprocal
// (Markstein 1990).  An infinite d gives a NaN, which the caller's minimum drops for its bound.
__device__ __forceinline__ float fifteenth(float d) {
  constexpr float kInv = 1.f / 15.f;
  const float q = d * kInv;
  return fmaf(fmaf(-15.f, q, d), kInv, q);
}

// Scale and zero of a head (returned, fp16 each) and this lane's eight codes: u[j] is a float 1.5 * 2^23 + code, so
// that the code stands in its low bits.
constexpr float kMagic = 12582912.f;
template <int LANES>
__device__ __forceinline__ uint32_t quantize8(const F2 (&pairs)[4], uint32_t (&u)[8]) {
  float x[8];
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const float2 f = pairs[p].get();
    x[2 * p] = f.x;
    x[2 * p + 1] = f.y;
  }
  float low = min_nan(min_nan(x[0], x[1], x[2]), min_nan(x[3], x[4], x[5]), min_nan(x[6], x[7], x[7]));
  float high = max_nan(max_nan(x[0], x[1], x[2]), max_nan(x[3], x[4], x[5]), max_nan(x[6], x[7], x[7]));
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) {
    const float l = __shfl_xor_sync(0xFFFFFFFFu, low, o, LANES), h = __shfl_xor_sync(0xFFFFFFFFu, high, o, LANES);
    low = min_nan(low, l, l);
    high = max_nan(high, h, h);
  }
  const __half zero = __float2half_rn(fminf(fmaxf(low, -65504.f), 65504.f));
  const __half scale = __float2half_rn(fminf(fifteenth(__fsub_rn(high, low)), 65504.f));
  const float s = __half2float(scale), z = __half2float(zero);
  float inv;  // a reciprocal to a few units in the last place is enough
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  if (s == 0.f) inv = 0.f;
  // (x - z) * inv is within 2^-18 of the correctly rounded quotient, so only next to a half-integer (0.5 - 2^-17 and
  // more away from the integer) can its integer differ; there, and where the rounding of zero and scale puts a code outside 0..15, the slow way is taken.
  // Adding 1.5 * 2^23 rounds to the nearest integer, ties to even.
  float far = fmaxf(-(low - z) * inv, (high - z) * inv - 15.f);
  const F2 minus_z(-z, -z), inv2(inv, inv), magic(kMagic, kMagic), minus(-1.f, -1.f);
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const F2 d = add2(pairs[p], minus_z), m = fma2(d, inv2, magic);
    const float2 e = fma2(d, inv2, fma2(m, minus, magic)).get(), w = m.get();
    far = fmaxf(far, fmaxf(fabsf(e.x), fabsf(e.y)));
    u[2 * p] = __float_as_uint(w.x);
    u[2 * p + 1] = __float_as_uint(w.y);
  }
  const bool finite = low >= -FLT_MAX && high <= FLT_MAX;
  if (!(far < 0.49999f && finite)) {
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
  float minus_zero;
};

// A round is what a warp does at once: 32 / LANES heads of a token.  The rounds of all tokens (for the append, each one's
// queries, then keys, then values) are cut into equal contiguous ranges, one for each warp of a grid that fills the GPU
// once (a token for each warp instead came to 1.7 waves of warps for 8165 tokens: 80 us instead of 77).
struct WarpShare {
  int64_t token;  // the range begins at round `first` of this token
  int first, rounds;
};
__device__ __forceinline__ WarpShare share_of(int64_t total, int rounds) {
  const int64_t warps = gridDim.x * (int64_t)kAWarps, me = blockIdx.x * (int64_t)kAWarps + threadIdx.x / 32;
  const int64_t each = total / warps, rest = total - each * warps, begin = me * each + min(me, rest);
  WarpShare s;
  s.token = begin / rounds;
  s.first = (int)(begin - s.token * rounds);
  s.rounds = (int)each + (me < rest ? 1 : 0);
  return s;
}
// Blocks of a grid for so many rounds.
unsigned blocks_for(int64_t rounds, int resident) {
  const int64_t most = resident * (int64_t)device_sm_count(), blocks = (rounds + kAWarps - 1) / kAWarps;
  return (unsigned)(blocks < most ? blocks : most);
}

template <int D, bool BF16, Rotation HOW>
__global__ void __launch_bounds__(kAThreads, kACtas) kv4_append_kernel(const AppendArgs a) {
  // a dependent launched early waits for this grid before it reads what is written here
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int LANES = D / 8, HEADS = 32 / LANES;  // lanes of a head, heads of a warp
  const int sub = threadIdx.x % 32 / LANES, lane = threadIdx.x % LANES;
  const int q_rounds = (a.heads + HEADS - 1) / HEADS, kv_rounds = (a.c.kv_heads + HEADS - 1) / HEADS;
  const int rounds = q_rounds + 2 * kv_rounds;
  const WarpShare share = share_of(a.T * rounds, rounds);
  int64_t t = share.token;
  const int own = sub * D + 8 * lane;     // this lane's place in a round
  const uint4 none = make_uint4(0u, 0u, 0u, 0u);
  auto read = [&](const uint16_t* at, bool in) { return in ? *reinterpret_cast<const uint4*>(at) : none; };
  Turn<LANES, BF16, HOW> turn;
  for (int left = share.rounds, first = share.first; left > 0; ++t, first = 0) {
    const int last = min(first + left, rounds);
    left -= last - first;
    const int64_t pos = a.rope.rot ? a.rope.positions[t] : 0;
    const bool pos_ok = !a.rope.rot || (pos >= 0 && pos < a.rope.max_pos);
    const int64_t slot = a.c.kv_heads ? a.slots[t] : -1;
    {
      const uint16_t* src = a.q + t * a.q_stride + first * (HEADS * D) + own;
      uint16_t* dst = a.q_out + t * a.q_out_stride + first * (HEADS * D) + own;
      const int end = min(last, q_rounds);
      int h = first * HEADS + sub;
      uint4 next = read(src, first < end && h < a.heads);
      turn.load(a.rope.table + (pos_ok ? pos * a.rope.rot : 0), a.rope, pos_ok && first < q_rounds + kv_rounds, a.minus_zero, lane);
      for (int r = first; r < end; ++r) {
        const uint4 raw = next;
        const bool mine = h < a.heads;
        h += HEADS;
        src += HEADS * D;
        next = read(src, r + 1 < end && h < a.heads);
        F2 x[4];
        turn.apply(raw, x);
        if (mine)
          *reinterpret_cast<uint4*>(dst) =
              pos_ok ? make_uint4(narrow2<BF16>(x[0]), narrow2<BF16>(x[1]), narrow2<BF16>(x[2]), narrow2<BF16>(x[3])) : none;
        dst += HEADS * D;
      }
    }
    if (!(pos_ok && slot >= 0 && slot < a.c.num_pages * a.c.page_size)) continue;  // the whole warp
    int in_page;
    const int64_t page = page_of(slot, a.c.page_size, in_page);
    const int units = a.c.page_size / kKv4Unit, token = in_page % kKv4Unit;
    const int64_t head_bytes = units * kv4_unit_bytes(D);
    uint8_t* unit0 = a.cache + (page * a.c.kv_heads * units + in_page / kKv4Unit) * kv4_unit_bytes(D);
#pragma unroll
    for (int is_v = 0; is_v < 2; ++is_v) {
      const int base = q_rounds + is_v * kv_rounds;  // the first round of the keys, or of the values
      const int begin_r = max(first - base, 0), end_r = min(last - base, kv_rounds);
      int h = begin_r * HEADS + sub;
      const uint16_t* src = (is_v ? a.v + t * a.v_stride : a.k + t * a.k_stride) + begin_r * (HEADS * D) + own;
      uint8_t* unit = unit0 + h * head_bytes;
      const int code_at = is_v ? kv4_value_offset(D, token, 8 * lane) : kv4_key_offset(D, token) + 4 * lane;
      const int meta_at = kv4_meta_offset(D, token) + 4 * is_v;
      uint4 next = read(src, begin_r < end_r && h < a.c.kv_heads);
      for (int r = begin_r; r < end_r; ++r) {
        const uint4 raw = next;
        const bool mine = h < a.c.kv_heads;
        h += HEADS;
        src += HEADS * D;
        next = read(src, r + 1 < end_r && h < a.c.kv_heads);
        F2 x[4];
        if (is_v)
          widen8<BF16>(raw, x);
        else
          turn.apply(raw, x);
        uint32_t u[8];
        const uint32_t meta = quantize8<LANES>(x, u);
        if (mine) {
          if (is_v) {  // the channels of a lane are two halves, four bytes apart
#pragma unroll
            for (int p = 0; p < 2; ++p)
              *reinterpret_cast<uint16_t*>(unit + code_at + 4 * p) =
                  (uint16_t)(u[4 * p] + (u[4 * p + 1] << 4) + (u[4 * p + 2] << 8) + (u[4 * p + 3] << 12));
          } else {  // AWQ order: 0, 2, 4, 6, 1, 3, 5, 7; the upper bits of the floats are taken off the sum
            constexpr uint32_t kOff = 0x4B400000u * 0x11111111u;
            *reinterpret_cast<uint32_t*>(unit + code_at) = u[0] + (u[2] << 4) + (u[4] << 8) + (u[6] << 12) + (u[1] << 16) +
                                                           (u[3] << 20) + (u[5] << 24) + (u[7] << 28) - kOff;
          }
          if (lane == 0) *reinterpret_cast<uint32_t*>(unit + meta_at) = meta;
        }
        unit += HEADS * head_bytes;
      }
    }
  }
}

// zero + u * scale of eight codes, given as pairs in bits 0-3 and 16-19 of w >> shift: exact halves 1024 + u first.
template <bool BF16>
__device__ __forceinline__ uint32_t two_values(uint32_t pair, float2 sz) {
  const uint32_t w = (pair & 0x000F000Fu) | 0x64006400u;
  const float2 f = __half22float2(__hsub2(*reinterpret_cast<const __half2*>(&w), __float2half2_rn(1024.f)));
  return pack2<BF16>(__fadd_rn(sz.y, __fmul_rn(f.x, sz.x)), __fadd_rn(sz.y, __fmul_rn(f.y, sz.x)));
}

// Rounds cut as in the append; the reads of kGBatch of them are on the way at once (with 8165 tokens of 32 heads: 2 on
// 6 CTAs an SM 34 us, 4 on 4 35, 8 on 4 38; a CTA for each token, one at a time, 37).
constexpr int kGBatch = 2, kGCtas = 6;

template <int D, bool BF16>
__global__ void __launch_bounds__(kAThreads, kGCtas)
kv4_gather_kernel(const uint8_t* __restrict__ cache, const int64_t* __restrict__ slots, uint16_t* __restrict__ k,
                  uint16_t* __restrict__ v, const Kv4Shape c, int64_t T) {
  constexpr int LANES = D / 8, HEADS = 32 / LANES;
  const int sub = threadIdx.x % 32 / LANES, lane = threadIdx.x % LANES;
  const int rounds = (c.kv_heads + HEADS - 1) / HEADS;
  const WarpShare mine = share_of(T * rounds, rounds);
  int64_t t = mine.token;
  const int units = c.page_size / kKv4Unit;
  const int64_t head_bytes = units * kv4_unit_bytes(D);
  for (int left = mine.rounds, first = mine.first; left > 0; ++t, first = 0) {
    const int last = min(first + left, rounds);
    left -= last - first;
    const int64_t slot = slots[t];
    const bool in = slot >= 0 && slot < c.num_pages * c.page_size;
    int in_page;
    const int64_t page = page_of(in ? slot : 0, c.page_size, in_page);
    const int token = in_page % kKv4Unit;
    const uint8_t* unit0 = cache + (page * c.kv_heads * units + in_page / kKv4Unit) * kv4_unit_bytes(D);
    for (int r = first; r < last; r += kGBatch) {
      uint2 m[kGBatch];
      uint32_t w[kGBatch], a[kGBatch], b[kGBatch];
#pragma unroll
      for (int i = 0; i < kGBatch; ++i) {
        const int h = (r + i) * HEADS + sub;
        const uint8_t* unit = unit0 + h * head_bytes;
        m[i] = make_uint2(0u, 0u);
        w[i] = a[i] = b[i] = 0u;
        if (in && r + i < last && h < c.kv_heads) {
          m[i] = *reinterpret_cast<const uint2*>(unit + kv4_meta_offset(D, token));
          w[i] = *reinterpret_cast<const uint32_t*>(unit + kv4_key_offset(D, token) + 4 * lane);
          a[i] = *reinterpret_cast<const uint16_t*>(unit + kv4_value_offset(D, token, 8 * lane));
          b[i] = *reinterpret_cast<const uint16_t*>(unit + kv4_value_offset(D, token, 8 * lane + 4));
        }
      }
#pragma unroll
      for (int i = 0; i < kGBatch; ++i) {
        const int h = (r + i) * HEADS + sub;
        if (r + i >= last || h >= c.kv_heads) break;
        const float2 ks = unpack2<false>(m[i].x), vs = unpack2<false>(m[i].y);
        const int64_t at = (t * c.kv_heads + h) * D + 8 * lane;
        // codes 0 with scale and zero 0, of a slot outside the cache, are zeros
        if (k)
          *reinterpret_cast<uint4*>(k + at) = make_uint4(two_values<BF16>(w[i], ks), two_values<BF16>(w[i] >> 4, ks),
                                                         two_values<BF16>(w[i] >> 8, ks), two_values<BF16>(w[i] >> 12, ks));
        // a half holds its four codes side by side: nibbles 0, 1 and 2, 3 become pairs
        if (v)
          *reinterpret_cast<uint4*>(v + at) =
              make_uint4(two_values<BF16>(a[i] | a[i] << 12, vs), two_values<BF16>(a[i] >> 8 | a[i] << 4, vs),
                         two_values<BF16>(b[i] | b[i] << 12, vs), two_values<BF16>(b[i] >> 8 | b[i] << 4, vs));
      }
    }
  }
}

template <int D, bool BF16>
void run_append(const AppendArgs& a, unsigned grid, cudaStream_t s) {
  const auto fn = a.rope.rot != D        ? kv4_append_kernel<D, BF16, kAnyRotation>
                  : a.rope.interleaved ? kv4_append_kernel<D, BF16, kNeighbours>
                                       : kv4_append_kernel<D, BF16, kHalves>;
  fn<<<grid, kAThreads, 0, s>>>(a);
}

}  // namespace

cudaError_t launch_kv4_append(const uint16_t* q, const uint16_t* k, const uint16_t* v, int64_t q_stride,
                              int64_t k_stride, int64_t v_stride, const int64_t* slots, const Kv4Rope& rope,
                              uint16_t* q_out, int64_t q_out_stride, uint8_t* cache, const Kv4Shape& c, int64_t T,
                              int heads, bool bf16, cudaStream_t s) {
  const int at_once = 256 / c.dim;
  const int64_t rounds = T * ((heads + at_once - 1) / at_once + 2 * ((c.kv_heads + at_once - 1) / at_once));
  const unsigned grid = blocks_for(rounds, kACtas);
  const AppendArgs a{q, k, v, q_stride, k_stride, v_stride, slots, rope, q_out, q_out_stride, cache, c, T, heads, -0.f};
  if (c.dim == 128)
    bf16 ? run_append<128, true>(a, grid, s) : run_append<128, false>(a, grid, s);
  else
    bf16 ? run_append<64, true>(a, grid, s) : run_append<64, false>(a, grid, s);
  return cudaGetLastError();
}

cudaError_t launch_kv4_gather(const uint8_t* cache, const int64_t* slots, uint16_t* k, uint16_t* v, const Kv4Shape& c,
                              int64_t T, bool bf16, cudaStream_t s) {
  const auto fn = c.dim == 128 ? (bf16 ? kv4_gather_kernel<128, true> : kv4_gather_kernel<128, false>)
                               : (bf16 ? kv4_gather_kernel<64, true> : kv4_gather_kernel<64, false>);
  const int at_once = 256 / c.dim;
  fn<<<blocks_for(T * ((c.kv_heads + at_once - 1) / at_once), kGCtas), kAThreads, 0, s>>>(cache, slots, k, v, c, T);
  return cudaGetLastError();
}

}  // namespace awq
