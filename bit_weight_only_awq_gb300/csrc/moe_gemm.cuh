// What the two kernels of the grouped product share: operands from codes, the experts' tables, a CTA's share of the work.
#pragma once

#include "awq_internal.h"
#include "awq_ptx.cuh"
#include "awq_types.cuh"

namespace awq {
namespace {

// Operands (q - z) 2^-kDown, exact, of a word of eight codes: k pairs 0..3.  A masked nibble is a subnormal 16-bit number, q or
// 16 q of the smallest (in bf16 16 q reaches the lowest bit of the exponent, where numbers are still as far apart); one
// multiplication and addition gives it its size and takes the zero point off.  One AND and one fma for two codes: 315
// cycles a group for eight warps, where exponents put in by AND and OR took 670.
template <bool BF16>
constexpr int kDown = BF16 ? 7 : 10;
template <bool BF16>
__device__ __forceinline__ uint32_t fma16(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  if constexpr (BF16) asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  else asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
template <bool BF16>
__device__ __forceinline__ void operands(uint32_t w, uint32_t z, uint32_t* o, int at) {
  constexpr uint32_t kOne = BF16 ? 0x7E807E80u : 0x74007400u;        // 2^126, 2^14
  constexpr uint32_t kSixteenth = BF16 ? 0x7C807C80u : 0x64006400u;  // 2^122, 2^10
  const uint32_t v = w >> 8;
  o[at] = fma16<BF16>(w & 0x000F000Fu, kOne, z);
  o[at + 1] = fma16<BF16>(w & 0x00F000F0u, kSixteenth, z);
  o[at + 2] = fma16<BF16>(v & 0x000F000Fu, kOne, z);
  o[at + 3] = fma16<BF16>(v & 0x00F000F0u, kSixteenth, z);
}

constexpr int kMinUnits = 4;  // groups that a CTA gets at least of what is cut along K

// What a CTA works on, in order: parts of tiles, groups g0 .. g1 - 1 of each.
struct Walk {
  int grid, me, groups, rounds, tiles;  // whole rounds of tiles; the tiles that are left
  int round, u, u1;
  long long units;
  int ctas;
  __device__ __forceinline__ Walk(int total, int groups_) : grid(gridDim.x), me(blockIdx.x), groups(groups_) {
    rounds = total % grid == 0 ? total / grid : max(0, total / grid - 1);
    tiles = total - rounds * grid;
    units = (long long)tiles * groups;
    ctas = (int)max(1ll, min((long long)grid, units / kMinUnits));
    round = 0;
    u = me < ctas ? begin_of(me) : 0;
    u1 = me < ctas ? begin_of(me + 1) : 0;
  }
  __device__ __forceinline__ int begin_of(int cta) const { return (int)(units * cta / ctas); }
  __device__ __forceinline__ bool next(int& tile, int& g0, int& g1) {
    if (round < rounds) {
      tile = me + grid * round++;
      g0 = 0;
      g1 = groups;
      return true;
    }
    if (u >= u1) return false;
    const int t = u / groups;
    g0 = u - t * groups;
    g1 = min(groups, g0 + u1 - u);
    tile = rounds * grid + t;
    u += g1 - g0;
    return true;
  }
};

struct Tile {
  int expert, pair, row, rows;  // rows of y: row .. row + rows - 1
};
// Tables: first row of each expert, and items (row tiles) before it.  Within an expert the items of a column pair are
// neighbours, so that the CTAs of one time share weights.
template <int BT>
__device__ __forceinline__ Tile find_tile(const int* first, const int* items, int experts, int pairs, int t) {
  int lo = 0, hi = experts;  // the last expert with items[lo] * pairs <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (items[mid] * pairs <= t) lo = mid;
    else hi = mid;
  }
  const int n = items[lo + 1] - items[lo], local = t - items[lo] * pairs, count = first[lo + 1] - first[lo];
  const int pair = local / n, item = local - pair * n;
  const int share = ((count + n - 1) / n + 15) / 16 * 16;  // rows even out over an expert's items
  return Tile{lo, pair, first[lo] + item * share, min(share, count - item * share)};
}

// Tables of the experts, by one warp: offsets held to [0, R] and made to run forwards, and the items before each expert.
template <int BT>
__device__ __forceinline__ void expert_tables(const MoeGemmArgs& a, int lane, int* first, int* items) {
  int row = 0, item = 0;
  for (int e0 = 0; e0 <= a.experts; e0 += 32) {
    const int e = e0 + lane;
    int v = e <= a.experts ? min(max(a.offsets[e], 0), (int)a.R) : 0;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, v, d);
      if (lane >= d) v = max(v, o);
    }
    v = max(v, row);
    int before = __shfl_up_sync(0xFFFFFFFFu, v, 1);
    if (lane == 0) before = e0 == 0 ? v : row;  // rows before the first expert's are nobody's
    int n = e <= a.experts ? (v - before + BT - 1) / BT : 0;  // items of expert e - 1
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, n, d);
      if (lane >= d) n += o;
    }
    if (e <= a.experts) {
      first[e] = v;
      items[e] = item + n;
    }
    row = __shfl_sync(0xFFFFFFFFu, v, 31);
    item += __shfl_sync(0xFFFFFFFFu, n, 31);
  }
}

// A source row of x for row `row` of the plan's order; one that makes no sense reads row 0.
__device__ __forceinline__ int source_row(const MoeGemmArgs& a, int row) {
  const int src = a.order ? a.order[row] / a.top_k : row;
  return src >= 0 && src < a.x_rows ? src : 0;
}

// The calling warp's lanes wait for flags [from, to), all at once.
__device__ __forceinline__ bool wait_flags(const int* flags, int from, int to, int lane, volatile int* abort, int* err, int id) {
  bool seen = true;
  for (int q = from + lane; q < to && seen; q += 32) {
    const long long t0 = now_ns();
    for (uint32_t spin = 1;; ++spin) {
      int v;
      asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(flags + q) : "memory");
      if (v) break;
      if ((spin & 255u) == 0) {
        if (*abort) seen = false;
        else if (now_ns() - t0 > kWaitLimitNs) {
          if (err) atomicExch(err, id);
          *abort = 1;
          seen = false;
        }
        if (!seen) break;
      }
    }
  }
  seen = __all_sync(0xFFFFFFFFu, seen);
  __threadfence();
  return seen;
}

__device__ __forceinline__ float silu_times(float gate, float up) { return __fdividef(gate, 1.f + expf(-gate)) * up; }

}  // namespace

// Rows of up to 16 for each expert (moe_gemv.cu).
constexpr int kMoeGemvRows = 16;
constexpr size_t kMoeGemvPartBytes = (size_t)256 * kMoeGemvRows * 4;
cudaError_t launch_moe_gemv(const MoeGemmArgs& a, bool gated, bool wide, bool bf16, int* flags, float* parts, int* err,
                            cudaStream_t s);

}  // namespace awq
