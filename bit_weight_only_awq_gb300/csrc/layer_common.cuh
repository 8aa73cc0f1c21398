// What the tensor-memory products of the layer with experts and of the fp8 layers share: waits, a CTA's share of the work and
// the flags of sums that cross CTAs.
#pragma once

#include "awq_internal.h"
#include "awq_ptx.cuh"

namespace awq {
namespace {

// Waits for this thread's tensor memory loads; `r` is not used before.
__device__ __forceinline__ void wait_loaded(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// The first look comes before the clock is read for the limit.
__device__ __forceinline__ bool wait_for(uint32_t bar, uint32_t parity, volatile int* abort, int* err, int id) {
  return mbar_try(bar, parity) || wait_bounded_inline(bar, parity, abort, err, id);
}

// Arrives on `bar` once the products issued before have completed; executed by the whole warp, issued by the lane that
// elect.sync chooses (always the same, which issued the products).
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xFFFFFFFF;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar)
      : "memory");
}
constexpr int kMinUnits = 4;  // groups that a CTA gets at least of what is cut along K

// What a CTA works on, in order: parts of tiles, groups g0 .. g1 - 1 of each.  Counts stay within 32 bits: fewer than 2 grid
// tiles are cut along K, each of at most 8192 groups.
struct Walk {
  int grid, me, groups, rounds;  // whole rounds of tiles; what is left is cut
  int round, u, u1;
  int ctas, share, longer;  // CTAs that have some of it: `share` groups each, the first `longer` of them one more
  __device__ __forceinline__ Walk(int total, int groups_) : grid(gridDim.x), me(blockIdx.x), groups(groups_) {
    rounds = total / grid;
    int tiles = total - rounds * grid;
    if (tiles > 0 && rounds > 0) {
      --rounds;
      tiles += grid;
    }
    const int units = tiles * groups;
    ctas = max(1, min(grid, units / kMinUnits));
    share = units / ctas;
    longer = units - share * ctas;
    round = 0;
    u = me < ctas ? begin_of(me) : 0;
    u1 = me < ctas ? begin_of(me + 1) : 0;
  }
  __device__ __forceinline__ int begin_of(int cta) const { return cta * share + min(cta, longer); }
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

// Sums that cross CTAs: each summing warp has a flag of its own, as what it adds up was written by the same warp of the other CTA; so
// the warps of a CTA do not wait for one another (one flag for all, with barriers between them: 1.5 us more a product of one
// token's rows, 2.7 more of 192 rows).
//
// This warp's part, which all its lanes have written, may be read.
__device__ __forceinline__ void raise_flag(int* flag, int lane) {
  __syncwarp();
  if (lane == 0) asm volatile("st.release.gpu.global.b32 [%0], %1;" ::"l"(flag), "r"(1) : "memory");
}
// The calling warp's lanes wait for the flags of CTAs [from, to), `stride` apart, all at once.
__device__ __forceinline__ bool wait_flags(const int* flags, int stride, int from, int to, int lane, volatile int* abort, int* err,
                                           int id) {
  bool seen = true;
  for (int q = from + lane; q < to && seen; q += 32) {
    const long long t0 = now_ns();
    for (uint32_t spin = 1;; ++spin) {
      int v;
      asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(flags + (size_t)q * stride) : "memory");
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
  __syncwarp();  // what one lane has seen, the others may read
  return seen;
}

}  // namespace
}  // namespace awq
