// What the attention kernels over the 4-bit cache share: the call's arguments, a sequence's place in them.
#pragma once

#include "awq_internal.h"

namespace awq {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct Args : Kv4AttnArgs {
  int per;             // query heads of a cache head
  int rows;            // the sequences of this launch: at most so many query rows of a cache head, or more than that
  int units_page;      // units of a page
  uint32_t page_magic; // unit / units_page = high word of unit * page_magic (0: one unit a page)
};

inline Args make_args(const Kv4AttnArgs& args) {
  Args a;
  static_cast<Kv4AttnArgs&>(a) = args;
  a.per = args.heads / args.kv_heads;
  a.units_page = args.page_size / kKv4Unit;
  // exact for units below 2^32 / units_page >= 2^26: lengths are at most 2^30 tokens
  a.page_magic = a.units_page == 1 ? 0u : (uint32_t)(((1ull << 32) + a.units_page - 1) / a.units_page);
  return a;
}

// Query tokens and length of sequence b, as the device memory has them.
__device__ __forceinline__ int3 read_seq(const Args& a, int b) {
  int begin = b, n = 1;
  if (a.q_start) {
    begin = min(max(a.q_start[b], 0), (int)a.T);
    n = min(min(max(a.q_start[b + 1], begin), (int)a.T) - begin, a.max_q);
  }
  return make_int3(begin, n, min(max(a.kv_len[b], 0), a.max_pages * a.page_size));
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

}  // namespace
}  // namespace awq
