// The grouped product for experts with few rows: bound by the weights' bytes.
//
// The same sums as moe_gemm.cu's: codes q - z as exact 16-bit operands, each group's sum scaled and added in fp32.  Here the
// products are mma.sync m16n8k16 with the weights as A (16 columns x 16 k) straight from registers and 8 rows of x as B:
// nothing is handed from one warp to another.  (On the tensor memory kernel with tiles of 16 rows a group took 1180
// cycles, which went to the barriers between its roles and to idle warps that polled them; the bytes take 725.)
//
// A CTA works on tiles of 256 columns x up to 16 rows of one expert.  A warp copies: for each group one unit of weights and the
// rows' 256 bytes each into a ring.  Eight warps have 16 columns of each half, gate and up of a gated layer in one thread.  Lane
// (g, t) holds columns g and g + 8 and, of a group's 128 rows of weights, the 32 of chunk t: 16 bytes of each column in the
// prepared copy.  The order of k within a product is free as long as both operands agree, so product i takes codes 4 i ..
// 4 i + 3 of every lane's chunk, and the lane's B is x[row g][32 t + 4 i ..], 64 bytes in one piece for a group.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "awq_host.h"
#include "moe_gemm.cuh"

namespace awq {
namespace {

constexpr int kWarps = 8, kThreads = (kWarps + 1) * 32, kSumThreads = kWarps * 32;
constexpr int kRows = kMoeGemvRows;
// A stage: unit | rows of x, 288 bytes apart (with words in the layout's places no two lanes' reads meet in a bank).
constexpr int kXAt = kMoeUnitBytes, kXStride = 288, kStageBytes = (kXAt + kRows * kXStride + 127) / 128 * 128, kStages = 9;
constexpr int kSmem = kStages * kStageBytes + 128;
static_assert(kSmem <= 227 * 1024 - 8192, "shared memory");

template <bool BF16>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <bool BF16, bool GATED, bool WIDE>
__global__ void __launch_bounds__(kThreads, 1)
moe_gemv_kernel(const MoeGemmArgs a, int* flags, float* parts, int* err) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ int first[kMoeMaxExperts + 1], items[kMoeMaxExperts + 1];
  __shared__ uint64_t full[kStages], empty[kStages], join_bar;
  __shared__ int abort_word, s_ok;
  volatile int* abort_flag = &abort_word;
  uint8_t* smem = smem_raw + ((128u - (smem_u32(smem_raw) & 127u)) & 127u);
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int groups = (int)(a.K / 128), pairs = a.tiles;
  if (tid == 32) {
    abort_word = 0;
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&full[i]), 1);
      mbar_init(smem_u32(&empty[i]), kWarps);
    }
    mbar_init(smem_u32(&join_bar), kWarps);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 0) expert_tables<kRows>(a, lane, first, items);
  __syncthreads();
  Walk walk(items[a.experts] * pairs, groups);
  int tile, g0, g1, st = 0;
  bool ok = true;

  if (warp == kWarps) {
    // ------------------------------------------------ copies: lane 0 the unit, lane r row r
    uint32_t phase = 1;
    int issued = 0;
    while (ok && walk.next(tile, g0, g1)) {
      const Tile t = find_tile<kRows>(first, items, a.experts, pairs, tile);
      const uint8_t* unit = a.packed + ((int64_t)t.expert * pairs + t.pair) * groups * kMoeUnitBytes;
      const uint16_t* row = a.x + source_row(a, t.row + min(lane, t.rows - 1)) * a.x_stride;
      for (int g = g0; g < g1; ++g) {
        ok = __all_sync(0xFFFFFFFFu, mbar_try(smem_u32(&empty[st]), phase) ||
                                         wait_bounded_slow(smem_u32(&empty[st]), phase, abort_flag, err, 752));
        if (!ok) break;
        const uint32_t to = smem_u32(smem + st * kStageBytes), bar = smem_u32(&full[st]);
        if (lane == 0) {
          mbar_arrive_tx(bar, (uint32_t)(kMoeUnitBytes + t.rows * 256));
          bulk_load(to, unit + (int64_t)g * kMoeUnitBytes, kMoeUnitBytes, bar);
        }
        __syncwarp();
        if (lane < t.rows) bulk_load(to + kXAt + lane * kXStride, row + g * 128, 256, bar);
        ++issued;
        if (++st == kStages) {
          st = 0;
          phase ^= 1u;
        }
      }
    }
    // never leave the CTA with copies in flight
    volatile int no_abort = 0;
    for (int j = max(0, issued - kStages); j < issued; ++j)
      wait_bounded(smem_u32(&full[j % kStages]), (uint32_t)(j / kStages) & 1u, &no_abort, err, 753);
  } else {
    const int g8 = lane / 4, t4 = lane % 4;
    uint32_t phase = 0, join_phase = 0;
    auto join = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&join_bar));
      const bool all = __all_sync(0xFFFFFFFFu, wait_bounded(smem_u32(&join_bar), join_phase, abort_flag, err, 754));
      join_phase ^= 1u;
      return all;
    };
    while (ok && walk.next(tile, g0, g1)) {
      const Tile t = find_tile<kRows>(first, items, a.experts, pairs, tile);
      const bool two = t.rows > 8;
      // rows beyond the tile's repeat its last one
      const int x0 = kXAt + min(g8, t.rows - 1) * kXStride + t4 * 64, x1 = kXAt + min(8 + g8, t.rows - 1) * kXStride + t4 * 64;
      float acc[2][2][4] = {};  // [half][rows 0..7, 8..15]
      for (int g = g0; g < g1; ++g) {
        ok = __all_sync(0xFFFFFFFFu, wait_bounded(smem_u32(&full[st]), phase, abort_flag, err, 755));
        if (!ok) break;
        const uint8_t* stage = smem + st * kStageBytes;
        uint4 w[2][2], xv[2][4];  // [half][column g, g + 8], [rows][piece]: word and piece i are moe_word_place(i, t)
        uint32_t zz[2][2];
        float s[2][2];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int c = 128 * b + 16 * warp + g8 + 8 * h;
            w[b][h] = *reinterpret_cast<const uint4*>(stage + moe_code_offset(c, t4));
            const uint32_t z = stage[kMoeZeroOffset + c / 2] >> (4 * (g8 & 1)) & 15u;
            zz[b][h] = fma16<BF16>(z | z << 16, BF16 ? 0xFE80FE80u : 0xF400F400u, 0u);
            s[b][h] = unpack2<BF16>(*reinterpret_cast<const uint16_t*>(stage + kMoeScaleOffset + 2 * c)).x *
                      (float)(1 << kDown<BF16>);
          }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = 16 * (i ^ (t4 >> 1));
          xv[0][i] = *reinterpret_cast<const uint4*>(stage + x0 + at);
          if (two) xv[1][i] = *reinterpret_cast<const uint4*>(stage + x1 + at);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&empty[st]));
        if (++st == kStages) {
          st = 0;
          phase ^= 1u;
        }
        float d[2][2][4] = {};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const uint32_t w0 = i == 0 ? w[b][0].x : i == 1 ? w[b][0].y : i == 2 ? w[b][0].z : w[b][0].w;
            const uint32_t w1 = i == 0 ? w[b][1].x : i == 1 ? w[b][1].y : i == 2 ? w[b][1].z : w[b][1].w;
            uint32_t o0[4], o1[4];
            operands<BF16>(w0, zz[b][0], o0, 0);
            operands<BF16>(w1, zz[b][1], o1, 0);
            mma16816<BF16>(d[b][0], o0[0], o1[0], o0[1], o1[1], xv[0][i].x, xv[0][i].y);
            mma16816<BF16>(d[b][0], o0[2], o1[2], o0[3], o1[3], xv[0][i].z, xv[0][i].w);
            if (two) {
              mma16816<BF16>(d[b][1], o0[0], o1[0], o0[1], o1[1], xv[1][i].x, xv[1][i].y);
              mma16816<BF16>(d[b][1], o0[2], o1[2], o0[3], o1[3], xv[1][i].z, xv[1][i].w);
            }
          }
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[b][n][i] = fmaf(d[b][n][i], s[b][i / 2], acc[b][n][i]);
      }
      if (!ok) break;
      if (g0 > 0) {
        // another CTA has the tile's first group: this one's sums go to it
        float4* part = reinterpret_cast<float4*>(parts + (size_t)walk.me * (kMoeGemvPartBytes / 4)) + tid;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int n = 0; n < 2; ++n)
            if (n == 0 || two)
              __stcg(part + (b * 2 + n) * kSumThreads, make_float4(acc[b][n][0], acc[b][n][1], acc[b][n][2], acc[b][n][3]));
        __threadfence();
        ok = join();
        if (ok && tid == 0) atomicExch(flags + walk.me, 1);
        continue;
      }
      if (g1 < groups) {
        // the others' sums, in the order of their groups
        const int end = (tile - walk.rounds * walk.grid + 1) * groups;
        int last = walk.me + 1;
        while (last < walk.ctas && walk.begin_of(last) < end) ++last;
        if (warp == 0) {
          const bool seen = wait_flags(flags, walk.me + 1, last, lane, abort_flag, err, 751);
          if (lane == 0) s_ok = seen;
        }
        ok = join() && s_ok != 0;
        if (!ok) break;
        for (int q = walk.me + 1; q < last; ++q) {
          const float4* part = reinterpret_cast<const float4*>(parts + (size_t)q * (kMoeGemvPartBytes / 4)) + tid;
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int n = 0; n < 2; ++n)
              if (n == 0 || two) {
                const float4 v = __ldcg(part + (b * 2 + n) * kSumThreads);
                acc[b][n][0] += v.x;
                acc[b][n][1] += v.y;
                acc[b][n][2] += v.z;
                acc[b][n][3] += v.w;
              }
        }
        ok = join();
        if (!ok) break;
        if (warp == 0)
          for (int q = walk.me + 1 + lane; q < last; q += 32) atomicExch(flags + q, 0);
      }
      using Out = typename std::conditional<WIDE, float, uint16_t>::type;
      const int64_t outs = GATED ? a.N / 2 : a.N;
#pragma unroll
      for (int b = 0; b < (GATED ? 1 : 2); ++b)
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = 8 * n + 2 * t4 + i % 2;
            const int64_t col = (int64_t)t.pair * (GATED ? 128 : 256) + 128 * b + 16 * warp + g8 + i / 2 * 8;
            if (row < t.rows && col < outs) {
              const float v = GATED ? silu_times(acc[0][n][i], acc[1][n][i]) : acc[b][n][i];
              Out* p = static_cast<Out*>(a.y) + (int64_t)(t.row + row) * outs + col;
              if constexpr (WIDE) *p = v;
              else *p = (uint16_t)pack2<BF16>(v, 0.f);
            }
          }
    }
  }
}

}  // namespace

cudaError_t launch_moe_gemv(const MoeGemmArgs& a, bool gated, bool wide, bool bf16, int* flags, float* parts, int* err,
                            cudaStream_t s) {
  const auto fn = bf16 ? (gated ? (wide ? moe_gemv_kernel<true, true, true> : moe_gemv_kernel<true, true, false>)
                                : (wide ? moe_gemv_kernel<true, false, true> : moe_gemv_kernel<true, false, false>))
                       : (gated ? (wide ? moe_gemv_kernel<false, true, true> : moe_gemv_kernel<false, true, false>)
                                : (wide ? moe_gemv_kernel<false, false, true> : moe_gemv_kernel<false, false, false>));
  const cudaError_t e = set_smem_once(reinterpret_cast<const void*>(fn), kSmem);
  if (e != cudaSuccess) return e;
  fn<<<device_sm_count(), kThreads, kSmem, s>>>(a, flags, parts, err);
  return cudaGetLastError();
}

}  // namespace awq
