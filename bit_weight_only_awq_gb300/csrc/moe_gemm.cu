// Products grouped by expert on prepared 4-bit weights (layout: include/awq.h), on the 5th-generation tensor cores.
//
// y[r, n] = sum_g s[g, n] sum_{k in g} x[src(r), k] (q[k, n] - z[g, n]) over an expert's rows; gated: silu(gate) * up.
// The weights enter the products as the integers q - z, exact in fp16 and bf16; each group of 128 rows has a sum of its
// own in tensor memory, which is scaled and added to the running sum in fp32 registers, where a column's scale is one
// register of its lane.  So no weight is rounded, and a code costs one operation less than with its scale on it.
//
// A CTA works on tiles of 256 columns x up to BT rows of one expert:
//   D[column][row] = A B,  A = weights, in tensor memory (128 columns x 64 k at once), B = rows of x, K-major in shared
//   memory.  Weights in shared memory would cost it 192 bytes a cycle at the full rate of the products; so it moves
//   64 (the operand B) and what the copies bring.
// Roles: the first warps add the groups' sums up and write results (a thread has one column of each half and some rows: gate and
// up of a gated layer meet in it), eight warps turn codes into operands (a thread has a column), then come those that issue the
// products, one that copies weights (one 17 KB unit a group) and one that copies rows of x.
// Sums and operands in tensor memory go round, so that the products need not wait for either.  A step of the products is a half
// of a group in tiles of 128 rows, each half's issued by a warp of its own (one warp for both took 6 % longer for 8192 rows over
// 8 experts), and a whole group in smaller ones, by one warp (two took 13 and 7 % longer for up and down of 192 rows); whoever
// waits for its products waits on one barrier.
// Rows of x come in any order.  Up to 16 of them are copied four an instruction (tile::gather4, about 30 cycles each); more,
// 32 KB a group with 128, are put in order first and copied in boxes of neighbouring rows (at 32008 rows over 126 experts an
// earlier form took 484 us with four rows an instruction, 406 with 16 bytes a thread, 273 without any copies).
//
// Tiles are dealt out to a persistent grid in whole rounds; what is left over is cut evenly along K, and a tile that several
// CTAs share is finished by the one that has its first group, which adds the others' sums in their order.
//
// Measured in graphs, inputs out of L2 (gate and up, then down): 8192 rows over 8 experts, 4096 x 2 x 14336 and back, 1410 and
// 720 us, 1365 and 1335 TFLOP/s: a group takes 1770 cycles of which the products are 1024; the rest are hand-overs between the roles
// and, in the first, the epilogue (37 us).  2 rows of one token: 34 and 21 us, 3.6 TB/s, at 1050 cycles a group: issue slots 54 %
// busy, operands 315 cycles, the rest their hand-over (750 a group with no work but theirs) and the 7 us of start and joins.  192 rows
// over 8 experts: 129 and 75 us, 3.8 TB/s.  32008 rows over 126 experts, 2048 x 2 x 768: 230 and 144 us, of which 27 put rows in order
// and 12 and 31 are the epilogue.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "awq_host.h"
#include "awq_internal.h"
#include "awq_ptx.cuh"
#include "awq_types.cuh"
#include "layer_common.cuh"

namespace awq {
namespace {

constexpr int kScaleSlots = 8;  // groups whose scales are kept, see below
constexpr int kRing = 4;        // groups whose products' barriers and rows are kept
constexpr int kBoxRows = 32;    // rows of a box of x

// Tiles of up to BT rows.
template <int BT>
struct Geo {
  static constexpr int kSteps = BT == 128 ? 2 : 1;       // steps of a group, each of 2 / kSteps halves
  static constexpr int kSumCols = BT * 2 / kSteps;       // columns of a step's sums
  static constexpr int kSums = BT == 16 ? 4 : BT == 64 ? 2 : 1;  // groups whose sums are kept in tensor memory
  static constexpr int kACol = kSums * kSteps * kSumCols;  // operands come behind them: [half][buffer] of 64 columns (128 k)
  static constexpr int kABufs = BT == 16 ? 3 : 2;        // groups whose operands are kept
  static constexpr int kXBytes = BT * 256;               // a group's rows: two blocks of 64 k, 128 bytes a row, swizzled
  static constexpr bool kBoxes = BT > 16;                // rows in order, copied in boxes; else four rows in any order at once
  static constexpr int kQStages = BT == 128 ? 5 : BT == 64 ? 8 : 10;
  // warps that add up, then eight that make operands, then products and copies
  static constexpr int kSumWarps = BT == 16 ? 4 : 8;
  static constexpr int kCodeWarp = kSumWarps, kMmaWarp = kCodeWarp + 8;
  static constexpr int kSumThreads = kSumWarps * 32, kThreads = (kMmaWarp + 4) * 32;
  // registers of a thread: at launch, then by role
  static constexpr int kLaunchRegs = BT == 16 ? 128 : 96, kSumRegs = BT == 16 ? 128 : BT == 64 ? 128 : 176,
                       kCodeRegs = BT == 16 ? 128 : BT == 64 ? 72 : 48, kOtherRegs = BT == 16 ? 128 : BT == 64 ? 72 : 32;
  static_assert(kSumThreads * kSumRegs + 256 * kCodeRegs + 128 * kOtherRegs <= kThreads * kLaunchRegs &&
                kThreads * kLaunchRegs <= 65536, "no more than was launched with");
  // shared memory: rows of x | units | scales | expert tables
  static constexpr int kQAt = kRing * kXBytes, kScaleAt = kQAt + kQStages * kMoeUnitBytes;
  static constexpr int kTableAt = kScaleAt + kScaleSlots * 256 * 4;
  static constexpr int kSmem = kTableAt + 2 * (kMoeMaxExperts + 1) * 4 + 1024;
  static constexpr int kRows = BT / (kSumWarps / 4), kPairs = kRows / 2;  // rows of a summing thread, and pairs of them, in each half
  static constexpr int kAtOnce = BT == 64 ? 2 : 1;       // loads of 16 columns of sums at once
  // a CTA's part of a shared tile: a sum for each of a summing thread's columns and rows
  static constexpr size_t kPartBytes = (size_t)256 * BT * 4;
  static_assert(kACol + 2 * kABufs * 64 <= 512 && kSmem <= 227 * 1024 - 1024, "tensor memory, shared memory");
  static_assert(kABufs <= kRing && kSums <= kRing, "barriers of products");
  static_assert(kBoxes || kSteps == 1, "rows copied four at a time wait for one step's products");
  static_assert(kScaleSlots >= kABufs + kSums + 1, "scales");
};

template <int BT>
struct Bars {
  uint64_t x_full[kRing], q_full[Geo<BT>::kQStages], q_empty[Geo<BT>::kQStages],
      a_full[Geo<BT>::kABufs][Geo<BT>::kSteps], done[kRing][Geo<BT>::kSteps], d_empty[Geo<BT>::kSums][Geo<BT>::kSteps], end;
};

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
// The products of one half and group, 128 k in steps of 16, into a fresh sum.  A in tensor memory: a lane for each column
// of the weights, two k a column of it; B: two blocks of 64 k.  Executed by the whole warp with uniform operands, issued by
// the lane that elect.sync chooses (always the same); one choice for all eight, which with one each took 60 cycles a product.
__device__ __forceinline__ void mma_group(uint32_t d, uint32_t a, uint64_t b0, uint64_t b1, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred q, no, yes;\n .reg .b32 a1, a2, a3, a4, a5, a6, a7;\n .reg .b64 b01, b02, b03, b11, b12, b13;\n"
      " setp.ne.b32 no, 0, 0;\n setp.eq.b32 yes, 0, 0;\n"
      " add.u32 a1, %1, 8;\n add.u32 a2, %1, 16;\n add.u32 a3, %1, 24;\n add.u32 a4, %1, 32;\n add.u32 a5, %1, 40;\n"
      " add.u32 a6, %1, 48;\n add.u32 a7, %1, 56;\n"
      " add.u64 b01, %2, 2;\n add.u64 b02, %2, 4;\n add.u64 b03, %2, 6;\n"
      " add.u64 b11, %3, 2;\n add.u64 b12, %3, 4;\n add.u64 b13, %3, 6;\n"
      " elect.sync _|q, 0xFFFFFFFF;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %4, no;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], b01, %4, yes;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], b02, %4, yes;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b03, %4, yes;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [a4], %3, %4, yes;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [a5], b11, %4, yes;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [a6], b12, %4, yes;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [a7], b13, %4, yes;\n}\n" ::"r"(d),
      "r"(a), "l"(b0), "l"(b1), "r"(idesc)
      : "memory");
}
// Four rows, 64 k each, of a tensor map whose box is one row high.
__device__ __forceinline__ void gather4(uint32_t dst, const CUtensorMap* map, int col, const int (&r)[4], uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cta.global.tile::gather4.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, "
      "%6}], [%7];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(col), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(bar)
      : "memory");
}

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

// silu(gate) up from e = exp(-|gate|), which neither overflows nor makes the divisor leave [1, 2], so that gates below -88 give
// their subnormal results too.  Results of 16 bits take the approximate exponential, off by 2 + 1.2 |gate| units in the last place of
// fp32 (expf: 16 us more of 1427 for 8192 rows of 14336 columns), fp32 ones the exact functions: 2.5 2^-22 of the value in all.
template <bool WIDE>
__device__ __forceinline__ float silu_times(float gate, float up) {
  const float e = WIDE ? expf(-fabsf(gate)) : __expf(-fabsf(gate));
  const float top = gate < 0.f ? gate * e : gate;
  return (WIDE ? __fdiv_rn(top, 1.f + e) : __fdividef(top, 1.f + e)) * up;
}

template <int BT, bool BF16, bool GATED, bool WIDE>
__global__ void __launch_bounds__(Geo<BT>::kThreads, 1)
moe_gemm_kernel(const __grid_constant__ CUtensorMap tm_x, const MoeGemmArgs a, int* flags, float* parts, int* err) {
  using G = Geo<BT>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Bars<BT> bars;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;
  const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid / 32, 0), lane = tid % 32;
  uint8_t* smem = align_smem_1024(smem_raw);
  const uint32_t sm = smem_u32(smem);
  int* first = reinterpret_cast<int*>(smem + G::kTableAt);
  int* items = first + kMoeMaxExperts + 1;
  const int groups = (int)(a.K / 128);

  if (tid == 32) {
    abort_word = 0;
    for (int i = 0; i < kRing; ++i) {
      mbar_init(smem_u32(&bars.x_full[i]), 1);
      for (int h = 0; h < G::kSteps; ++h) mbar_init(smem_u32(&bars.done[i][h]), 1);
    }
    for (int i = 0; i < G::kQStages; ++i) {
      mbar_init(smem_u32(&bars.q_full[i]), 1);
      mbar_init(smem_u32(&bars.q_empty[i]), 8);
    }
    for (int i = 0; i < G::kABufs * G::kSteps; ++i) mbar_init(smem_u32(&bars.a_full[0][i]), 8 / G::kSteps);
    for (int i = 0; i < G::kSums * G::kSteps; ++i) mbar_init(smem_u32(&bars.d_empty[0][i]), G::kSumWarps);
    mbar_init(smem_u32(&bars.end), G::kSteps);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == G::kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (!a.early) wait_then_release_dependents();
  if (warp == 0) expert_tables<BT>(a, lane, first, items);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const int pairs = a.tiles;
  Walk walk(items[a.experts] * pairs, groups);
  int tile, g0, g1;
  bool ok = true;

  if (warp < G::kSumWarps) {
    if constexpr (G::kSumRegs > G::kLaunchRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(G::kSumRegs));
    // ------------------------------------------------ running sums: column n of each half, rows kRows wg ..
    const int wg = warp / 4, n = warp % 4 * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(warp % 4 * 32) << 16) + G::kRows * wg;
    const float* scales = reinterpret_cast<const float*>(smem + G::kScaleAt);
    int d = 0, count = 0;  // count: groups so far, of this CTA
    if (a.early) wait_then_release_dependents();
    auto take = [&](int step) {  // a sum is in registers
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&bars.d_empty[d][step]));
    };
    while (ok && walk.next(tile, g0, g1)) {
      const Tile t = find_tile<BT>(first, items, a.experts, pairs, tile);
      const int mine = min(max(t.rows - G::kRows * wg, 0), G::kRows);  // of this thread's rows
      F2 acc[2][G::kPairs];
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int i = 0; i < G::kPairs; ++i) acc[b][i] = F2(0.f, 0.f);
      for (int g = g0; g < g1 && ok; ++g, ++count) {
#pragma unroll
        for (int step = 0; step < G::kSteps; ++step) {
          ok = __all_sync(0xFFFFFFFFu, wait_for(smem_u32(&bars.done[count % kRing][step]), (uint32_t)(count / kRing) & 1u,
                                                abort_flag, err, 702));
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int bb = 0; bb < 2 / G::kSteps; ++bb) {
            const int b = G::kSteps == 2 ? step : bb;
            const float s = scales[count % kScaleSlots * 256 + b * 128 + n];
            const F2 s2(s, s);
            const uint32_t from = lanes + (d * G::kSteps + step) * G::kSumCols + bb * BT;
#pragma unroll
            for (int c = 0; c < G::kRows / 16; c += G::kAtOnce) {
              uint32_t v[G::kAtOnce][16];
              const bool any = 16 * c < mine;
              if (any) {
#pragma unroll
                for (int h = 0; h < G::kAtOnce; ++h) tmem_ld16_nowait(from + 16 * (c + h), v[h]);
#pragma unroll
                for (int h = 0; h < G::kAtOnce; ++h) wait_loaded(v[h]);
              }
              if (bb == 2 / G::kSteps - 1 && c + G::kAtOnce == G::kRows / 16) take(step);
              if (any) {
#pragma unroll
                for (int h = 0; h < G::kAtOnce; ++h)
#pragma unroll
                  for (int i = 0; i < 8; ++i) {
                    F2& to = acc[b][8 * (c + h) + i];
                    to = fma2(F2(__uint_as_float(v[h][2 * i]), __uint_as_float(v[h][2 * i + 1])), s2, to);
                  }
              }
            }
          }
        }
        if (++d == G::kSums) d = 0;
      }
      if (!ok) break;
      if (g0 > 0) {
        // another CTA has the tile's first group: this one's sums go to it
        F2* part = reinterpret_cast<F2*>(parts) + (size_t)walk.me * (G::kPartBytes / 8) + tid;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int i = 0; i < G::kPairs; ++i)
            if (2 * i < mine) __stcg(reinterpret_cast<unsigned long long*>(part + (b * G::kPairs + i) * G::kSumThreads), acc[b][i].v);
        raise_flag(flags + walk.me * G::kSumWarps + warp, lane);
        continue;
      }
      if (g1 < groups) {
        // the others' sums, in the order of their groups; a warp's lanes wait for all of them at once
        const int end = (tile - walk.rounds * walk.grid + 1) * groups;
        int last = walk.me + 1;
        while (last < walk.ctas && walk.begin_of(last) < end) ++last;
        ok = wait_flags(flags + warp, G::kSumWarps, walk.me + 1, last, lane, abort_flag, err, 703);
        if (!ok) break;
        for (int q = walk.me + 1; q < last; ++q) {
          const F2* part = reinterpret_cast<const F2*>(parts) + (size_t)q * (G::kPartBytes / 8) + tid;
#pragma unroll
          for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int i = 0; i < G::kPairs; ++i)
              if (2 * i < mine) {
                F2 o;
                o.v = __ldcg(reinterpret_cast<const unsigned long long*>(part + (b * G::kPairs + i) * G::kSumThreads));
                acc[b][i] = add2(acc[b][i], o);
              }
        }
        __syncwarp();
        for (int q = walk.me + 1 + lane; q < last; q += 32) flags[q * G::kSumWarps + warp] = 0;
      }
      // Two neighbouring lanes swap one of a pair of rows each, so that a lane writes two columns of one row.  Whether a column
      // exists is the same for all lanes: there are multiples of 32.
      const int64_t outs = GATED ? a.N / 2 : a.N;
      const bool odd = lane & 1;
      using Out = typename std::conditional<WIDE, float2, uint32_t>::type;
#pragma unroll
      for (int b = 0; b < (GATED ? 1 : 2); ++b) {
        const int64_t col = GATED ? (int64_t)t.pair * 128 + n : (int64_t)t.pair * 256 + b * 128 + n;
        Out* p = static_cast<Out*>(a.y) + ((int64_t)(t.row + G::kRows * wg + odd) * outs + col - odd) / 2;
        const int rows = col < outs ? mine : 0;
#pragma unroll
        for (int c = 0; c < G::kPairs; c += 4) {
          if (2 * c >= rows) break;
          // eight rows at once, those beyond the tile's among them: one after another, each waits for its exponential
          float2 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            v[i] = acc[b][c + i].get();
            if constexpr (GATED) {
              const float2 u = acc[1][c + i].get();
              v[i] = make_float2(silu_times<WIDE>(v[i].x, u.x), silu_times<WIDE>(v[i].y, u.y));
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            Out w;
            if constexpr (WIDE) {
              const float got = __shfl_xor_sync(0xFFFFFFFFu, odd ? v[i].x : v[i].y, 1);
              w = odd ? make_float2(got, v[i].y) : make_float2(v[i].x, got);
            } else {
              const uint32_t own = pack2<BF16>(v[i].x, v[i].y), got = __shfl_xor_sync(0xFFFFFFFFu, own, 1);
              w = __byte_perm(own, got, odd ? 0x3276 : 0x5410);
            }
            if (2 * (c + i) + odd < rows) *p = w;
            p += outs;
            asm volatile("" : "+l"(p));  // one address at a time, not all made ahead
          }
        }
      }
    }
  } else if (warp < G::kMmaWarp) {
    if constexpr (G::kCodeRegs < G::kLaunchRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(G::kCodeRegs));
    // ------------------------------------------------ operands: column n of half b
    const int b = (warp - G::kCodeWarp) / 4, n = warp % 4 * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(warp % 4 * 32) << 16) + G::kACol + 64 * G::kABufs * b;
    const int step = G::kSteps == 2 ? b : 0, c = b * 128 + n;
    int q = 0, buf = 0, count = 0;
    uint32_t q_phase = 0, z = 0u;
    uint16_t raw = 0;
    uint4 w;
    bool have = false;  // the first codes of the next group are in registers
    auto start = [&]() {
      const uint8_t* unit = smem + G::kQAt + q * kMoeUnitBytes;
      w = lds128(sm + G::kQAt + q * kMoeUnitBytes + moe_code_offset(c, 0));
      z = unit[kMoeZeroOffset + c / 2];
      raw = *reinterpret_cast<const uint16_t*>(unit + kMoeScaleOffset + 2 * c);
    };
    while (ok && walk.next(tile, g0, g1)) {
      for (int g = g0; g < g1; ++g, ++count) {
        if (!have) {
          ok = __all_sync(0xFFFFFFFFu, wait_for(smem_u32(&bars.q_full[q]), q_phase, abort_flag, err, 711));
          if (!ok) break;
          start();
        }
        const uint32_t codes = sm + G::kQAt + q * kMoeUnitBytes;
        const uint32_t zn = z >> (4 * (c & 1)) & 15u;
        const uint32_t zz = fma16<BF16>(zn | zn << 16, BF16 ? 0xFE80FE80u : 0xF400F400u, 0u);  // -z 2^-kDown
        const float scale = unpack2<BF16>(raw).x * (float)(1 << kDown<BF16>);
#pragma unroll
        for (int chunk = 0; chunk < 4; ++chunk) {
          uint32_t o[16];
          operands<BF16>(w.x, zz, o, 4 * moe_word_place(0, chunk));
          operands<BF16>(w.y, zz, o, 4 * moe_word_place(1, chunk));
          operands<BF16>(w.z, zz, o, 4 * moe_word_place(2, chunk));
          operands<BF16>(w.w, zz, o, 4 * moe_word_place(3, chunk));
          if (chunk < 3) w = lds128(codes + moe_code_offset(c, chunk + 1));
          if (chunk == 0 && count >= G::kABufs) {
            // the products that read this buffer last
            const int last = count - G::kABufs;
            ok = __all_sync(0xFFFFFFFFu, wait_for(smem_u32(&bars.done[last % kRing][step]), (uint32_t)(last / kRing) & 1u,
                                                  abort_flag, err, 712));
            if (!ok) break;
            tc_fence_after();
          }
          tmem_st16(lanes + 64 * buf + 16 * chunk, o);
        }
        if (!ok) break;
        // Scales for the sums.  A slot is written again 8 groups later: the products of kABufs groups back are done, which
        // waited until the sums of the steps kSums before them had been taken out, their scales read.
        reinterpret_cast<float*>(smem + G::kScaleAt)[count % kScaleSlots * 256 + c] = scale;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars.q_empty[q]));  // all codes are in registers
        if (++q == G::kQStages) {
          q = 0;
          q_phase ^= 1u;
        }
        // the next group's first codes, if they are there, while the stores arrive
        have = g + 1 < g1 && __all_sync(0xFFFFFFFFu, mbar_try(smem_u32(&bars.q_full[q]), q_phase));
        if (have) start();
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars.a_full[buf][step]));
        if (++buf == G::kABufs) buf = 0;
      }
    }
  } else {
    if constexpr (G::kOtherRegs < G::kLaunchRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(G::kOtherRegs));
    if (warp < G::kMmaWarp + G::kSteps) {
      // ------------------------------------------------ products of a step; each step's warp has sums of its own
      const int step = warp - G::kMmaWarp;
      const uint64_t bdesc0 = smem_desc_sw128(sm, 16, 1024);
      int d = 0, buf = 0, count = 0;
      uint32_t d_phase = 1, a_phase = 0;
      while (ok && walk.next(tile, g0, g1)) {
        const Tile t = find_tile<BT>(first, items, a.experts, pairs, tile);
        const uint32_t idesc = (1u << 4) | (BF16 ? (1u << 7) | (1u << 10) : 0u) | ((uint32_t)((t.rows + 15) / 16 * 2) << 17) |
                               (8u << 24);
#pragma unroll 1
        for (int g = g0; g < g1; ++g, ++count) {
          const int x = count % kRing;
          ok = wait_for(smem_u32(&bars.x_full[x]), (uint32_t)(count / kRing) & 1u, abort_flag, err, 721);
          ok = __all_sync(0xFFFFFFFFu, ok && wait_for(smem_u32(&bars.d_empty[d][step]), d_phase, abort_flag, err, 722) &&
                                           wait_for(smem_u32(&bars.a_full[buf][step]), a_phase, abort_flag, err, 723));
          if (!ok) break;
          tc_fence_after();
          const uint64_t bd = bdesc0 + (uint64_t)((x * G::kXBytes) >> 4);
#pragma unroll
          for (int bb = 0; bb < 2 / G::kSteps; ++bb)
            mma_group(tmem + (d * G::kSteps + step) * G::kSumCols + bb * BT, tmem + G::kACol + 64 * (G::kABufs * (step + bb) + buf), bd,
                      bd + (uint64_t)(G::kXBytes >> 5), idesc);
          commit(smem_u32(&bars.done[x][step]));
          if (++d == G::kSums) {
            d = 0;
            d_phase ^= 1u;
          }
          if (++buf == G::kABufs) {
            buf = 0;
            a_phase ^= 1u;
          }
        }
      }
      commit(smem_u32(&bars.end));  // arrives once every product of this warp has completed
      volatile int no_abort = 0;
      wait_for(smem_u32(&bars.end), 0, &no_abort, err, 724);
    } else if (warp == G::kMmaWarp + G::kSteps) {
      // ------------------------------------------------ copies of weights
      if (lane == 0) {
        int q = 0, issued = 0;
        uint32_t q_phase = 1;
        while (ok && walk.next(tile, g0, g1)) {
          const Tile t = find_tile<BT>(first, items, a.experts, pairs, tile);
          const uint8_t* src = a.packed + ((int64_t)t.expert * pairs + t.pair) * groups * kMoeUnitBytes;
          for (int g = g0; g < g1; ++g) {
            ok = wait_for(smem_u32(&bars.q_empty[q]), q_phase, abort_flag, err, 731);
            if (!ok) break;
            mbar_arrive_tx(smem_u32(&bars.q_full[q]), kMoeUnitBytes);
            bulk_load(sm + G::kQAt + q * kMoeUnitBytes, src + (int64_t)g * kMoeUnitBytes, kMoeUnitBytes, smem_u32(&bars.q_full[q]));
            ++issued;
            if (++q == G::kQStages) {
              q = 0;
              q_phase ^= 1u;
            }
          }
        }
        // never leave the CTA with copies in flight
        volatile int no_abort = 0;
        for (int j = max(0, issued - G::kQStages); j < issued; ++j)
          wait_for(smem_u32(&bars.q_full[j % G::kQStages]), (uint32_t)(j / G::kQStages) & 1u, &no_abort, err, 732);
      }
    } else if constexpr (G::kBoxes) {
      // ------------------------------------------------ copies of rows, boxes of 32 rows x 64 k
      if (warp == G::kMmaWarp + G::kSteps + 1 && lane == 0) {
        if (a.early) asm volatile("griddepcontrol.wait;" ::: "memory");
        int count = 0;
        while (ok && walk.next(tile, g0, g1)) {
          const Tile t = find_tile<BT>(first, items, a.experts, pairs, tile);
          const int boxes = (t.rows + kBoxRows - 1) / kBoxRows;
          for (int g = g0; g < g1; ++g, ++count) {
            const int x = count % kRing;
            if (count >= kRing) {
              for (int h = 0; h < G::kSteps && ok; ++h)
                ok = wait_for(smem_u32(&bars.done[x][h]), (uint32_t)(count / kRing - 1) & 1u, abort_flag, err, 743);
              if (!ok) break;
            }
            const uint32_t bar = smem_u32(&bars.x_full[x]);
            mbar_arrive_tx(bar, (uint32_t)(boxes * kBoxRows * 256));
            for (int i = 0; i < boxes; ++i) {
              const uint32_t dst = sm + x * G::kXBytes + i * (kBoxRows * 128);
              tma_load_2d(dst, &tm_x, g * 128, t.row + i * kBoxRows, bar);
              tma_load_2d(dst + G::kXBytes / 2, &tm_x, g * 128 + 64, t.row + i * kBoxRows, bar);
            }
          }
        }
        volatile int no_abort = 0;
        for (int j = max(0, count - kRing); j < count; ++j)
          wait_for(smem_u32(&bars.x_full[j % kRing]), (uint32_t)(j / kRing) & 1u, &no_abort, err, 744);
      }
    } else if (warp == G::kMmaWarp + G::kSteps + 1) {
      // ------------------------------------------------ copies of rows: lane l has rows 4 l .. 4 l + 3
      int count = 0;
      if (a.early) asm volatile("griddepcontrol.wait;" ::: "memory");
      while (ok && walk.next(tile, g0, g1)) {
        const Tile t = find_tile<BT>(first, items, a.experts, pairs, tile);
        int r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = source_row(a, t.row + min(4 * lane + i, t.rows - 1));
        const int fours = (t.rows + 3) / 4;
        for (int g = g0; g < g1; ++g, ++count) {
          const int x = count % kRing;
          if (count >= kRing) {
            ok = __all_sync(0xFFFFFFFFu, wait_for(smem_u32(&bars.done[x][0]), (uint32_t)(count / kRing - 1) & 1u, abort_flag, err,
                                                  741));
            if (!ok) break;
          }
          const uint32_t bar = smem_u32(&bars.x_full[x]), dst = sm + x * G::kXBytes + lane * 512;
          if (lane == 0) mbar_arrive_tx(bar, (uint32_t)fours * 1024u);
          __syncwarp();
          if (lane < fours) {
            gather4(dst, &tm_x, g * 128, r, bar);
            gather4(dst + G::kXBytes / 2, &tm_x, g * 128 + 64, r, bar);
          }
        }
      }
      volatile int no_abort = 0;
      for (int j = max(0, count - kRing); j < count; ++j)
        wait_for(smem_u32(&bars.x_full[j % kRing]), (uint32_t)(j / kRing) & 1u, &no_abort, err, 742);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == G::kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

// Rows of x in the plan's order, a warp for each (32008 x 2048: 35 us with a thread for 16 bytes, each
// looking its row up, 27 so, 131 MB of them written).
__global__ void __launch_bounds__(256) moe_order_kernel(const MoeGemmArgs a, uint16_t* out) {
  wait_then_release_dependents();
  const int vec = (int)(a.K / 8), rows = min(max(a.offsets[a.experts], 0), (int)a.R), lane = threadIdx.x % 32;
  for (int r = (int)(blockIdx.x * 8 + threadIdx.x / 32); r < rows; r += (int)gridDim.x * 8) {
    const uint4* from = reinterpret_cast<const uint4*>(a.x + source_row(a, r) * a.x_stride);
    uint4* to = reinterpret_cast<uint4*>(out + (int64_t)r * a.K);
    for (int i0 = 0; i0 < vec; i0 += 256) {
      uint4 v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i0 + 32 * j + lane < vec) v[j] = from[i0 + 32 * j + lane];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i0 + 32 * j + lane < vec) to[i0 + 32 * j + lane] = v[j];
    }
  }
}

// Rows of a tile: by the rows that an expert has on average, choices without an expert counted, as more is known on the device
// only; a hot expert among idle ones, or a rank that holds few of the experts, gets tiles that are small or large for it.  Tiles of 16, 64
// and 128 rows, us: 8 experts of 4096 x 2 x 14336, 8 rows of each 118, 121, 135; 12 rows 133, 123, 138; 60 rows 452, 189, 199; 128
// experts of 2048 x 2 x 768, 8 rows 60, 61, 67; 12 rows 71, 64, 73; 80 rows 270, 118, 120; 64 experts of 2048 x 2 x 1408, 100 rows 301,
// 121, 111.
int tile_rows(int64_t R, int experts) {
  const double mean = (double)R / experts;
  return R <= 16 || mean <= 8 ? 16 : mean <= 80 ? 64 : 128;
}
// Workspace: flags | parts of shared tiles | rows in order, where x holds tokens
size_t parts_bytes(int bt) { return align256((size_t)device_sm_count() * 256 * (size_t)bt * 4); }

template <int BT, bool BF16>
cudaError_t launch(MoeGemmArgs a, bool gated, bool wide, void* ws, int* err, cudaStream_t s) {
  using G = Geo<BT>;
  const auto fn = gated ? (wide ? moe_gemm_kernel<BT, BF16, true, true> : moe_gemm_kernel<BT, BF16, true, false>)
                        : (wide ? moe_gemm_kernel<BT, BF16, false, true> : moe_gemm_kernel<BT, BF16, false, false>);
  cudaError_t e = set_smem_once(reinterpret_cast<const void*>(fn), G::kSmem);
  if (e != cudaSuccess) return e;
  int* flags = static_cast<int*>(ws);
  float* parts = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kCounterBytes);
  if (G::kBoxes && a.order) {
    uint16_t* rows = reinterpret_cast<uint16_t*>(reinterpret_cast<uint8_t*>(parts) + parts_bytes(BT));
    e = launch_dependent(moe_order_kernel, dim3(device_sm_count() * 8), 256, 0, s, a, rows);
    if (e != cudaSuccess) return e;
    a.x = rows;
    a.x_rows = a.R;
    a.x_stride = a.K;
    a.order = nullptr;
  }
  CUtensorMap tm;
  if (!make_map_2d(&tm, BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, a.x, (uint64_t)a.K,
                   (uint64_t)a.x_rows, 64, G::kBoxes ? kBoxRows : 1, CU_TENSOR_MAP_SWIZZLE_128B, (uint64_t)a.x_stride))
    return cudaErrorInvalidValue;
  return launch_dependent(fn, dim3(device_sm_count()), G::kThreads, G::kSmem, s, tm, a, flags, parts, err);
}

}  // namespace

size_t moe_gemm_workspace(int64_t R, int experts, int64_t K, bool tokens) {
  const int bt = tile_rows(R, experts);
  return kCounterBytes + parts_bytes(bt) + (tokens && bt > 16 ? (size_t)R * (size_t)K * 2 : 0);
}

cudaError_t launch_moe_gemm(const MoeGemmArgs& a, bool gated, bool wide, bool bf16, void* ws, int* err, cudaStream_t s) {
  const int bt = tile_rows(a.R, a.experts);
  const auto fn = bt == 16   ? (bf16 ? launch<16, true> : launch<16, false>)
                  : bt == 64 ? (bf16 ? launch<64, true> : launch<64, false>)
                             : (bf16 ? launch<128, true> : launch<128, false>);
  return fn(a, gated, wide, ws, err, s);
}

}  // namespace awq
