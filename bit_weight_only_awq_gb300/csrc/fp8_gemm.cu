// Product of e4m3 activations and weights with scales for blocks of 128, on the 5th-generation tensor cores.
//
// y[m, n] = sum_g s_x[g, m] s_w[n / 128, g] sum_{k in block g} xq[m, k] wq[n, k].
// Each block of 128 k has a sum of its own in tensor memory (fp32; its products are exact), which is multiplied by the
// two scales and added to the running sum in fp32 registers.
//
// Two forms of tcgen05.mma kind::f8f6f4, both operands K-major in shared memory:
//   few tokens, or so many that tiles of 64 suffice, D[output][token]: 128 outputs x up to 16 or 64 tokens; a column's factor s_x s_w is one of these numbers in
//     shared memory, the same for all lanes;
//   more tokens, D[token][output]: 128 tokens x 256 outputs; a lane has a token, whose factor is one register (the first form with
//     256 tokens spent its time on loading factors: 574 us against 460 for 4096 tokens through 4096 x 28672).
// Roles: the first warps add up and write results (a thread has a lane of D and some of its columns), then come a warp that issues
// the products, one that copies the operands (128 bytes of a row a block) and two that make the first form's factors, or for one or
// two tokens given in 16 bits the codes too: such a layer is one launch.  The persistent grid and sums that cross CTAs are
// those of the grouped product.
//
// Measured: 4096 tokens through 4096 x 28672 in 399 us, 2410 TFLOP/s.  A block's products take 517 cycles, the sums of its 128 x 256
// numbers by 16 warps about 570, its 48 KB of operands 768 at 64 bytes a cycle; all three at once 1020.  None of them alone is
// the limit: without the sums 362 us, without the copies 375, without the stores 378; without all three and the products 245,
// the barriers' round trips between the roles.  48 tokens through 14336 x 4096: 19 us, 3.2 TB/s, bound by those round trips too;
// one token through 4096 x 6144: 10.5 us, of which 3.7 are its bytes.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "awq_host.h"
#include "awq_internal.h"
#include "awq_ptx.cuh"
#include "fp8_common.cuh"
#include "layer_common.cuh"

namespace awq {
namespace {

constexpr int kLanes = 128, kABytes = kLanes * 128;  // lanes of D; bytes of a block of their operand

// BT: columns of D, tokens at 16 and 64, outputs at 256.
template <int BT>
struct Geo {
  static constexpr bool kTokenLanes = BT == 256;
  static constexpr int kBytes = kABytes + BT * 128;     // a stage: the lanes' operand | the columns'
  static constexpr int kStages = BT == 256 ? 4 : BT == 64 ? 8 : 11;
  static constexpr int kSums = BT == 256 ? 2 : 4;       // blocks whose sums are kept in tensor memory, BT columns each
  // A factor's slot is written again when the products kStages before it are done; those waited for the sums kSums
  // further back to be taken out, and the factors of the block before these had been read by then.
  static constexpr int kSlots = kStages + kSums + 1;
  static constexpr int kBoxRows = BT < 64 ? BT : 64;
  static constexpr int kSumWarps = BT == 16 ? 4 : 16, kMmaWarp = kSumWarps;
  static constexpr int kSumThreads = kSumWarps * 32, kThreads = (kMmaWarp + 4) * 32;
  // registers of a thread: at launch, then by role (256 columns: 64 sums)
  static constexpr int kLaunchRegs = BT == 16 ? 248 : 96, kSumRegs = BT == 16 ? 248 : BT == 64 ? 96 : 112,
                       kOtherRegs = BT == 16 ? 248 : BT == 64 ? 96 : 32;
  static_assert(kSumThreads * kSumRegs + 128 * kOtherRegs <= kThreads * kLaunchRegs && kThreads * kLaunchRegs <= 65536,
                "no more than was launched with");
  static constexpr int kRows = BT / (kSumWarps / 4), kPairs = kRows / 2;  // columns of a summing thread, and pairs of them
  // behind the stages: factors, or for token lanes 2 KB of each summing warp, through which rows of results leave
  static constexpr int kFactorAt = kStages * kBytes, kSmem = kFactorAt + (kTokenLanes ? kSumWarps * 2048 : kSlots * BT * 4) + 1024;
  static constexpr int kTmem = kSums * BT < 64 ? 64 : kSums * BT;
  static constexpr size_t kPartBytes = (size_t)kLanes * BT * 4;
  static_assert(kSmem <= 227 * 1024 - 1024 && kTmem <= 512, "shared memory, tensor memory");
};

template <int BT>
struct Bars {
  uint64_t full[Geo<BT>::kStages], done[Geo<BT>::kStages], d_empty[Geo<BT>::kSums], end;
};

// The products of one block, 128 k in steps of 32, into a fresh sum.
__device__ __forceinline__ void mma_block(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc) {
  asm volatile(
      "{\n .reg .pred q, no, yes;\n .reg .b64 a1, a2, a3, b1, b2, b3;\n"
      " setp.ne.b32 no, 0, 0;\n setp.eq.b32 yes, 0, 0;\n"
      " add.u64 a1, %1, 2;\n add.u64 a2, %1, 4;\n add.u64 a3, %1, 6;\n add.u64 b1, %2, 2;\n add.u64 b2, %2, 4;\n add.u64 b3, %2, 6;\n"
      " elect.sync _|q, 0xFFFFFFFF;\n"
      " @q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, no;\n"
      " @q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a1, b1, %3, yes;\n"
      " @q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a2, b2, %3, yes;\n"
      " @q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], a3, b3, %3, yes;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc)
      : "memory");
}

// Rows of the two operands that a tile has: `lane`.. (128 of them) and `col` .. col + cols - 1.
struct Tile {
  int lane, col, cols;
};
// Token tiles are neighbours; in the first form tokens even out over them.
template <int BT>
__device__ __forceinline__ Tile find_tile(int tile, int m_tiles, const Fp8GemmArgs& a) {
  const int n = tile / m_tiles, m = tile - n * m_tiles;
  if constexpr (Geo<BT>::kTokenLanes) return Tile{m * kLanes, n * BT, min(BT, (int)a.N - n * BT)};
  const int M = (int)a.M, share = ((M + m_tiles - 1) / m_tiles + 15) / 16 * 16;
  return Tile{n * kLanes, m * share, min(share, M - m * share)};
}

// QUANT: the activations are 16-bit, quantized here.
template <int BT, bool BF16, bool QUANT>
__global__ void __launch_bounds__(Geo<BT>::kThreads, 1)
fp8_gemm_kernel(const __grid_constant__ CUtensorMap tm_lanes, const __grid_constant__ CUtensorMap tm_cols, const Fp8GemmArgs a,
                int m_tiles, int tiles, int* flags, float* parts, int* err) {
  using G = Geo<BT>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Bars<BT> bars;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;
  const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid / 32, 0), lane = tid % 32;
  uint8_t* smem = align_smem_1024(smem_raw);
  const uint32_t sm = smem_u32(smem);
  const int blocks = (int)((a.K + 127) / 128), M = (int)a.M;

  if (tid == 0) {
    abort_word = 0;
    for (int i = 0; i < G::kStages; ++i) {
      mbar_init(smem_u32(&bars.full[i]), QUANT ? 3 : G::kTokenLanes ? 1 : 2);  // the copies and the factors
      mbar_init(smem_u32(&bars.done[i]), 1);
    }
    for (int i = 0; i < G::kSums; ++i) mbar_init(smem_u32(&bars.d_empty[i]), G::kSumWarps);
    mbar_init(smem_u32(&bars.end), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == G::kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)),
                 "r"((uint32_t)G::kTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  wait_then_release_dependents();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  Walk walk(tiles, blocks);
  int tile, g0, g1, count = 0;  // count: blocks so far, of this CTA
  bool ok = true;

  if (warp < G::kSumWarps) {
    if constexpr (G::kSumRegs > G::kLaunchRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(G::kSumRegs));
    // ------------------------------------------------ running sums: lane n of D, columns kRows wg ..
    const int wg = warp / 4, n = warp % 4 * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(warp % 4 * 32) << 16) + G::kRows * wg;
    int d = 0, stage = 0, slot = 0;
    uint32_t phase = 0;
    while (ok && walk.next(tile, g0, g1)) {
      const Tile t = find_tile<BT>(tile, m_tiles, a);
      const int mine = min(max(t.cols - G::kRows * wg, 0), G::kRows);  // of this thread's columns
      F2 acc[G::kPairs];
#pragma unroll
      for (int i = 0; i < G::kPairs; ++i) acc[i] = F2(0.f, 0.f);
      // token lanes: the factor, read a block ahead
      const float* s_x = a.s_x + (int64_t)g0 * a.M + min(t.lane + n, M - 1);
      const float* s_w = a.s_w + (int64_t)min(t.col / 128 + wg * G::kRows / 128, (int)((a.N + 127) / 128) - 1) * blocks + g0;
      float next_x = 0.f, next_w = 0.f;
      if constexpr (G::kTokenLanes) {
        next_x = *s_x;
        next_w = __ldg(s_w);
      }
      for (int g = g0; g < g1 && ok; ++g) {
        const float f = next_x * next_w;
        const F2 f2(f, f);
        if constexpr (G::kTokenLanes) {
          if (g + 1 < g1) {
            next_x = *(s_x += a.M);
            next_w = __ldg(++s_w);
          }
        }
        ok = __all_sync(0xFFFFFFFFu, wait_for(smem_u32(&bars.done[stage]), phase, abort_flag, err, 802));
        if (!ok) break;
        tc_fence_after();
        const uint32_t factors = sm + G::kFactorAt + (slot * BT + G::kRows * wg) * 4;
#pragma unroll
        for (int c = 0; c < G::kRows / 16; ++c) {
          uint32_t v[16];
          const bool any = 16 * c < mine;
          if (any) {
            tmem_ld16_nowait(lanes + d * BT + 16 * c, v);
            wait_loaded(v);
          }
          if (c + 1 == G::kRows / 16) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars.d_empty[d]));  // the sum is in registers
          }
          if (any && G::kTokenLanes) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              acc[8 * c + i] = fma2(F2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])), f2, acc[8 * c + i]);
          } else if (any) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                float4 f;
                asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                             : "=f"(f.x), "=f"(f.y), "=f"(f.z), "=f"(f.w)
                             : "r"(factors + (16 * c + 4 * i) * 4));
                F2& s0 = acc[8 * c + 2 * i];
                F2& s1 = acc[8 * c + 2 * i + 1];
                s0 = fma2(F2(__uint_as_float(v[4 * i]), __uint_as_float(v[4 * i + 1])), F2(f.x, f.y), s0);
                s1 = fma2(F2(__uint_as_float(v[4 * i + 2]), __uint_as_float(v[4 * i + 3])), F2(f.z, f.w), s1);
              }
          }
        }
        if (++d == G::kSums) d = 0;
        if (++slot == G::kSlots) slot = 0;
        if (++stage == G::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
      if (g0 > 0) {
        // another CTA has the tile's first block: this one's sums go to it
        F2* part = reinterpret_cast<F2*>(parts) + (size_t)walk.me * (G::kPartBytes / 8) + tid;
#pragma unroll
        for (int i = 0; i < G::kPairs; ++i)
          if (2 * i < mine) __stcg(reinterpret_cast<unsigned long long*>(part + i * G::kSumThreads), acc[i].v);
        raise_flag(flags + walk.me * G::kSumWarps + warp, lane);
        continue;
      }
      if (g1 < blocks) {
        // the others' sums, in the order of their blocks; a warp's lanes wait for all of them at once
        const int end = (tile - walk.rounds * walk.grid + 1) * blocks;
        int last = walk.me + 1;
        while (last < walk.ctas && walk.begin_of(last) < end) ++last;
        ok = wait_flags(flags + warp, G::kSumWarps, walk.me + 1, last, lane, abort_flag, err, 803);
        if (!ok) break;
        for (int q = walk.me + 1; q < last; ++q) {
          const F2* part = reinterpret_cast<const F2*>(parts) + (size_t)q * (G::kPartBytes / 8) + tid;
#pragma unroll
          for (int i = 0; i < G::kPairs; ++i)
            if (2 * i < mine) {
              F2 o;
              o.v = __ldcg(reinterpret_cast<const unsigned long long*>(part + i * G::kSumThreads));
              acc[i] = add2(acc[i], o);
            }
        }
        __syncwarp();
        for (int q = walk.me + 1 + lane; q < last; q += 32) flags[q * G::kSumWarps + warp] = 0;
      }
      if constexpr (G::kTokenLanes) {
        // 32 columns of the warp's 32 tokens at once go through shared memory, so that four lanes write 64 bytes of a row
        // (each lane its own row's 16 bytes: 466 us against 399 for 4096 tokens through 4096 x 28672).  16-byte piece c of row r is at c ^ (r / 2) % 4: no bank conflicts.
        uint8_t* own = smem + G::kFactorAt + warp * 2048;
        const int row = lane / 4, piece = lane % 4, m = t.lane + warp % 4 * 32 + row;
        uint16_t* p = a.y + (int64_t)m * a.N + t.col + G::kRows * wg + 8 * piece;
#pragma unroll
        for (int h = 0; h < G::kRows / 32; ++h) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = pack2<BF16>(acc[16 * h + 4 * i + j].get().x, acc[16 * h + 4 * i + j].get().y);
            *reinterpret_cast<uint4*>(own + lane * 64 + ((i ^ (lane / 2 & 3)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 v = *reinterpret_cast<const uint4*>(own + (row + 8 * i) * 64 + ((piece ^ (row / 2 & 3)) << 4));
            if (m + 8 * i < M && 32 * h + 8 * piece < mine)  // N % 8 == 0
              *reinterpret_cast<uint4*>(p + (int64_t)(8 * i) * a.N + 32 * h) = v;
          }
          __syncwarp();
        }
      } else {
        // Two neighbouring lanes swap one of a pair of tokens each, so that a lane writes two outputs of one token.
        const int64_t col = (int64_t)t.lane + (n & ~1);
        const bool odd = lane & 1;
        uint16_t* p = a.y + (int64_t)(t.col + G::kRows * wg + odd) * a.N + col;
        const int rows = col < a.N ? mine - odd : 0;  // N is even
#pragma unroll
        for (int i = 0; i < G::kPairs; ++i) {
          const float2 v = acc[i].get();
          const float got = __shfl_xor_sync(0xFFFFFFFFu, odd ? v.x : v.y, 1);
          const uint32_t w = odd ? pack2<BF16>(got, v.y) : pack2<BF16>(v.x, got);
          if (2 * i < rows) *reinterpret_cast<uint32_t*>(p) = w;
          p += 2 * a.N;
          asm volatile("" : "+l"(p));  // one address at a time, not all made ahead
        }
      }
    }
  } else {
    if constexpr (G::kOtherRegs < G::kLaunchRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(G::kOtherRegs));
    if (warp == G::kMmaWarp) {
      // ------------------------------------------------ products
      const uint64_t desc0 = smem_desc_sw128(sm, 16, 1024);
      int d = 0, stage = 0;
      uint32_t phase = 0, d_phase = 1;
      while (ok && walk.next(tile, g0, g1)) {
        const Tile t = find_tile<BT>(tile, m_tiles, a);
        const uint32_t idesc = (1u << 4) | ((uint32_t)((t.cols + 15) / 16 * 2) << 17) | (8u << 24);  // e4m3 x e4m3, fp32 sums
#pragma unroll 1
        for (int g = g0; g < g1; ++g) {
          ok = wait_for(smem_u32(&bars.full[stage]), phase, abort_flag, err, 821);
          ok = __all_sync(0xFFFFFFFFu, ok && wait_for(smem_u32(&bars.d_empty[d]), d_phase, abort_flag, err, 822));
          if (!ok) break;
          tc_fence_after();
          const uint64_t at = desc0 + (uint64_t)((stage * G::kBytes) >> 4);
          mma_block(tmem + d * BT, at, at + (uint64_t)(kABytes >> 4), idesc);
          commit(smem_u32(&bars.done[stage]));
          if (++d == G::kSums) {
            d = 0;
            d_phase ^= 1u;
          }
          if (++stage == G::kStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      commit(smem_u32(&bars.end));  // arrives once every product has completed
      volatile int no_abort = 0;
      wait_for(smem_u32(&bars.end), 0, &no_abort, err, 824);
    } else if (warp == G::kMmaWarp + 1) {
      // ------------------------------------------------ copies of weights and codes
      if (lane == 0) {
        int stage = 0;
        uint32_t phase = 1;
        while (ok && walk.next(tile, g0, g1)) {
          const Tile t = find_tile<BT>(tile, m_tiles, a);
          const int boxes = (t.cols + G::kBoxRows - 1) / G::kBoxRows;
          for (int g = g0; g < g1; ++g, ++count) {
            ok = wait_for(smem_u32(&bars.done[stage]), phase, abort_flag, err, 831);
            if (!ok) break;
            const uint32_t bar = smem_u32(&bars.full[stage]), to = sm + stage * G::kBytes;
            mbar_arrive_tx(bar, (uint32_t)(kABytes + (QUANT ? 0 : boxes * G::kBoxRows * 128)));
            tma_load_2d(to, &tm_lanes, g * 128, t.lane, bar);
            for (int i = 0; !QUANT && i < boxes; ++i)
              tma_load_2d(to + kABytes + i * G::kBoxRows * 128, &tm_cols, g * 128, t.col + i * G::kBoxRows, bar);
            if (++stage == G::kStages) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
        // never leave the CTA with copies in flight; one limit is enough for all, where factors are missing after an abort
        volatile int no_abort = 0;
        for (int j = max(0, count - G::kStages); j < count; ++j)
          if (!wait_for(smem_u32(&bars.full[j % G::kStages]), (uint32_t)(j / G::kStages) & 1u, &no_abort, err, 832)) break;
      }
    } else if constexpr (!G::kTokenLanes) {
      // ------------------------------------------------ factors s_x s_w of a block's tokens, and the codes if need be
      // What a block needs is read kAhead blocks before; `ahead` is the walk that far on.
      constexpr int kAhead = 4;
      float* factors = reinterpret_cast<float*>(smem + G::kFactorAt);
      int stage = 0, slot = 0, tile_a, a0 = 0, a1 = 0;
      uint32_t phase = 1;
      Walk ahead = walk;
      Tile ta = {0, 0, 0};
      auto more = [&]() {  // the next block of `ahead` is a0 of tile ta
        if (a0 < a1) return true;
        if (!ahead.next(tile_a, a0, a1)) return false;
        ta = find_tile<BT>(tile_a, m_tiles, a);
        return true;
      };
      if constexpr (QUANT) {
        // kAhead blocks at once, their (block, token) pairs dealt out to the four half warps in one round for a token; one fence
        // makes all their codes visible to the products.  Loops, not unrolled: a call of one token runs through here three
        // times, and code that has to be fetched first costs more than it does (19 us unrolled, 12 so).
        const int w = warp - G::kMmaWarp - 2, sub = lane % 16, item = 2 * w + lane / 16;
        static_assert(kFp8FusedTokens == 2, "one or two tokens, an even share of a block's items for each");
        const int lg = M - 1, rounds = M;
        while (ok) {
          int block[kAhead], out[kAhead], n = 0;
#pragma unroll
          for (int j = 0; j < kAhead; ++j) {
            block[j] = out[j] = 0;
            if (more()) {
              block[j] = a0++;
              out[j] = ta.lane / kLanes;
              ++n;
            }
          }
          if (n == 0) break;
          uint4 x;
          float s_w;
          auto read = [&](int p) {
            const int it = 4 * p + item, j = it >> lg, row = it & (rounds - 1);
            const int g = j == 0 ? block[0] : j == 1 ? block[1] : j == 2 ? block[2] : block[3];
            const int o = j == 0 ? out[0] : j == 1 ? out[1] : j == 2 ? out[2] : out[3];
            const int k = g * 128 + sub * 8;
            x = row < M && k < (int)a.K ? *reinterpret_cast<const uint4*>(a.x + row * a.x_stride + k) : make_uint4(0u, 0u, 0u, 0u);
            s_w = __ldg(a.s_w + (int64_t)o * blocks + g);
          };
          read(0);
#pragma unroll 1
          for (int j = 0; j < n && ok; ++j) {
            const int at = stage + j;
            ok = wait_for(smem_u32(&bars.done[at < G::kStages ? at : at - G::kStages]), at < G::kStages ? phase : phase ^ 1u,
                          abort_flag, err, 842);
          }
          ok = __all_sync(0xFFFFFFFFu, ok);
          if (!ok) break;
#pragma unroll 1
          for (int p = 0; p < rounds; ++p) {
            const uint4 now = x;
            const float w_now = s_w;
            if (p + 1 < rounds) read(p + 1);
            float scale;
            const uint2 codes = quantize8<BF16>(now, scale);
            const int it = 4 * p + item, j = it >> lg, row = it & (rounds - 1);
            if (j < n && row < M) {
              const int at = stage + j < G::kStages ? stage + j : stage + j - G::kStages;
              const int sl = slot + j < G::kSlots ? slot + j : slot + j - G::kSlots;
              *reinterpret_cast<uint2*>(smem + at * G::kBytes + kABytes + row * 128 + (((sub / 2) ^ (row & 7)) << 4) + sub % 2 * 8) =
                  codes;
              if (sub == 0) factors[sl * BT + row] = scale * w_now;
            }
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
#pragma unroll 1
          for (int j = 0; j < n; ++j) {
            if (lane == 0) mbar_arrive(smem_u32(&bars.full[stage]));
            if (++slot == G::kSlots) slot = 0;
            if (++stage == G::kStages) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
      } else if (warp == G::kMmaWarp + 2) {
        constexpr int kEach = (BT + 31) / 32;  // factors of a lane
        struct Block {
          float f[kEach];
          bool in;
        } ring[kAhead];
        auto read = [&](Block& b) {
          b.in = more();
          if (!b.in) return;
          const float w = __ldg(a.s_w + (int64_t)(ta.lane / kLanes) * blocks + a0);
          const float* s_x = a.s_x + (int64_t)a0 * a.M + ta.col;
#pragma unroll
          for (int i = 0; i < kEach; ++i) b.f[i] = lane + 32 * i < ta.cols ? s_x[lane + 32 * i] * w : 0.f;
          ++a0;
        };
#pragma unroll
        for (int j = 0; j < kAhead; ++j) read(ring[j]);
        while (ok) {
#pragma unroll
          for (int j = 0; j < kAhead; ++j) {
            if (!ring[j].in || !ok) {
              ok = false;
              break;
            }
            ok = __all_sync(0xFFFFFFFFu, wait_for(smem_u32(&bars.done[stage]), phase, abort_flag, err, 841));
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < kEach; ++i)
              if (lane + 32 * i < BT) factors[slot * BT + lane + 32 * i] = ring[j].f[i];
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars.full[stage]));  // no product starts without them: `done` cannot run two rounds ahead
            read(ring[j]);
            if (++slot == G::kSlots) slot = 0;
            if (++stage == G::kStages) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == G::kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"((uint32_t)G::kTmem) : "memory");
  }
}

// 16 or 64 token columns (4096 x 28672: 16 tokens 28.7 and 30.0 us, 24 tokens 40.2 and 29.7), or 256 output columns.  Above 64
// tokens the form that is expected to be faster, both in microseconds, fitted to 80 to 768 tokens, 1024 to 28672 outputs and 2048
// to 14336 inputs: a block of a CTA takes 0.37 and 0.53; the larger tiles, where they are few, are joined from many CTAs' parts
// of 131 KB (64 and 256 columns, 4096 x 4096: 128 tokens 15.1 and 33.1, 512 tokens 27.9 and 27.4, 768 tokens 38.2 and 28.2;
// 4096 x 28672: 64 tokens 30.5 and 37.2, 80 tokens 44.1 and 38.2).
int tile_columns(int64_t M, int64_t K, int64_t N) {
  if (M <= 64) return M <= 16 ? 16 : 64;
  const double blocks = (double)((K + 127) / 128) / device_sm_count();
  const double small = (double)((M + 63) / 64) * (double)((N + 127) / 128), large = (double)((M + 127) / 128) * (double)((N + 255) / 256);
  return 10 + 0.37 * small * blocks <= 15 + 320 / large + 0.53 * large * blocks ? 64 : 256;
}

template <int BT, bool BF16, bool QUANT = false>
cudaError_t launch(const Fp8GemmArgs& a, void* ws, int* err, cudaStream_t s) {
  using G = Geo<BT>;
  const auto fn = fp8_gemm_kernel<BT, BF16, QUANT>;
  const cudaError_t e = set_smem_once(reinterpret_cast<const void*>(fn), G::kSmem);
  if (e != cudaSuccess) return e;
  // the operand of the lanes in one box, that of the columns in boxes of up to 64 rows
  const auto map = [&](CUtensorMap* tm, const uint8_t* p, int64_t rows, bool lanes) {
    return make_map_2d(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, p, (uint64_t)a.K, (uint64_t)rows, 128, lanes ? kLanes : G::kBoxRows,
                       CU_TENSOR_MAP_SWIZZLE_128B);
  };
  CUtensorMap tw, tx = {};
  if (!map(&tw, a.wq, a.N, !G::kTokenLanes) || (!QUANT && !map(&tx, a.xq, a.M, G::kTokenLanes))) return cudaErrorInvalidValue;
  const int64_t m_tiles = (a.M + (G::kTokenLanes ? kLanes : BT) - 1) / (G::kTokenLanes ? kLanes : BT);
  const int64_t n_tiles = (a.N + (G::kTokenLanes ? BT : kLanes) - 1) / (G::kTokenLanes ? BT : kLanes);
  if (n_tiles * m_tiles > INT32_MAX) return cudaErrorInvalidValue;
  int* flags = static_cast<int*>(ws);
  float* parts = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kCounterBytes);
  return launch_dependent(fn, dim3(device_sm_count()), G::kThreads, G::kSmem, s, G::kTokenLanes ? tx : tw,
                          G::kTokenLanes ? tw : tx, a, (int)m_tiles, (int)(n_tiles * m_tiles), flags, parts, err);
}

}  // namespace

// flags | parts of shared tiles
size_t fp8_gemm_workspace(int64_t M, int64_t K, int64_t N) {
  return kCounterBytes + (size_t)device_sm_count() * kLanes * (size_t)tile_columns(M, K, N) * 4;
}

cudaError_t launch_fp8_gemm(const Fp8GemmArgs& a, bool bf16, void* ws, int* err, cudaStream_t s) {
  const int bt = tile_columns(a.M, a.K, a.N);
  if (a.x) return bf16 ? launch<16, true, true>(a, ws, err, s) : launch<16, false, true>(a, ws, err, s);
  const auto fn = bt == 16   ? (bf16 ? launch<16, true> : launch<16, false>)
                  : bt == 64 ? (bf16 ? launch<64, true> : launch<64, false>)
                             : (bf16 ? launch<256, true> : launch<256, false>);
  return fn(a, ws, err, s);
}

}  // namespace awq
