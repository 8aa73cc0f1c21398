// Attention of many new tokens over the 4-bit paged cache on the 5th-generation tensor cores.
//
// The mathematics is kv4_attention.cu's: with keys zk + u sk and values zv + u sv,
//   T_j = sk_j (q' . u_j) + zk_j r,  p_j = 2^(qk T_j - base),
//   out = (sum_j (p_j sv_j) (u_j - 8) + sum_j p_j (zv_j + 8 sv_j)) / sum_j p_j
// where q' is the query row times a power of two, exact in fp16, and qk, r carry that factor, the scale and sum(q).
// Only codes and exact fp16 queries enter the score's products, so the scores are as exact as fp32 sums are; the
// weights p sv are rounded to fp16 once.
//
// A CTA takes 256 query rows (query token, head) of one cache head in two tiles of 128, and goes over the cache in
// tiles of 128 tokens, in two steps of 64.  tcgen05.mma kind::f16, M = 128:
//   S[row][token] = Q' U_k^T   A = queries, B = key codes, both K-major in shared memory, N = 64
//   O[row][channel] += W U_v   A = weights, in tensor memory where S was, B = value codes, K-major, N = D
// A key's codes become fp16 halves with one AND for two of them: u 2^-24 in the lowest nibble, 16 u 2^-24 in the next
// (the factor 16 is taken out of the queries' channels 2, 3 of four).  A value's become u - 8, with one operation more,
// so that the rounding of the weights counts by the code's distance from the middle: a third of the error.
//
// Roles: warps 0-3 and 4-7 are the softmax of the two row tiles (a thread has a row), warps 8 and 9 issue their
// products, warp 10 copies units, warps 11-14 turn codes into operands.  While one row tile's softmax runs, the other's
// products do; a tile's two halves of 64 tokens have an S each, so that a row tile's next scores are there before it is done
// with the present ones.  The output stays in tensor memory; it is rescaled only when a row's maximum has grown by more
// than 2^8, so the weights are at most 2^8 and enter fp16 as p sv 2^(5 - e), 2^e the largest value scale so far.
//
// Measured: 2 x 1024 tokens over 4095 and 2376, 32 heads on 8, 122 us, 748 TFLOP/s (the products alone would take 47 at
// the library GEMM's rate).  A step of 64 tokens takes a softmax warp 1900 cycles when it is alone on its sub-partition,
// 2500 beside another.  Two things are near their limits in a capture: shared memory, with 0.5 wavefronts a cycle of loads
// and stores and 0.3 of the products' operands, and the issue slots, 57 % busy between dependences; which of them bounds
// a step has not been separated.  256 CTAs of 24 to 64 steps on 152 SMs also leave a sixth of the SMs' time unused.  A CTA's start and end cost 6 us.  Slower and left out: two
// threads for a row (176 us against 159), threads with a row of both row tiles (196 against 161), one product warp for
// both row tiles (180 against 161), weights made with the maximum of the steps before, in one pass (147 against 121).
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "awq_host.h"
#include "awq_internal.h"
#include "awq_ptx.cuh"
#include "awq_types.cuh"
#include "kv4_attention.cuh"

namespace awq {
namespace {

constexpr int kRows = 256;   // query rows of a CTA
constexpr int kTok = 128;    // tokens of a tile
constexpr int kHalf = 64;    // tokens of a raw slot, and of one step of the softmax
constexpr int kBufs = 4;     // operand buffers of a step's keys, and of its values
// Scales and zeros of a step stay until its weights are made.  A step's keys are made at the earliest when the values
// of the one before it are, which is after the weights of five steps before: six buffers.  They have full barriers of
// their own: the keys' come round again when the products alone have read the keys, before a softmax warp need have looked.
constexpr int kMetas = 6;
constexpr int kRaw = 3;      // raw slots
constexpr int kDqThreads = 128;
constexpr int kThreads = 512;  // the last warp has no work: setmaxnreg wants whole groups of four warps
// Registers.  At 128 for every thread, the softmax warps have too few to keep enough of a step's 64 scores, scales
// and zeros under way: the chunk of 2 x 1024 tokens took 138 us, at 160 / 96 and more it takes 121, at 176 / 80 120.
constexpr int kLaunchRegs = 128, kSoftmaxRegs = 176, kOtherRegs = 80;
static_assert(256 * kSoftmaxRegs + (kThreads - 256) * kOtherRegs <= kThreads * kLaunchRegs, "no more than was launched with");
constexpr float kGrow = 8.f;  // growth of the maximum (base 2) that rescales the output

template <int D>
struct Geo {
  static constexpr int kUnitBytes = kv4_unit_bytes(D);
  static constexpr int kUnitStride = kUnitBytes + 32;  // units 32 bytes apart in the banks: the value words' reads
  static constexpr int kRawBytes = 4 * kUnitStride;
  static constexpr int kQTile = 128 * D * 2;           // one row tile, D / 64 blocks of 128 rows x 128 bytes
  static constexpr int kKStep = kHalf * D * 2;         // a step's keys, D / 64 blocks of 64 rows x 128 bytes
  static constexpr int kVStep = kHalf * D * 2;         // a step's values, D rows x 128 bytes
  static constexpr int kQ = 0, kK = kQ + 2 * kQTile, kV = kK + kBufs * kKStep, kMeta = kV + kBufs * kVStep;
  static constexpr int kMetaBytes = 4 * kHalf * 4 + 16;  // key scale, key zero, value scale, value zero; largest exponents
  static constexpr int kRawAt = kMeta + kMetas * kMetaBytes;
  static constexpr int kSmem = kRawAt + kRaw * kRawBytes + 1024;
  static constexpr uint32_t kIdescS = (1u << 4) | ((kHalf / 8) << 17) | ((128 / 16) << 24);
  static constexpr uint32_t kIdescO = (1u << 4) | ((D / 8) << 17) | ((128 / 16) << 24);
  static_assert(kSmem <= 227 * 1024 - 512, "shared memory");
};

// Waits for this thread's tensor memory loads; `r` is not used before.
__device__ __forceinline__ void wait_loaded(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

struct Bars {
  uint64_t raw_full[kRaw], raw_empty[kRaw], k_full[kBufs], k_empty[kBufs], v_full[kBufs], v_empty[kBufs], meta_full[kMetas],
      s_full[2][2], p_full[2][2], o_done[2][2], q_full, done;
};

// The products and commits are executed by the whole warp, with the same operands in every lane, and issued by
// the one that elect.sync chooses (always the same): operands that the compiler sees as uniform need no moves between
// register files before each product, which cost more than the product itself.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n elect.sync _|q, 0xFFFFFFFF;\n setp.ne.b32 p, %4, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// A in tensor memory: a lane for each row, two halves a column.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n elect.sync _|q, 0xFFFFFFFF;\n setp.ne.b32 p, %4, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xFFFFFFFF;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Two codes of a word as exact halves u - 8: nibbles 0 and 4 (odd = 0), or 1 and 5.
__device__ __forceinline__ uint32_t centred(int odd, uint32_t w) {
  // 1024 + u, or 1024 + 16 u
  const uint32_t b = (w & (odd ? 0x00F000F0u : 0x000F000Fu)) | 0x64006400u;
  const __half2 h = *reinterpret_cast<const __half2*>(&b);
  const __half2 r = odd ? __hfma2(h, __float2half2_rn(0.0625f), __float2half2_rn(-72.f)) : __hsub2(h, __float2half2_rn(1032.f));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// What one CTA does: rows row0 .. of cache head kv_head of a sequence, and the tiles of its share of the cache.
struct Job {
  int begin, n, len, lo;  // query tokens, cached tokens, the first token that any row sees
  int row0, kv_head;
  int tile0;              // first tile
  int count[2];           // tiles of each row tile
  int total;              // the larger one
};
__device__ __forceinline__ Job job_of(const Args& a, int row_block, int kv_head, int b, int split, int splits) {
  const int3 s = read_seq(a, b);
  Job j;
  j.begin = s.x;
  j.n = s.y;
  j.len = s.z;
  j.row0 = row_block * kRows;
  j.kv_head = kv_head;
  j.lo = 0;
  j.tile0 = 0;
  j.count[0] = j.count[1] = j.total = 0;
  const int rows = s.y * a.per;
  if (j.row0 >= rows || rows <= a.rows) {
    j.n = 0;  // nothing to do here
    return j;
  }
  const int first = s.z - s.y + j.row0 / a.per;  // the first row's position
  j.lo = a.window > 0 ? min(max(0, first - a.window + 1), s.z) : 0;
  const int base = j.lo / kTok;
  int want[2];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const int last = min(j.row0 + 128 * m + 127, rows - 1);
    const int end = s.z - s.y + last / a.per + 1;  // tokens that the row tile's last row sees
    want[m] = j.row0 + 128 * m < rows && end > 0 ? max(0, (end + kTok - 1) / kTok - base) : 0;
  }
  const int all = max(want[0], want[1]);
  const int t0 = (int)((long long)all * split / splits), t1 = (int)((long long)all * (split + 1) / splits);
  j.tile0 = base + t0;
#pragma unroll
  for (int m = 0; m < 2; ++m) j.count[m] = min(max(want[m] - t0, 0), t1 - t0);
  j.total = max(j.count[0], j.count[1]);
  return j;
}

// Floats of a CTA's partial result: output [channel / 4][row][channel % 4], then maximum and sum of every row.
__host__ __device__ constexpr long long part_floats(int dim) { return (long long)kRows * (dim + 2); }

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1)
kv4_prefill_kernel(const Args a, int splits, float* parts, int* err) {
  using G = Geo<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Bars bars;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;
  // the join, launched early, waits for this grid before it reads what is written here
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid / 32, 0), lane = tid % 32;
  // heads of a row block first, then the row blocks from the one that sees the most tokens down: CTAs start in the
  // order of their work, and the short ones fill what the long ones leave.  All on the grid's x, the one without a limit.
  const int place = blockIdx.x / a.kv_heads, kv_head = blockIdx.x - place * a.kv_heads;
  const int split = place % splits, row_blocks = gridDim.x / a.kv_heads / splits;
  const int row_block = row_blocks - 1 - place / splits;
  const Job job = job_of(a, row_block, kv_head, blockIdx.y, split, splits);
  if (job.row0 >= job.n * a.per) return;
  uint8_t* smem = align_smem_1024(smem_raw);
  const uint32_t sm = smem_u32(smem);

  if (tid == 0) {
    abort_word = 0;
    for (int i = 0; i < kRaw; ++i) {
      mbar_init(smem_u32(&bars.raw_full[i]), 1);
      mbar_init(smem_u32(&bars.raw_empty[i]), kDqThreads);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(smem_u32(&bars.k_full[i]), kDqThreads);
      mbar_init(smem_u32(&bars.v_full[i]), kDqThreads);
      mbar_init(smem_u32(&bars.k_empty[i]), 2);
      mbar_init(smem_u32(&bars.v_empty[i]), 2);
    }
    for (int i = 0; i < kMetas; ++i) mbar_init(smem_u32(&bars.meta_full[i]), kHalf);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&bars.s_full[i][0]), 1);
      mbar_init(smem_u32(&bars.s_full[i][1]), 1);
      mbar_init(smem_u32(&bars.o_done[i][0]), 1);
      mbar_init(smem_u32(&bars.o_done[i][1]), 1);
      mbar_init(smem_u32(&bars.p_full[i][0]), 128);
      mbar_init(smem_u32(&bars.p_full[i][1]), 128);
    }
    mbar_init(smem_u32(&bars.q_full), 256);
    mbar_init(smem_u32(&bars.done), 2);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async();
  }
  if (warp == 8) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&tmem_slot)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;  // S of row tile m at column 128 m, O at 256 + 128 m

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // ------------------------------------------------ softmax: a thread has a row
    const int m = warp / 4, r = tid % 128;
    const int col = job.row0 + 128 * m + r, i = col / a.per;
    const bool in = i < job.n;
    const int64_t token = job.begin + i;
    const int head = job.kv_head * a.per + col - i * a.per;
    constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes;  // lanes of a row, rows of a warp at once
    // chunk c (16 bytes) of row `row` of this row tile's queries, later of its output
    auto row_at = [&](int row, int c) {
      return sm + G::kQ + m * G::kQTile + (c / 8) * 16384 + row * 128 + ((c % 8) ^ (row % 8)) * 16;
    };
    const float sign = a.scale > 0.f ? 1.f : a.scale < 0.f ? -1.f : 0.f;
    const float factor = a.scale == 0.f ? kLog2e : fabsf(a.scale) * kLog2e;
    float qk, qr;
    {
      // The warp's rows come into the operand's place as they are, whole rows at once; then a thread scales its own.
      const int64_t at = in ? token * a.q_stride + head * D : -1;
      uint4 v[kLanes];
#pragma unroll
      for (int k = 0; k < kLanes; ++k) {
        const int64_t from = __shfl_sync(0xFFFFFFFFu, at, k * kAtOnce + lane / kLanes);
        v[k] = from >= 0 ? *reinterpret_cast<const uint4*>(a.q + from + 8 * (lane % kLanes)) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int k = 0; k < kLanes; ++k)
        sts128(row_at(warp % 4 * 32 + k * kAtOnce + lane / kLanes, lane % kLanes), v[k].x, v[k].y, v[k].z, v[k].w);
      __syncwarp();
      float top = 0.f, sum = 0.f;
#pragma unroll
      for (int c = 0; c < kLanes; ++c) {
        v[c] = lds128(row_at(r, c));
        const uint32_t w[4] = {v[c].x, v[c].y, v[c].z, v[c].w};
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const float2 f = unpack2<BF16>(w[p]);
          top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
          sum += f.x + f.y;
        }
      }
      // a power of two takes the largest element to [2^14, 2^15): exact in fp16 down to 2^-24 of it, sixteenths too
      const int e = min(max((int)(__float_as_uint(top) >> 23) - 127, -100), 127);
      const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23) * sign, up16 = up * 0.0625f;
#pragma unroll
      for (int c = 0; c < kLanes; ++c) {
        const float2 f0 = unpack2<BF16>(v[c].x), f1 = unpack2<BF16>(v[c].y), f2 = unpack2<BF16>(v[c].z), f3 = unpack2<BF16>(v[c].w);
        sts128(row_at(r, c), pack2<false>(f0.x * up, f0.y * up), pack2<false>(f1.x * up16, f1.y * up16),
               pack2<false>(f2.x * up, f2.y * up), pack2<false>(f3.x * up16, f3.y * up16));
      }
      // not 0, which would make a NaN of a masked score, -inf; below that the weights are equal anyway
      qk = fmaxf(__uint_as_float((uint32_t)max(127 + e - 14, 1) << 23) * 16777216.f * factor, FLT_MIN);
      qr = sum * (up * 5.9604644775390625e-8f);
    }
    fence_async();
    mbar_arrive(smem_u32(&bars.q_full));

    const int pos = in ? job.len - job.n + i : -1;
    const int first_pos = job.len - job.n + (job.row0 + 128 * m) / a.per;  // of the row tile's first row
    const int last_pos = job.len - job.n + min((job.row0 + 128 * m + 127) / a.per, job.n - 1);
    const uint32_t s_addr = tmem + 128 * m + ((uint32_t)(warp % 4 * 32) << 16);
    const uint32_t o_addr = s_addr + 256;
    float top = -INFINITY, l = 0.f, z = 0.f;
    int vexp = -16;
    bool ok = true;
    const int count = job.count[m];
    const F2 qr2(qr, qr), qk2(qk, qk);
    for (int j = 0; j < count && ok; ++j) {
#pragma unroll 1
      for (int h = 0; h < 2; ++h) {
        const int j0 = (job.tile0 + j) * kTok + h * kHalf;
        const int step = 2 * j + h;
        const uint8_t* meta = smem + G::kMeta + step % kMetas * G::kMetaBytes;
        ok = __all_sync(0xFFFFFFFFu,
                        wait_bounded_inline(smem_u32(&bars.s_full[m][h]), j & 1, abort_flag, err, 621) &&
                            wait_bounded_inline(smem_u32(&bars.meta_full[step % kMetas]), step / kMetas & 1, abort_flag, err, 622));
        if (!ok) break;
        tc_fence_after();
        uint32_t raw[4][16];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld16_nowait(s_addr + h * kHalf + 16 * c, raw[c]);
#pragma unroll
        for (int c = 0; c < 4; ++c) wait_loaded(raw[c]);
        const float4* ks = reinterpret_cast<const float4*>(meta + 0 * kHalf * 4);
        const float4* kz = reinterpret_cast<const float4*>(meta + 1 * kHalf * 4);
        const float4* vs = reinterpret_cast<const float4*>(meta + 2 * kHalf * 4);
        const float4* vz = reinterpret_cast<const float4*>(meta + 3 * kHalf * 4);
        const int2 ve2 = *reinterpret_cast<const int2*>(meta + 4 * kHalf * 4);
        F2 t[32];
#pragma unroll
        for (int q = 0; q < 16; ++q) {
          const float4 s4 = ks[q], z4 = kz[q];
          const uint32_t* x = &raw[q / 4][q % 4 * 4];
          t[2 * q] = fma2(F2(s4.x, s4.y), F2(__uint_as_float(x[0]), __uint_as_float(x[1])), mul2(F2(z4.x, z4.y), qr2));
          t[2 * q + 1] = fma2(F2(s4.z, s4.w), F2(__uint_as_float(x[2]), __uint_as_float(x[3])), mul2(F2(z4.z, z4.w), qr2));
        }
        const bool edge = j0 + kHalf > first_pos + 1 || (a.window > 0 && j0 < last_pos + 1 - a.window) || j0 < job.lo;
        int most = max(ve2.x, ve2.y);
        if (edge) {
          // a token hidden from this row takes no bits from its weights: the largest scale of those it sees
          const int from = a.window > 0 ? pos - a.window + 1 : 0;
          float seen = 0.f;
#pragma unroll
          for (int q = 0; q < 32; ++q) {
            const float2 v = t[q].get();
            const int at = j0 + 2 * q;
            const bool no0 = at > pos || at < from, no1 = at + 1 > pos || at + 1 < from;
            t[q] = F2(no0 ? -INFINITY : v.x, no1 ? -INFINITY : v.y);
            const float2 s2 = reinterpret_cast<const float2*>(vs)[q];
            seen = fmaxf(seen, fmaxf(no0 ? 0.f : fabsf(s2.x), no1 ? 0.f : fabsf(s2.y)));
          }
          most = min((int)(__float_as_uint(seen) >> 23) - 126, 17);  // below 2^most; infinity as in the scales' exponents
        }
        float highs[8] = {top, top, top, top, top, top, top, top};
#pragma unroll
        for (int q = 0; q < 32; ++q) {
          const float2 v = t[q].get();
          highs[q % 8] = fmaxf(highs[q % 8], fmaxf(v.x, v.y));
        }
#pragma unroll
        for (int q = 4; q; q /= 2)
#pragma unroll
          for (int k = 0; k < q; ++k) highs[k] = fmaxf(highs[k], highs[k + q]);
        const float high = highs[0];
        const int ve = max(vexp, most);
        const bool grown = ve != vexp || (high > top && !((high - top) * qk <= kGrow));
        if (__any_sync(0xFFFFFFFFu, grown)) {
          const float f = (high > top ? ex2((top - high) * qk) : 1.f) * __uint_as_float((uint32_t)(127 + vexp - ve) << 23);
          top = high;
          vexp = ve;
          l *= f;
          z *= f;
          if (j > 0 || h > 0) {
            // the products into O so far: the last ones, of the half before, may still run
            ok = __all_sync(0xFFFFFFFFu, wait_bounded_inline(smem_u32(&bars.o_done[m][h ^ 1]), (j - 1 + h) & 1, abort_flag, err, 623));
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t o[16];
              tmem_ld16_nowait(o_addr + c, o);
              wait_loaded(o);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tmem_st16(o_addr + c, o);
            }
          }
        }
        // weights in units of 2^(vexp - 5)
        const float base = (top == -INFINITY ? 0.f : -top * qk) + (float)(5 - vexp);
        const F2 base2(base, base);
        uint32_t w[2][16];
        F2 l2(l, 0.f), z2(z, 0.f);
        auto weigh = [&](auto hides) {
#pragma unroll
          for (int q = 0; q < 16; ++q) {
            const float4 s4 = vs[q], z4 = vz[q];
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              const F2 v = t[2 * q + p];
              const float2 x = fma2(v, qk2, base2).get();
              const F2 e(ex2(x.x), ex2(x.y));
              float sa = p ? s4.z : s4.x, sb = p ? s4.w : s4.y, za = p ? z4.z : z4.x, zb = p ? z4.w : z4.y;
              if (decltype(hides)::value) {  // a token hidden from one row and seen by another may hold a NaN
                const float2 y = v.get();
                if (y.x == -INFINITY) sa = za = 0.f;
                if (y.y == -INFINITY) sb = zb = 0.f;
              }
              l2 = add2(l2, e);
              z2 = fma2(e, F2(za, zb), z2);
              const float2 y = mul2(e, F2(sa, sb)).get();
              // the values of every second eight tokens stand pair by pair the other way round
              const int pair = 2 * q + p;
              const int at = pair / 4 % 2 ? pair ^ 1 : pair;
              w[at / 16][at % 16] = pack2<false>(y.x, y.y);
            }
          }
        };
        if (edge)
          weigh(std::true_type{});
        else
          weigh(std::false_type{});
        const float2 ls = l2.get(), zs = z2.get();
        l = ls.x + ls.y;
        z = zs.x + zs.y;
#pragma unroll
        for (int c = 0; c < 2; ++c) tmem_st16(s_addr + h * kHalf + 16 * c, w[c]);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(smem_u32(&bars.p_full[m][h]));
      }
    }
    // ---- the row's result
    if (ok && count > 0) {
      // the second half's products of the last tile
      ok = __all_sync(0xFFFFFFFFu, wait_bounded_inline(smem_u32(&bars.o_done[m][1]), (count - 1) & 1, abort_flag, err, 624));
      tc_fence_after();
    }
    const float unit = __uint_as_float((uint32_t)(127 + vexp - 5) << 23);
    const int64_t row = token * a.heads + head;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    float* part = parts + ((((long long)blockIdx.y * a.kv_heads + kv_head) * row_blocks + row_block) * splits + split) * part_floats(D);
    const int pr = 128 * m + r;
    if (ok) {
#pragma unroll 1
      for (int c = 0; c < D; c += 16) {
        uint32_t o[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) o[k] = 0u;
        if (count > 0) {
          tmem_ld16_nowait(o_addr + c, o);
          wait_loaded(o);
        }
        float v[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(o[k]) + z;
        if (splits == 1) {
          uint32_t w[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) w[k] = pack2<BF16>(v[2 * k] * inv, v[2 * k + 1] * inv);
          sts128(row_at(r, c / 8), w[0], w[1], w[2], w[3]);
          sts128(row_at(r, c / 8 + 1), w[4], w[5], w[6], w[7]);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            reinterpret_cast<float4*>(part)[(c / 4 + k) * kRows + pr] =
                make_float4(v[4 * k] * unit, v[4 * k + 1] * unit, v[4 * k + 2] * unit, v[4 * k + 3] * unit);
        }
      }
      if (splits == 1) {  // whole rows at once, as the queries came
        __syncwarp();
        const int64_t at = in ? row * D : -1;
#pragma unroll
        for (int k = 0; k < kLanes; ++k) {
          const int from = k * kAtOnce + lane / kLanes;
          const int64_t to = __shfl_sync(0xFFFFFFFFu, at, from);
          const uint4 x = lds128(row_at(warp % 4 * 32 + from, lane % kLanes));
          if (to >= 0) *reinterpret_cast<uint4*>(a.out + to + 8 * (lane % kLanes)) = x;
        }
      }
      const float high = top == -INFINITY ? -INFINITY : top * qk;
      if (splits > 1) {
        part[(long long)kRows * D + pr] = high;
        part[(long long)kRows * D + kRows + pr] = l * unit;
      } else if (in && a.lse) {
        a.lse[row] = l == 0.f ? -INFINITY : (high + log2f(l * unit)) * kLn2;
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp < 10) {
      // ------------------------------------------------ products: a warp for each row tile
      const int m = warp - 8, mine = 2 * job.count[m], steps = 2 * job.total;
      auto wait = [&](uint64_t& bar, uint32_t parity, int id) {
        return __all_sync(0xFFFFFFFFu, wait_bounded_inline(smem_u32(&bar), parity, abort_flag, err, id)) != 0;
      };
      bool ok = wait(bars.q_full, 0, 611);
      const uint64_t qa = smem_desc_sw128(sm + G::kQ + m * G::kQTile, 16, 1024);
      const uint64_t kb = smem_desc_sw128(sm + G::kK, 16, 1024), vb = smem_desc_sw128(sm + G::kV, 16, 1024);
      // step: 64 tokens; the scores of even and odd steps have an S each
      auto scores = [&](int step) {
        const int buf = step % kBufs;
        ok = ok && wait(bars.k_full[buf], step / kBufs & 1, 612);
        if (!ok) return;
        tc_fence_after();
        if (step < mine) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k)
            mma_ss(tmem + 128 * m + step % 2 * kHalf, qa + (uint64_t)((k / 4) * (16384 >> 4) + (k % 4) * 2),
                   kb + (uint64_t)(buf * (G::kKStep >> 4) + (k / 4) * (kHalf * 128 >> 4) + (k % 4) * 2), G::kIdescS, k > 0 ? 1u : 0u);
          commit(smem_u32(&bars.s_full[m][step % 2]));
        }
        commit(smem_u32(&bars.k_empty[buf]));
      };
      for (int step = 0; step < 2 && step < steps; ++step) scores(step);
      for (int step = 0; step < steps && ok; ++step) {
        const int buf = step % kBufs;
        ok = wait(bars.v_full[buf], step / kBufs & 1, 614);
        if (ok && step < mine) {
          ok = wait(bars.p_full[m][step % 2], step / 2 & 1, 613);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ts(tmem + 256 + 128 * m, tmem + 128 * m + step % 2 * kHalf + 8 * k,
                   vb + (uint64_t)(buf * (G::kVStep >> 4) + k * 2), G::kIdescO, (step | k) ? 1u : 0u);
          commit(smem_u32(&bars.o_done[m][step % 2]));
        }
        if (!ok) break;
        commit(smem_u32(&bars.v_empty[buf]));
        // the scores of the step after the next go where these weights were
        if (step + 2 < steps) scores(step + 2);
      }
      // every product has completed before tensor memory is given back
      commit(smem_u32(&bars.done));
      volatile int no_abort = 0;
      wait_bounded_inline(smem_u32(&bars.done), 0, &no_abort, err, 615);
    } else if (warp == 10) {
      // ------------------------------------------------ copies: lane u takes unit u of a half tile
      const int halves = 2 * job.total;
      int issued = 0;
      for (int k = 0; k < halves; ++k) {
        const int st = k % kRaw;
        const int unit = job.tile0 * (kTok / kKv4Unit) + k * 4 + lane;
        const bool valid = lane < 4 && unit * kKv4Unit < job.len && (unit + 1) * kKv4Unit > job.lo;
        const int p = a.page_magic ? (int)__umulhi((uint32_t)unit, a.page_magic) : unit;
        int64_t page = valid ? a.block_table[blockIdx.y * a.table_stride + p] : 0;
        if ((uint64_t)page >= (uint64_t)a.num_pages) page = 0;
        if (k >= kRaw &&
            !__all_sync(0xFFFFFFFFu, wait_bounded_inline(smem_u32(&bars.raw_empty[st]), (uint32_t)(k / kRaw - 1) & 1u, abort_flag, err, 601)))
          break;
        const uint32_t n = __popc(__ballot_sync(0xFFFFFFFFu, valid));
        const uint32_t bar = smem_u32(&bars.raw_full[st]);
        if (lane == 0) mbar_arrive_tx(bar, n * G::kUnitBytes);
        __syncwarp();
        if (valid) {
          const uint8_t* src = a.cache + ((page * a.kv_heads + job.kv_head) * a.units_page + (unit - p * a.units_page)) * G::kUnitBytes;
          bulk_load(sm + G::kRawAt + st * G::kRawBytes + lane * G::kUnitStride, src, G::kUnitBytes, bar);
        }
        issued = k + 1;
      }
      // every copy lands before the CTA ends
      volatile int no_abort = 0;
      for (int k = max(0, issued - kRaw); k < issued; ++k)
        wait_bounded_inline(smem_u32(&bars.raw_full[k % kRaw]), (uint32_t)(k / kRaw) & 1u, &no_abort, err, 602);
    } else if (warp < 15) {
      // ------------------------------------------------ operands from codes
      const int d = tid - 352, w = d / 32;
      bool ok = true;
      for (int k = 0; k < 2 * job.total && ok; ++k) {
        const int st = k % kRaw, buf = k % kBufs;
        ok = __all_sync(0xFFFFFFFFu, wait_bounded_inline(smem_u32(&bars.raw_full[st]), (uint32_t)(k / kRaw) & 1u, abort_flag, err, 631));
        if (ok && k >= kBufs)
          ok = __all_sync(0xFFFFFFFFu, wait_bounded_inline(smem_u32(&bars.k_empty[buf]), (uint32_t)(k / kBufs - 1) & 1u, abort_flag, err, 632));
        if (!ok) break;
        const uint8_t* raw = smem + G::kRawAt + st * G::kRawBytes;
        // scales and zeros as fp32, zeros for tokens outside the sequence: their bytes may be anything
        if (d < kHalf) {
          const int at = job.tile0 * kTok + k * kHalf + d;
          uint2 mt = *reinterpret_cast<const uint2*>(raw + (d / 16) * G::kUnitStride + 16 * D + (d % 16) * 8);
          if (at < job.lo || at >= job.len) mt = make_uint2(0u, 0u);
          const float2 ksz = unpack2<false>(mt.x), vsz = unpack2<false>(mt.y);
          uint8_t* meta = smem + G::kMeta + k % kMetas * G::kMetaBytes;
          float* f = reinterpret_cast<float*>(meta) + d;
          f[0] = ksz.x;
          f[kHalf] = ksz.y;
          f[2 * kHalf] = vsz.x;
          f[3 * kHalf] = fmaf(8.f, vsz.x, vsz.y);
          // the value scales of these 32 tokens are below 2^(that)
          const uint32_t most = __reduce_max_sync(0xFFFFFFFFu, mt.y & 0x7FFFu);
          if (lane == 0) *reinterpret_cast<int*>(meta + 4 * kHalf * 4 + 4 * w) = (int)(most >> 10) - 14;
          mbar_arrive(smem_u32(&bars.meta_full[k % kMetas]));
        }
        // keys: a word is eight channels of a token, one 16-byte chunk of its row.  A thread has one chunk of every
        // kPass-th token, so that all its addresses are two bases and constants.
        {
          constexpr int kChunks = D / 8, kPass = kDqThreads / kChunks;
          const int c = d % kChunks, tok = d / kChunks;
          const uint8_t* src = raw + tok * (D / 2) + 4 * c;
          const uint32_t dst = sm + G::kK + buf * G::kKStep + (c / 8) * (kHalf * 128) + tok * 128 + ((c % 8) ^ (tok % 8)) * 16;
#pragma unroll
          for (int i = 0; i < kHalf / kPass; ++i) {
            const int t = i * kPass;  // a multiple of 8
            const uint32_t x = *reinterpret_cast<const uint32_t*>(src + (t / 16) * G::kUnitStride + (t % 16) * (D / 2));
            const uint32_t y = x >> 8;
            sts128(dst + t * 128, x & 0x000F000Fu, x & 0x00F000F0u, y & 0x000F000Fu, y & 0x00F000F0u);
          }
        }
        fence_async();
        mbar_arrive(smem_u32(&bars.k_full[buf]));
        if (k >= kBufs) {
          ok = __all_sync(0xFFFFFFFFu, wait_bounded_inline(smem_u32(&bars.v_empty[buf]), (uint32_t)(k / kBufs - 1) & 1u, abort_flag, err, 633));
          if (!ok) break;
        }
        // values: eight tokens of a channel are one chunk of its row.  Thread: eight tokens tc, channels [g D / 8, ...),
        // a part of its quads; odd eights read their words pair by pair the other way round, so that the reads of
        // eight lanes fall into different banks.
        {
          constexpr int kQuads = D / 32;               // quads of a group of D / 8 channels
          constexpr int kEach = kQuads / 2;            // of a thread
          const int tc = lane % 8, s = tc % 2, g = 4 * (w % 2) + lane / 8;
          const int q0 = ((w / 2) ^ (kEach == 2 ? g % 2 : 0)) * kEach;  // two groups of a half-warp: different banks
          const uint8_t* src = raw + (tc / 2) * G::kUnitStride + 8 * D + ((s * 8 + g) * 4 * kQuads + q0) * 4;
          uint32_t x[4][kEach];
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const uint8_t* at = src + (t ^ s) * kQuads * 4;
            if constexpr (kEach == 2) {
              const uint2 v = *reinterpret_cast<const uint2*>(at);
              x[t][0] = v.x;
              x[t][1] = v.y;
            } else {
              x[t][0] = *reinterpret_cast<const uint32_t*>(at);
            }
          }
          // channel g D / 8 + 4 (q0 + q) + e: rows of 128 bytes, their chunks swizzled by the channel's last three bits
          const uint32_t dst = sm + G::kV + buf * G::kVStep + (g * (D / 8) + 4 * q0) * 128 + tc * 16;
          const uint32_t swap = kEach == 1 ? 64u * (uint32_t)(q0 % 2) : 0u;
#pragma unroll
          for (int q = 0; q < kEach; ++q) {
            uint32_t y[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) y[t] = x[t][q] >> 8;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const bool v = e / 2 != 0;
              sts128((dst ^ (uint32_t)((4 * q + e) % 8 * 16) ^ swap) + (4 * q + e) * 128, centred(e % 2, v ? y[0] : x[0][q]),
                     centred(e % 2, v ? y[1] : x[1][q]), centred(e % 2, v ? y[2] : x[2][q]), centred(e % 2, v ? y[3] : x[3][q]));
            }
          }
        }
        fence_async();
        mbar_arrive(smem_u32(&bars.v_full[buf]));
        mbar_arrive(smem_u32(&bars.raw_empty[st]));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
  }
}

// The partial results of a row's splits become its output: a CTA for eight rows, a thread for four channels of one.
constexpr int kJoinRows = 8;
template <int D, bool BF16>
__global__ void __launch_bounds__(kJoinRows * D / 4)
kv4_prefill_join_kernel(const Args a, int splits, const float* __restrict__ parts) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int row = threadIdx.x % kJoinRows, c4 = threadIdx.x / kJoinRows;
  const int blocks = gridDim.x / (kRows / kJoinRows), row_block = blockIdx.x / (kRows / kJoinRows);
  const int pr = blockIdx.x % (kRows / kJoinRows) * kJoinRows + row;
  const int3 s = read_seq(a, blockIdx.z);
  const int col = row_block * kRows + pr, i = col / a.per;
  if (i >= s.y || s.y * a.per <= a.rows) return;
  const float* part = parts + (((long long)blockIdx.z * a.kv_heads + blockIdx.y) * blocks + row_block) * splits * part_floats(D);
  float top = -INFINITY;
  for (int k = 0; k < splits; ++k) top = fmaxf(top, part[k * part_floats(D) + (long long)kRows * D + pr]);
  const float base = top == -INFINITY ? 0.f : top;
  float l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = 0; k < splits; ++k) {
    const float* p = part + k * part_floats(D);
    const float f = ex2(p[(long long)kRows * D + pr] - base);
    const float4 x = reinterpret_cast<const float4*>(p)[c4 * kRows + pr];
    l = fmaf(p[(long long)kRows * D + kRows + pr], f, l);
    o = make_float4(fmaf(x.x, f, o.x), fmaf(x.y, f, o.y), fmaf(x.z, f, o.z), fmaf(x.w, f, o.w));
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t at = (int64_t)(s.x + i) * a.heads + blockIdx.y * a.per + col - i * a.per;
  reinterpret_cast<uint2*>(a.out + at * D)[c4] = make_uint2(pack2<BF16>(o.x * inv, o.y * inv), pack2<BF16>(o.z * inv, o.w * inv));
  if (a.lse && c4 == 0) a.lse[at] = l == 0.f ? -INFINITY : (top + log2f(l)) * kLn2;
}

struct Plan {
  int blocks;  // row blocks of a (sequence, cache head)
  int splits;  // shares of the cache, each a CTA
};
// CTAs that leave half of the SMs without work are split over the cache; the partial results of a split stay
// within 4 CTAs for each SM (81 MB at 128 channels).
Plan plan_of(int64_t T, int64_t B, int max_q, int heads, int kv_heads) {
  const int64_t per = heads / kv_heads, q = max_q < T ? max_q : T, sms = device_sm_count();
  const int64_t blocks = (q * per + kRows - 1) / kRows;
  const int64_t ctas = (blocks * B < T * per / kRows + B ? blocks * B : T * per / kRows + B) * kv_heads;
  int64_t splits = 2 * ctas > sms ? 1 : sms / ctas;
  if (splits * blocks * B * kv_heads > 4 * sms) splits = 4 * sms / (blocks * B * kv_heads);
  if (splits > 16) splits = 16;
  return {(int)blocks, (int)(splits < 1 ? 1 : splits)};
}

template <int D, bool BF16>
cudaError_t launch(const Kv4AttnArgs& args, int min_rows, float* parts, int* err, cudaStream_t s) {
  const void* fn = reinterpret_cast<const void*>(kv4_prefill_kernel<D, BF16>);
  cudaError_t e = set_smem_once(fn, Geo<D>::kSmem);
  if (e != cudaSuccess) return e;
  // the softmax warps wait for the registers that the others leave: launched with fewer, they would wait for ever
  static const bool enough = [fn] {
    cudaFuncAttributes f = {};
    return cudaFuncGetAttributes(&f, fn) == cudaSuccess && f.numRegs == kLaunchRegs;
  }();
  if (!enough) return cudaErrorLaunchOutOfResources;
  const Plan p = plan_of(args.T, args.B, args.max_q, args.heads, args.kv_heads);
  // a split has two tiles at least, as far as the page table tells: a CTA's start and end cost as much as those, and the
  // join is another launch
  const int64_t most = (int64_t)args.max_pages * args.page_size, seen = args.window > 0 ? (int64_t)args.window + args.max_q : most;
  const int64_t tiles = ((seen < most ? seen : most) + kTok - 1) / kTok;
  const int splits = (int)(p.splits < tiles / 2 ? p.splits : tiles / 2 > 1 ? tiles / 2 : 1);
  Args a = make_args(args);
  a.rows = min_rows;
  const int64_t ctas = (int64_t)a.kv_heads * p.blocks * splits;
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  kv4_prefill_kernel<D, BF16><<<dim3((unsigned)ctas, (unsigned)a.B), kThreads, Geo<D>::kSmem, s>>>(a, splits, parts, err);
  e = cudaGetLastError();
  if (e != cudaSuccess || splits == 1) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)(p.blocks * (kRows / kJoinRows)), (unsigned)a.kv_heads, (unsigned)a.B);
  cfg.blockDim = dim3(kJoinRows * D / 4);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kv4_prefill_join_kernel<D, BF16>, a, splits, (const float*)parts);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace

size_t kv4_prefill_workspace(int64_t T, int64_t B, int max_q, int heads, int kv_heads, int dim) {
  if (T == 0 || B == 0) return 0;
  const Plan p = plan_of(T, B, max_q, heads, kv_heads);
  return p.splits == 1 ? 0 : sizeof(float) * (size_t)p.blocks * p.splits * kv_heads * B * (size_t)part_floats(dim);
}

cudaError_t launch_kv4_prefill(const Kv4AttnArgs& a, int min_rows, int dim, bool bf16, void* ws, int* err, cudaStream_t s) {
  float* parts = static_cast<float*>(ws);
  if (dim == 128) return bf16 ? launch<128, true>(a, min_rows, parts, err, s) : launch<128, false>(a, min_rows, parts, err, s);
  return bf16 ? launch<64, true>(a, min_rows, parts, err, s) : launch<64, false>(a, min_rows, parts, err, s);
}

}  // namespace awq
