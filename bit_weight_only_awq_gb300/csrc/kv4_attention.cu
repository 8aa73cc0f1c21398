// Attention over the 4-bit paged cache, one or a few new tokens for each sequence: HBM bound.
//
//   S_j = scale q . k_j,  out = sum_j exp(S_j - m) v_j / sum_j exp(S_j - m),  m the running maximum of S
//
// with keys zk + u sk and values zv + u sv for each token and head (unit layout: include/awq.h), so that
//
//   S_j = scale (sk_j (q . u_j) + zk_j sum(q)),
//   sum_j p_j v_j = sum_j w_j u_j - 8 sum_j w_j + sum_j p_j (zv_j + 8 sv_j),  w_j = p_j sv_j rounded to fp16
//
// and only the products with the codes u need the tensor cores (mma.sync m16n8k16, fp32 sums).  The term 8 sum w
// makes the rounding of w count by its code's distance from the middle, 8, and not from 0: at 177 tokens the error is
// 2.2e-4 of the output instead of 3.0e-4, and the rounding of the fp16 output is 2.1e-4 of that.  The sum is taken of the
// rounded weights in fp32 beside the products: as a product with a subnormal operand it would lose bits (measured: a bias
// of 2^-12), since the tensor cores line such an operand up unnormalized.
//
// A code in the low bits of an fp16 half is the subnormal u 2^-24, exactly: one AND makes the operand register (two
// codes), with no offset to subtract afterwards.  Every other register holds 16 u 2^-24 (the next nibble): for keys, the matching
// query elements are divided by 16 beforehand; for values, the output rows are at the end.  The codes are the A
// operand (16 tokens or 16 channels), the queries that share a cache head the 8 columns of B, so a column for
// each of up to 8 query heads costs no more than one.
//
// Work.  The unit of work is a tile of 64 tokens of one (sequence, cache head, block of query columns).  All tiles
// of the call, in that order, are cut into equal contiguous ranges, one for each warp of a persistent grid (one
// CTA on each SM): the sequences' lengths are read on the device, and no warp waits for a longer one.  A warp
// streams its tiles through its own ring of bulk copies.  Where a head's tiles are shared, the partial results
// (maximum, sum, unnormalized output) are joined: inside a CTA after a barrier, across CTAs by the last one to
// arrive, always in the order of the tiles, so that results do not depend on timing.
//
// Measured, 32 heads on 8: 16 sequences of 32768 tokens 102 us, 5.6 TB/s of cache; 64 sequences of up to 8191 tokens
// 70 us, 4.1 TB/s; 177 tokens 9.1 us.  A call has 3 us from a CTA's start to its first copies, 3 us to the first tiles, a
// body at 6.9 TB/s, SMs that finish over 15 us (the same ones in every run) and 3 to 5 us of joins, so short
// calls are bound by latency and long ones by HBM with the uneven finish.  A tile takes 1005 instructions of a warp; at
// 8 sequences of 32768 half of the issue slots are busy.
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

constexpr int kTile = 64;    // tokens of a tile: 4 units
constexpr int kFewParts = 12;

// Eight query columns: twelve warps of 168 registers, three on each sub-partition.  Sixteen: eight warps of 255, which at
// 128 channels spill 60 bytes (and twelve far more: 16 columns of 32 x 8192 tokens 140 us).
constexpr int warps_of(int nt) { return nt == 1 ? 12 : 8; }

template <int D, int NT>
struct Geo {
  static constexpr int kWarps = warps_of(NT);
  static constexpr int kUnitBytes = kv4_unit_bytes(D);
  static constexpr int kTileBytes = 4 * kUnitBytes;
  static constexpr int kStages = (D == 128 ? 2 : 4) * 12 / kWarps;
  static constexpr int kRingBytes = kWarps * kStages * kTileBytes;
  static constexpr int kSmemBytes = kRingBytes + 128;
};

// Floats of one partial result: the unnormalized output, then maximum and sum of every column.
__host__ __device__ constexpr int part_floats(int dim, int cols) { return cols * (dim + 2); }

// What a sequence asks for.
struct Seq {
  int begin, n;      // its query tokens
  int len;           // cached tokens
  int lo;            // the first token that any of its queries sees
  int tile0, tiles;  // the first tile, and the tiles, of a (cache head, column block)
  int blocks;        // column blocks of a cache head
  int groups;        // (cache head, column block) pairs
};

template <int NT>
__device__ __forceinline__ Seq seq_of(const Args& a, const int3 v) {
  Seq s;
  s.begin = v.x;
  s.n = v.y;
  s.len = v.z;
  s.lo = a.window > 0 ? max(0, s.len - s.n + 1 - a.window) : 0;
  s.lo = min(s.lo, s.len);
  s.tile0 = s.lo / kTile;
  s.tiles = max(1, (s.len + kTile - 1) / kTile - s.tile0);
  s.blocks = s.n * a.per > a.rows ? 0 : (s.n * a.per + 8 * NT - 1) / (8 * NT);
  s.groups = a.kv_heads * s.blocks;
  return s;
}
// The first sequences, one for each thread, are kept in shared memory.
template <int NT>
__device__ __forceinline__ Seq seq_of(const Args& a, const int3* kept, int b) {
  return seq_of<NT>(a, b < 32 * warps_of(NT) ? kept[b] : read_seq(a, b));
}

// A position in the order of all tiles.
struct Cursor {
  int b, group, tile;
  Seq s;
};

template <int NT>
__device__ __forceinline__ void advance(const Args& a, const int3* kept, Cursor& c) {
  if (++c.tile < c.s.tiles) return;
  c.tile = 0;
  if (++c.group < c.s.groups) return;
  c.group = 0;
  do {
    if (++c.b >= a.B) return;
    c.s = seq_of<NT>(a, kept, c.b);
  } while (c.s.groups == 0);
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ float col_max(float v) {  // over the 8 lanes that share columns
  v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 4));
  v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 8));
  return fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, 16));
}
__device__ __forceinline__ float col_sum(float v) {
  v += __shfl_xor_sync(0xFFFFFFFFu, v, 4);
  v += __shfl_xor_sync(0xFFFFFFFFu, v, 8);
  return v + __shfl_xor_sync(0xFFFFFFFFu, v, 16);
}
template <int N>
__device__ __forceinline__ void lds_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  }
}

// Four channels of a column's partial result.
struct Joined {
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
};
// Joins element (col, channels 4 c4..) of N partials of COLS columns: all are read first, and rescaled to the
// largest maximum.  part(i) gives partial i < n; FAR: other CTAs wrote them.
template <int D, int COLS, int N, bool FAR, typename F>
__device__ __forceinline__ void join_parts(Joined& j, int n, int col, int c4, F part) {
  float m[N], l[N];
  float4 o[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
    o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (i < n) {
      const float* p = part(i);
      const float *pm = p + COLS * D + col, *pl = pm + COLS;
      const float4* po = reinterpret_cast<const float4*>(p + col * D + 4 * c4);
      m[i] = FAR ? __ldcg(pm) : *pm;
      l[i] = FAR ? __ldcg(pl) : *pl;
      o[i] = FAR ? __ldcg(po) : *po;
    }
  }
  float top = j.m;
#pragma unroll
  for (int i = 0; i < N; ++i) top = fmaxf(top, m[i]);
  const float base = top == -INFINITY ? 0.f : top, x = ex2(j.m - base);
  j.l *= x;
  j.o = make_float4(j.o.x * x, j.o.y * x, j.o.z * x, j.o.w * x);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float y = ex2(m[i] - base);
    j.l = fmaf(l[i], y, j.l);
    j.o = make_float4(fmaf(o[i].x, y, j.o.x), fmaf(o[i].y, y, j.o.y), fmaf(o[i].z, y, j.o.z), fmaf(o[i].w, y, j.o.w));
  }
  j.m = top;
}
template <int D, int COLS>
__device__ __forceinline__ void store_part(float* part, int col, int c4, const Joined& j) {
  *reinterpret_cast<float4*>(part + col * D + 4 * c4) = j.o;
  if (c4 == 0) {
    part[COLS * D + col] = j.m;
    part[COLS * D + COLS + col] = j.l;
  }
}

// The query token and head of a column, or false for a column beyond them.
__device__ __forceinline__ bool row_of(const Args& a, int begin, int n, int kv_head, int col, int64_t& token, int& head) {
  const int i = col / a.per;
  token = begin + i;
  head = kv_head * a.per + col - i * a.per;
  return i < n;
}

// One partial of a warp that does not cover its (sequence, head, column block).
struct Desc {
  long long first;  // the place of its tile 0 in the order of all tiles
  const float* part;
  int tiles, begin, n, kv_head, col0;
};

template <int D, bool BF16>
__device__ __forceinline__ void store_joined(const Args& a, const Desc& d, int col, int c4, const Joined& t) {
  int64_t token;
  int head;
  if (!row_of(a, d.begin, d.n, d.kv_head, d.col0 + col, token, head)) return;
  const float inv = t.l == 0.f ? 0.f : 1.f / t.l;
  const int64_t row = token * a.heads + head;
  reinterpret_cast<uint2*>(a.out + row * D)[c4] =
      make_uint2(pack2<BF16>(t.o.x * inv, t.o.y * inv), pack2<BF16>(t.o.z * inv, t.o.w * inv));
  if (a.lse && c4 == 0) a.lse[row] = t.l == 0.f ? -INFINITY : (t.m + log2f(t.l)) * kLn2;
}

// Part i of n equal contiguous parts of `total` tiles begins at i total / n; the part that holds a tile.  Divided
// in 32 bits where that is enough, as it mostly is.
__device__ __forceinline__ long long part_begin(long long i, long long total, long long n) {
  const unsigned long long x = (unsigned long long)i * (unsigned long long)total;
  return (x >> 32) == 0 ? (long long)((uint32_t)x / (uint32_t)n) : (long long)(x / (unsigned long long)n);
}
__device__ __forceinline__ int part_of(long long tile, long long total, long long n) {
  const unsigned long long x = (unsigned long long)(tile + 1) * (unsigned long long)n + (unsigned long long)(total - 1);
  return ((x | (unsigned long long)total) >> 32) == 0 ? (int)((uint32_t)x / (uint32_t)total) - 1
                                                      : (int)(x / (unsigned long long)total) - 1;
}

template <int D, bool BF16, int NT>
__global__ void __launch_bounds__(32 * warps_of(NT), 1)
kv4_attention_kernel(const Args a, float* warp_parts, float* cta_parts, int* counters,
                     int* err) {
  using G = Geo<D, NT>;
  constexpr int kWarps = G::kWarps, kThreads = 32 * kWarps;
  constexpr int kWords = D / 32;     // words of a lane for a token's keys, or for a token pair's values
  constexpr int kCols = 8 * NT;
  constexpr int kPart = part_floats(D, kCols);
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint64_t bars[kWarps * G::kStages];
  __shared__ long long before[kThreads];  // tiles before the sequences of each thread's share
  __shared__ long long warp_total[kWarps];
  __shared__ int3 kept[kThreads];         // the first sequences
  __shared__ Desc desc[2 * kWarps];       // of each warp: an earlier partial, the last one
  __shared__ int2 arrived[2];  // of a shared head whose last part came from here: its first CTA, its parts
  __shared__ int abort_word;
  volatile int* abort_flag = &abort_word;

  // the shuffle tells the compiler that a warp's number is the same in all its lanes
  const int tid = threadIdx.x, warp = __shfl_sync(0xFFFFFFFFu, tid / 32, 0), lane = tid % 32, g = lane / 4, t = lane % 4;
  uint8_t* ring = smem_raw + ((128u - (smem_u32(smem_raw) & 127u)) & 127u) + warp * G::kStages * G::kTileBytes;
  if (lane < G::kStages) mbar_init(smem_u32(&bars[warp * G::kStages + lane]), 1);
  if (lane < 2) desc[2 * warp + lane].part = nullptr;
  if (tid == 0) abort_word = 0;
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // ---- the order of all tiles: thread i counts the tiles of sequences [i share, (i + 1) share)
  const int share = (a.B + kThreads - 1) / kThreads;
  if (tid < a.B) kept[tid] = read_seq(a, tid);
  long long mine = 0;
  for (int b = tid * share; b < min(a.B, (tid + 1) * share); ++b) {
    const Seq s = seq_of<NT>(a, share == 1 ? kept[tid] : read_seq(a, b));
    mine += (long long)s.tiles * s.groups;
  }
  long long upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
    if (lane >= o) upto += v;
  }
  before[tid] = upto - mine;  // in this warp so far
  if (lane == 31) warp_total[warp] = upto;
  __syncthreads();
  // lane w: the tiles before warp w's sequences
  long long ahead = lane < kWarps ? warp_total[lane] : 0;
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) {
    const long long v = __shfl_up_sync(0xFFFFFFFFu, ahead, o);
    if (lane >= o) ahead += v;
  }
  const long long total = __shfl_sync(0xFFFFFFFFu, ahead, kWarps - 1);
  ahead -= lane < kWarps ? warp_total[lane] : 0;
  const long long ctas = min((long long)gridDim.x, (total + kWarps - 1) / kWarps);
  if (blockIdx.x >= ctas) return;

  const long long warps = ctas * kWarps, me = (long long)blockIdx.x * kWarps + warp;
  const long long u0 = part_begin(me, total, warps), u1 = part_begin(me + 1, total, warps);
  bool ok = true;

  if (u0 < u1) {
    // the sequence, head and tile of place u0
    Cursor use;
    {
      // the last warp's, then the last thread's, share that begins at or before u0
      const int w = __popc(__ballot_sync(0xFFFFFFFFu, lane < kWarps && ahead <= u0)) - 1;
      long long at = __shfl_sync(0xFFFFFFFFu, ahead, w);
      const int i = __popc(__ballot_sync(0xFFFFFFFFu, at + before[32 * w + lane] <= u0)) - 1;
      at += before[32 * w + i];
      use.b = (32 * w + i) * share;
      use.s = seq_of<NT>(a, kept, use.b);
      while (at + (long long)use.s.tiles * use.s.groups <= u0) {
        at += (long long)use.s.tiles * use.s.groups;
        use.s = seq_of<NT>(a, kept, ++use.b);
      }
      // a sequence may have 2^31 tiles and more; divided in 32 bits where that is enough
      const unsigned long long rest = (unsigned long long)(u0 - at), tiles = (unsigned)use.s.tiles;
      use.group = (rest >> 32) == 0 ? (int)((uint32_t)rest / (uint32_t)tiles) : (int)(rest / tiles);
      use.tile = (int)(rest - use.group * tiles);
    }
    Cursor next = use;  // the tile to be copied next
    const int count = (int)(u1 - u0);
    const int span = min(4, a.units_page);  // units that lie side by side in memory
    int next_head = next.group / next.s.blocks;
    const uint32_t bar0 = smem_u32(&bars[warp * G::kStages]);

    // lane i < 4 looks after unit i of the tile at `next`: its page, and its unit in that
    int page = 0, in_page = 0;
    auto look_up = [&]() {
      const int unit = (next.s.tile0 + next.tile) * 4 + lane;
      const int p = a.page_magic ? (int)__umulhi((uint32_t)unit, a.page_magic) : unit;
      in_page = unit - p * a.units_page;
      page = 0;
      if (lane < 4 && unit * kKv4Unit < next.s.len) page = a.block_table[next.b * a.table_stride + p];
    };
    look_up();
    auto issue = [&](int k) {  // copies tile k of this warp's range, the one at `next`
      const int j0 = (next.s.tile0 + next.tile) * kTile;
      const int first = max(0, (next.s.lo - j0) / kKv4Unit), last = min(4, (next.s.len - j0 + kKv4Unit - 1) / kKv4Unit);
      const int st = k % G::kStages;
      const uint32_t bar = bar0 + 8 * st;
      if (lane == 0) mbar_arrive_tx(bar, max(0, last - first) * G::kUnitBytes);
      __syncwarp();
      const int skip = max(first - lane, 0), to = min(lane + span, last);  // units of the span before the first one
      if (lane < 4 && (lane & (span - 1)) == 0 && lane + skip < to) {
        const int64_t p = (uint32_t)page < (uint32_t)a.num_pages ? page : 0;
        const uint8_t* src = a.cache + ((p * a.kv_heads + next_head) * a.units_page + in_page + skip) * G::kUnitBytes;
        bulk_load(smem_u32(ring + st * G::kTileBytes + (lane + skip) * G::kUnitBytes), src,
                  (to - lane - skip) * G::kUnitBytes, bar);
      }
      const int b = next.b, group = next.group;
      advance<NT>(a, kept, next);
      if ((next.b != b || next.group != group) && next.b < a.B) next_head = next.group / next.s.blocks;
      if (k + 1 < count) look_up();
    };
    int issued = 0;
    while (issued < min(count, G::kStages)) issue(issued++);

    // Scores are kept as T = S / qk with qk > 0, so that one multiply-add gives the exponent: the sign of the scale
    // goes into the queries, and a scale of zero makes them zero.
    const float sign = a.scale > 0.f ? 1.f : a.scale < 0.f ? -1.f : 0.f;
    const float factor = a.scale == 0.f ? kLog2e : fabsf(a.scale) * kLog2e;
    // a head's state: queries, running maximum, sum, zero sum, output
    uint32_t qf[NT][2 * kWords][2];
    float qk[NT][2], qr[NT][2];    // per column: the score's factor (base 2), and sum(q) over it
    int pos[NT][2];                // the last token it sees
    float m[NT][2], l[NT][2], z[NT][2], o[NT][2 * kWords][4];
    // Per column 13 - e, 2^e above the value scales it has seen: weights enter fp16 as p sv 2^(13 - e), and l, z and o are
    // in that unit, so a token hidden from a column takes no bits from its weights.  No column's e is below vexp.
    float lift[NT][2];
    int vexp = 0;
    int seg0 = 0;                  // the first tile of this warp in the current head
    int kv_head = 0, col0 = 0;

    // The queries of a head as they lie in memory: lane (g, t) reads channels [t D / 4, (t + 1) D / 4) of column g.
    uint4 raw[NT][kWords];
    auto read_q = [&](const Cursor& c) {
      const int head0 = c.group / c.s.blocks, first = (c.group - head0 * c.s.blocks) * kCols;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        int64_t token;
        int head;
        const bool in = row_of(a, c.s.begin, c.s.n, head0, first + 8 * n + g, token, head);
        const uint4* src = reinterpret_cast<const uint4*>(a.q + token * a.q_stride + head * D + t * (D / 4));
#pragma unroll
        for (int i = 0; i < kWords; ++i) raw[n][i] = in ? src[i] : make_uint4(0u, 0u, 0u, 0u);
      }
    };
    read_q(use);

    for (int k = 0; k < count; ++k) {
      if (k == 0 || use.tile == 0) {
        kv_head = use.group / use.s.blocks;
        col0 = (use.group - kv_head * use.s.blocks) * kCols;
        seg0 = use.tile;
        vexp = -16;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float x[8 * kWords];
#pragma unroll
          for (int i = 0; i < kWords; ++i) {
            const uint32_t w[4] = {raw[n][i].x, raw[n][i].y, raw[n][i].z, raw[n][i].w};
#pragma unroll
            for (int p = 0; p < 4; ++p) {
              const float2 f = unpack2<BF16>(w[p]);
              x[8 * i + 2 * p] = f.x * sign;
              x[8 * i + 2 * p + 1] = f.y * sign;
            }
          }
          float top = 0.f, sum = 0.f;
#pragma unroll
          for (int i = 0; i < 8 * kWords; ++i) {
            top = fmaxf(top, fabsf(x[i]));
            sum += x[i];
          }
          top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
          sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
          sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
          // a power of two takes the largest element to [2^14, 2^15): exact in fp16 down to 2^-24 of it, sixteenths too
          const int e = min(max((int)(__float_as_uint(top) >> 23) - 127, -100), 127);
          const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
#pragma unroll
          for (int i = 0; i < kWords; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float* y = x + 8 * i + 4 * h;
              qf[n][2 * i + h][0] = pack2<false>(y[0] * up, y[1] * up);
              qf[n][2 * i + h][1] = pack2<false>(y[2] * up * 0.0625f, y[3] * up * 0.0625f);
            }
          const float down = __uint_as_float((uint32_t)max(127 + e - 14, 1) << 23) * 16777216.f;
          // the accumulator's columns of this lane are 2t and 2t + 1
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            // not 0, which would make a NaN of a masked score, -inf; below that the weights are equal anyway
            qk[n][c] = fmaxf(__shfl_sync(0xFFFFFFFFu, down, 8 * t + 4 * c) * factor, FLT_MIN);
            qr[n][c] = __shfl_sync(0xFFFFFFFFu, sum * (up * 5.9604644775390625e-8f), 8 * t + 4 * c);
            const int i = (col0 + 8 * n + 2 * t + c) / a.per;
            pos[n][c] = i < use.s.n ? use.s.len - use.s.n + i : -1;
            m[n][c] = -INFINITY;
            l[n][c] = z[n][c] = 0.f;
            lift[n][c] = 13.f + 16.f;
          }
#pragma unroll
          for (int i = 0; i < 2 * kWords; ++i)
#pragma unroll
            for (int c = 0; c < 4; ++c) o[n][i][c] = 0.f;
        }
      }

      const int st = k % G::kStages;
      if (!__all_sync(0xFFFFFFFFu, wait_bounded(bar0 + 8 * st, (uint32_t)(k / G::kStages) & 1u, abort_flag, err, 601))) {
        ok = false;
        break;
      }
      const uint8_t* tile = ring + st * G::kTileBytes;
      const int j0 = (use.s.tile0 + use.tile) * kTile;

      // ---- scores: S[token][column], 16 tokens a unit
      float s[NT][4][4];
      uint2 meta[4][2];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint8_t* unit = tile + u * G::kUnitBytes;
        uint32_t ka[kWords], kb[kWords];
        lds_words<kWords>(unit + g * (D / 2) + t * (4 * kWords), ka);
        lds_words<kWords>(unit + (g + 8) * (D / 2) + t * (4 * kWords), kb);
        meta[u][0] = *reinterpret_cast<const uint2*>(unit + 16 * D + 8 * g);
        meta[u][1] = *reinterpret_cast<const uint2*>(unit + 16 * D + 8 * (g + 8));
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[n][u][c] = 0.f;
#pragma unroll
        for (int i = 0; i < kWords; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t x = ka[i] >> (8 * h), y = kb[i] >> (8 * h);
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma16816(s[n][u], x & 0x000F000Fu, y & 0x000F000Fu, x & 0x00F000F0u, y & 0x00F000F0u, qf[n][2 * i + h][0],
                       qf[n][2 * i + h][1]);
          }
      }
      // a tile that some column does not see whole: scales and zeros of tokens outside the sequence may be anything
      const int pos_lo = use.s.len - use.s.n;  // the position of the first query
      const bool edge = j0 + kTile > pos_lo + 1 || (a.window > 0 && j0 < use.s.len - a.window) || j0 < use.s.lo;
      if (edge) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int j = j0 + 16 * u + 8 * r + g;
            if (j < use.s.lo || j >= use.s.len) meta[u][r] = make_uint2(0u, 0u);
          }
      }
      uint32_t vtop = 0;
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float2 key = unpack2<false>(meta[u][r].x);
          vtop = max(vtop, meta[u][r].y & 0x7FFFu);  // without its sign: a cache may hold scales of either
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float& v = s[n][u][2 * r + c];
              v = fmaf(key.x, v, key.y * qr[n][c]);
            }
        }
      if (edge) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int j = j0 + 16 * u + 8 * r + g;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int c = 0; c < 2; ++c)
                if (j > pos[n][c] || (a.window > 0 && j <= pos[n][c] - a.window)) s[n][u][2 * r + c] = -INFINITY;
          }
      }

      // ---- running maximum; the largest value scale, rounded up to a power of two
      vtop = __reduce_max_sync(0xFFFFFFFFu, vtop);
      const int ve = (int)(vtop >> 10) - 14;
      bool grown = ve > vexp;
      float keep[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float top = m[n][c];
#pragma unroll
          for (int u = 0; u < 4; ++u) top = fmaxf(top, fmaxf(s[n][u][c], s[n][u][2 + c]));
          top = col_max(top);
          grown |= top > m[n][c];
          keep[n][c] = m[n][c];
          m[n][c] = top;
        }
      if (__any_sync(0xFFFFFFFFu, grown)) {
        int most[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) most[n][0] = most[n][1] = ve;
        if (__builtin_expect(edge && use.s.n > 1 && ve > vexp, 0)) {
          // columns of different tokens see different ones of this tile (what no column sees has scale 0); two in a word
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            uint32_t own = 0;
#pragma unroll
            for (int u = 0; u < 4; ++u)
#pragma unroll
              for (int r = 0; r < 2; ++r) {
                const uint32_t scale = meta[u][r].y & 0x7FFFu;
                own = __vmaxu2(own, (s[n][u][2 * r] == -INFINITY ? 0u : scale) | (s[n][u][2 * r + 1] == -INFINITY ? 0u : scale << 16));
              }
            own = __vmaxu2(own, __shfl_xor_sync(0xFFFFFFFFu, own, 4));
            own = __vmaxu2(own, __shfl_xor_sync(0xFFFFFFFFu, own, 8));
            own = __vmaxu2(own, __shfl_xor_sync(0xFFFFFFFFu, own, 16));
            most[n][0] = (int)(own >> 10 & 31u) - 14;
            most[n][1] = (int)(own >> 26) - 14;
          }
        } else {
          vexp = max(vexp, ve);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float to = fminf(lift[n][c], (float)(13 - most[n][c]));
            const float f = m[n][c] == -INFINITY ? 1.f : ex2(fmaf(keep[n][c] - m[n][c], qk[n][c], to - lift[n][c]));
            lift[n][c] = to;
            l[n][c] *= f;
            z[n][c] *= f;
#pragma unroll
            for (int i = 0; i < 2 * kWords; ++i) {
              o[n][i][c] *= f;
              o[n][i][2 + c] *= f;
            }
          }
      }

      // ---- probabilities, and their products with the values' scales as the B operand [token][column]
      float base[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) base[n][c] = m[n][c] == -INFINITY ? lift[n][c] : fmaf(-m[n][c], qk[n][c], lift[n][c]);
      uint32_t pf[NT][4][2];
      auto weigh = [&](auto hides) {
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float2 val = unpack2<false>(meta[u][r].y);
            const float zero = fmaf(8.f, val.x, val.y);
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              float p[2];
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const float v = s[n][u][2 * r + c], e = ex2(fmaf(v, qk[n][c], base[n][c]));
                // a token hidden from one column and seen by another may hold a NaN
                const bool hidden = decltype(hides)::value && v == -INFINITY;
                l[n][c] += e;
                z[n][c] = fmaf(e, hidden ? 0.f : zero, z[n][c]);
                p[c] = e * (hidden ? 0.f : val.x);
              }
              const uint32_t rounded = pack2<false>(p[0], p[1]);
              const float2 back8 = unpack2<false>(rounded);
              z[n][0] = fmaf(back8.x, -8.f, z[n][0]);
              z[n][1] = fmaf(back8.y, -8.f, z[n][1]);
              pf[n][u][r] = transpose8x8(rounded);
            }
          }
      };
      if (edge)
        weigh(std::true_type{});
      else
        weigh(std::false_type{});

      const bool last = use.tile + 1 == use.s.tiles || k + 1 == count;
      const Cursor was = use;
      advance<NT>(a, kept, use);
      if (last && k + 1 < count) read_q(use);  // arrives during the products below

      // ---- output: O[channel][column]
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint8_t* unit = tile + u * G::kUnitBytes + 8 * D;
        uint32_t va[kWords], vb[kWords];
        lds_words<kWords>(unit + lane * (4 * kWords), va);
        lds_words<kWords>(unit + (32 + lane) * (4 * kWords), vb);
#pragma unroll
        for (int i = 0; i < kWords; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t x = va[i] >> (8 * h), y = vb[i] >> (8 * h);
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma16816(o[n][2 * i + h], x & 0x000F000Fu, x & 0x00F000F0u, y & 0x000F000Fu, y & 0x00F000F0u, pf[n][u][0],
                       pf[n][u][1]);
          }
      }
      __syncwarp();  // every lane has read the stage
      if (issued < count) issue(issued++);

      if (last) {
        const bool whole = seg0 == 0 && was.tile + 1 == was.s.tiles;
        constexpr float kBack = 16777216.f;  // codes stood for u 2^-24, or 16 u 2^-24
        float* part = nullptr;
        if (!whole) {
          // the last partial of the range goes where the ring was, an earlier one to global memory
          const bool end = k + 1 == count;
          part = end ? reinterpret_cast<float*>(ring) : warp_parts + me * kPart;
          if (lane == 0) {
            Desc& d = desc[2 * warp + (end ? 1 : 0)];
            d.first = u0 + k - was.tile;
            d.part = part;
            d.tiles = was.s.tiles;
            d.begin = was.s.begin;
            d.n = was.s.n;
            d.kv_head = kv_head;
            d.col0 = col0;
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float ls = col_sum(l[n][c]), zs = col_sum(z[n][c]);
            const float unit = __uint_as_float((uint32_t)(127 - (int)lift[n][c]) << 23);
            const int col = 8 * n + 2 * t + c;
            // this lane's channels are [g D / 8, (g + 1) D / 8)
            if (whole) {
              int64_t token;
              int head;
              if (row_of(a, was.s.begin, was.s.n, kv_head, col0 + col, token, head)) {
                const float inv = ls == 0.f ? 0.f : 1.f / ls;
                const int64_t row = token * a.heads + head;
                uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + row * D + g * (D / 8));
                uint32_t w[2 * kWords];
#pragma unroll
                for (int i = 0; i < 2 * kWords; ++i)
                  w[i] = pack2<BF16>((o[n][i][c] * kBack + zs) * inv, (o[n][i][2 + c] * (kBack * 0.0625f) + zs) * inv);
#pragma unroll
                for (int i = 0; i < kWords / 2; ++i)
                  reinterpret_cast<uint4*>(dst)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                if (a.lse && g == 0)
                  a.lse[row] = ls == 0.f ? -INFINITY : (m[n][c] * qk[n][c] + log2f(ls * unit)) * kLn2;
              }
            } else {
              float* dst = part + col * D + g * (D / 8);
#pragma unroll
              for (int i = 0; i < kWords; ++i)
                reinterpret_cast<float4*>(dst)[i] =
                    make_float4((o[n][2 * i][c] * kBack + zs) * unit, (o[n][2 * i][2 + c] * (kBack * 0.0625f) + zs) * unit,
                                (o[n][2 * i + 1][c] * kBack + zs) * unit, (o[n][2 * i + 1][2 + c] * (kBack * 0.0625f) + zs) * unit);
              if (g == 0) {
                part[kCols * D + col] = m[n][c] * qk[n][c];
                part[kCols * D + kCols + col] = ls * unit;
              }
            }
          }
      }
    }
    if (!ok) {
      // leave no copy in flight behind: each one is waited for, with the same limit
      int quiet = 0;
      for (int k = max(0, issued - G::kStages); k < issued; ++k)
        wait_bounded(bar0 + 8 * (k % G::kStages), (uint32_t)(k / G::kStages) & 1u, &quiet, err, 602);
    }
  }

  // ---- the CTA's partials, in the order of the tiles
  __syncthreads();
  const long long cta0 = part_begin(blockIdx.x, total, ctas), cta1 = part_begin(blockIdx.x + 1, total, ctas);
  // lane i looks after partial i; a group is the partials of one head
  const bool some = lane < 2 * kWarps && desc[lane].part != nullptr;
  const uint32_t parts = __ballot_sync(0xFFFFFFFFu, some);
  const uint32_t below = parts & ((1u << lane) - 1u);
  const bool leads = some && (below == 0 || desc[31 - __clz(below)].first != desc[lane].first);
  const uint32_t leaders = __ballot_sync(0xFFFFFFFFu, leads);
  const bool shared = leads && (desc[lane].first < cta0 || desc[lane].first + desc[lane].tiles > cta1);
  const uint32_t open = __ballot_sync(0xFFFFFFFFu, shared);  // groups that other CTAs have a part of: two at most
  // A head shared with other CTAs has slot 1 of this CTA when it goes on after it, slot 0 when it ends here.
  auto slot = [&](int cta, bool goes_on) { return cta_parts + (2 * cta + (goes_on ? 1 : 0)) * (long long)kPart; };

  constexpr int kLanes = D / 4, kAtOnce = 32 / kLanes;  // lanes of a column, columns of a warp at once
  const int c4 = lane % kLanes;
  {
    uint32_t todo = leaders;
    for (int item = warp * kAtOnce + lane / kLanes, k = 0; todo; todo &= todo - 1, ++k) {
      const int lead = __ffs(todo) - 1;
      const uint32_t rest = todo & (todo - 1);
      const uint32_t members = parts & ~((1u << lead) - 1u) & (rest ? (rest & (0u - rest)) - 1u : 0xFFFFFFFFu);
      const Desc& d = desc[lead];
      for (; item < (k + 1) * kCols; item += kWarps * kAtOnce) {
        const int col = item - k * kCols;
        Joined j;
        for (uint32_t m = members; m;) {
          const int n = __popc(m);
          join_parts<D, kCols, 4, false>(j, n, col, c4, [&](int) {
            const float* p = desc[__ffs(m) - 1].part;
            m &= m - 1;
            return p;
          });
        }
        if (open >> lead & 1u)
          store_part<D, kCols>(slot(blockIdx.x, d.first + d.tiles > cta1), col, c4, j);
        else
          store_joined<D, BF16>(a, d, col, c4, j);
      }
    }
  }
  if (!open) return;

  // ---- heads shared with other CTAs: the last CTA to arrive joins all parts
  const int opens = __popc(open);
  auto open_desc = [&](int i) -> const Desc& { return desc[i == 0 ? __ffs(open) - 1 : 31 - __clz(open)]; };
  __syncthreads();
  if (tid < opens) {
    const Desc& d = open_desc(tid);
    const int first = part_of(d.first, total, ctas), n = part_of(d.first + d.tiles - 1, total, ctas) - first + 1;
    __threadfence();  // the CTA's parts, before its arrival
    const bool last = atomicAdd(&counters[first], 1) == n - 1;
    if (last) counters[first] = 0;  // for the next call
    arrived[tid] = last ? make_int2(first, n) : make_int2(0, 0);
    __threadfence();
  }
  __syncthreads();
  // few parts: a warp joins a column of them
  for (int item = warp * kAtOnce + lane / kLanes; item < opens * kCols; item += kWarps * kAtOnce) {
    const int i = item / kCols, col = item - i * kCols, first = arrived[i].x, n = arrived[i].y;
    if (n == 0 || n > kFewParts) continue;
    Joined j;
    for (int p = 0; p < n; p += 4)
      join_parts<D, kCols, 4, true>(j, n - p, col, c4, [&](int q) { return slot(first + p + q, p + q + 1 < n); });
    store_joined<D, BF16>(a, open_desc(i), col, c4, j);
  }
  // many: each warp joins an equal share of them, then the shares are joined
  for (int i = 0; i < opens; ++i) {
    const int first = arrived[i].x, n = arrived[i].y;
    if (n <= kFewParts) continue;
    const int p0 = n * warp / kWarps, p1 = n * (warp + 1) / kWarps;
    for (int col = lane / kLanes; col < kCols; col += 4 * kAtOnce) {  // the reads of four columns in flight
      Joined j[4];
      for (int p = p0; p < p1; p += 2)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          join_parts<D, kCols, 2, true>(j[x], p1 - p, col + x * kAtOnce, c4,
                                        [&](int q) { return slot(first + p + q, p + q + 1 < n); });
#pragma unroll
      for (int x = 0; x < 4; ++x) store_part<D, kCols>(reinterpret_cast<float*>(ring), col + x * kAtOnce, c4, j[x]);
    }
    __syncthreads();
    for (int col = warp * kAtOnce + lane / kLanes; col < kCols; col += kWarps * kAtOnce) {
      Joined j;
      join_parts<D, kCols, kWarps, false>(j, kWarps, col, c4, [&](int w) {
        return reinterpret_cast<const float*>(ring + (w - warp) * (G::kStages * G::kTileBytes));
      });
      store_joined<D, BF16>(a, open_desc(i), col, c4, j);
    }
    __syncthreads();  // the ring is written again
  }
}

template <int D, bool BF16, int NT>
cudaError_t launch(const Kv4AttnArgs& args, int max_rows, void* ws, int* err, cudaStream_t s) {
  const void* fn = reinterpret_cast<const void*>(kv4_attention_kernel<D, BF16, NT>);
  cudaError_t e = set_smem_once(fn, Geo<D, NT>::kSmemBytes);
  if (e != cudaSuccess) return e;
  const int ctas = device_sm_count();
  Args a = make_args(args);
  a.rows = max_rows;
  uint8_t* base = static_cast<uint8_t*>(ws);
  float* warp_parts = reinterpret_cast<float*>(base + kCounterBytes);
  float* cta_parts = warp_parts + (size_t)ctas * warps_of(NT) * part_floats(D, 8 * NT);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(32 * warps_of(NT));
  cfg.dynamicSmemBytes = Geo<D, NT>::kSmemBytes;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kv4_attention_kernel<D, BF16, NT>, a, warp_parts, cta_parts, reinterpret_cast<int*>(base), err);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

// Up to how many query rows of a cache head this kernel takes a sequence; the tcgen05 kernel, which makes operands of a
// tile once for 256 rows where this one goes over the cache again for every 8 or 16, takes longer ones.  us at 8 x 8192
// tokens, 8 cache heads of 128 channels, here / there: 16 rows 33 / 75, 32 rows 52 / 75, 48 rows 72 / 75, 56 rows 91 / 75;
// at 16 x 4096, 64 channels: 32 rows 39 / 67, 48 rows 53 / 67, 64 rows 66 / 67, 80 rows 80 / 67.
int rows_here(int dim) { return dim == 128 ? 48 : 64; }

// What a call takes: this kernel, with eight or sixteen columns, the other, or each for its sequences.  Sequences of
// different length (T < B max_q) may be of both kinds: 31 single tokens and 512 of a prompt, 8192 cached each, take 256 us
// so, 395 on this kernel alone and 434 on the other.
struct Route {
  bool here, there;
  int nt;
};
Route route_of(int64_t T, int64_t B, int max_q, int heads, int kv_heads, int dim) {
  const int64_t per = heads / kv_heads, rows = (max_q < T ? max_q : T) * per;
  Route r;
  r.there = rows > rows_here(dim);
  r.here = !r.there || (T < B * max_q && per <= rows_here(dim));
  r.nt = (r.there ? per : rows) <= 8 ? 1 : 2;
  return r;
}

// Counters, a partial for each warp, and two for each CTA; then the other kernel's partials.
size_t workspace_here(int nt, int dim) {
  return align256((size_t)device_sm_count() * (warps_of(nt) + 2) * sizeof(float) * part_floats(dim, 8 * nt));
}

}  // namespace

size_t kv4_attention_workspace(int64_t T, int64_t B, int max_q, int heads, int kv_heads, int dim) {
  const Route r = route_of(T, B, max_q, heads, kv_heads, dim);
  return kCounterBytes + (r.here ? workspace_here(r.nt, dim) : 0) +
         (r.there ? align256(kv4_prefill_workspace(T, B, max_q, heads, kv_heads, dim)) : 0);
}

cudaError_t launch_kv4_attention(const Kv4AttnArgs& a, int dim, bool bf16, void* ws, int* err, cudaStream_t s) {
  const Route r = route_of(a.T, a.B, a.max_q, a.heads, a.kv_heads, dim);
  if (r.here) {
    const int rows = r.there ? rows_here(dim) : INT32_MAX;
    const auto fn = r.nt == 1 ? (dim == 128 ? (bf16 ? launch<128, true, 1> : launch<128, false, 1>)
                                            : (bf16 ? launch<64, true, 1> : launch<64, false, 1>))
                              : (dim == 128 ? (bf16 ? launch<128, true, 2> : launch<128, false, 2>)
                                            : (bf16 ? launch<64, true, 2> : launch<64, false, 2>));
    const cudaError_t e = fn(a, rows, ws, err, s);
    if (e != cudaSuccess || !r.there) return e;
  }
  uint8_t* parts = static_cast<uint8_t*>(ws) + kCounterBytes + (r.here ? workspace_here(r.nt, dim) : 0);
  return launch_kv4_prefill(a, r.here ? rows_here(dim) : 0, dim, bf16, parts, err, s);
}

}  // namespace awq
