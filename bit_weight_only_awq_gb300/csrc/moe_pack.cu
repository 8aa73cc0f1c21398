// The experts' weights laid out for the grouped product (layout: include/awq.h), and back.
//
// A thread has 32 rows of one packed word, which is 32 rows of 8 columns: in the prepared copy 16 consecutive bytes of
// each column, the 8 columns next to one another in some order, so its writes are 128 bytes in one piece.  8 experts of
// 4096 x 28672: 213 us (4.6 TB/s), and 170 us back.
#include "awq_internal.h"

namespace awq {
namespace {

// Column of the AWQ layer that column c of a tile is, or -1 beyond the layer.
__device__ __forceinline__ int64_t moe_column(int tile, int c, int64_t N, bool gated) {
  if (gated) {
    const int64_t n = (int64_t)tile * 128 + (c & 127), half = N / 2;
    return n < half ? (c >> 7) * half + n : -1;
  }
  const int64_t n = (int64_t)tile * 256 + c;
  return n < N ? n : -1;
}

// grid (K / 128, tiles, experts), 128 threads: word column w = tid % 32 of the tile, rows 32 (tid / 32) .. + 31 of the group
__global__ void __launch_bounds__(128) moe_prepack_kernel(const uint32_t* __restrict__ qw, const uint32_t* __restrict__ qz,
                                                          const uint16_t* __restrict__ sc, int64_t K, int64_t N, bool gated,
                                                          uint8_t* __restrict__ packed) {
  const int g = blockIdx.x, tile = blockIdx.y, e = blockIdx.z, groups = gridDim.x;
  uint8_t* unit = packed + (((int64_t)e * gridDim.y + tile) * groups + g) * kMoeUnitBytes;
  const int w = threadIdx.x % 32, chunk = threadIdx.x / 32;
  const int64_t col = moe_column(tile, 8 * w, N, gated), nw = N / 8;  // eight columns lie on one side of every border
  const uint32_t* src = qw + ((int64_t)e * K + g * 128 + chunk * 32) * nw + col / 8;
  uint32_t out[8][4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t in[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) in[i] = col >= 0 ? src[(8 * q + order_map(i)) * nw] : 0u;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      uint32_t v = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) v |= (in[i] >> (4 * slot_of_col(c)) & 15u) << (4 * i);
      out[c][q] = v;
    }
  }
#pragma unroll
  for (int c = 0; c < 8; ++c)
    *reinterpret_cast<uint4*>(unit + moe_code_offset(8 * w + c, chunk)) =
        chunk < 2 ? make_uint4(out[c][0], out[c][1], out[c][2], out[c][3]) : make_uint4(out[c][1], out[c][0], out[c][3], out[c][2]);  // moe_word_place
  if (chunk == 0) {
    const uint32_t word = col < 0 ? 0u : qz ? qz[((int64_t)e * groups + g) * nw + col / 8] : 0x88888888u;
    uint32_t z = 0u;
#pragma unroll
    for (int c = 0; c < 8; ++c) z |= (word >> (4 * slot_of_col(c)) & 15u) << (4 * c);
    *reinterpret_cast<uint32_t*>(unit + kMoeZeroOffset + 4 * w) = z;
  } else if (chunk == 1) {
    const uint4 s = col < 0 ? make_uint4(0u, 0u, 0u, 0u)
                            : *reinterpret_cast<const uint4*>(sc + ((int64_t)e * groups + g) * N + col);
    *reinterpret_cast<uint4*>(unit + kMoeScaleOffset + 16 * w) = s;
  }
}

__global__ void __launch_bounds__(128) moe_unprepack_kernel(const uint8_t* __restrict__ packed, int64_t K, int64_t N,
                                                            bool gated, uint32_t* __restrict__ qw, uint32_t* __restrict__ qz,
                                                            uint16_t* __restrict__ sc) {
  const int g = blockIdx.x, tile = blockIdx.y, e = blockIdx.z, groups = gridDim.x;
  const uint8_t* unit = packed + (((int64_t)e * gridDim.y + tile) * groups + g) * kMoeUnitBytes;
  const int w = threadIdx.x % 32, chunk = threadIdx.x / 32;
  const int64_t col = moe_column(tile, 8 * w, N, gated), nw = N / 8;
  if (col < 0) return;
  uint32_t* dst = qw + ((int64_t)e * K + g * 128 + chunk * 32) * nw + col / 8;
  uint32_t in[8][4];
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    const uint4 v = *reinterpret_cast<const uint4*>(unit + moe_code_offset(8 * w + c, chunk));
    in[c][0] = chunk < 2 ? v.x : v.y;
    in[c][1] = chunk < 2 ? v.y : v.x;
    in[c][2] = chunk < 2 ? v.z : v.w;
    in[c][3] = chunk < 2 ? v.w : v.z;
  }
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t v = 0u;
#pragma unroll
      for (int c = 0; c < 8; ++c) v |= (in[c][q] >> (4 * i) & 15u) << (4 * slot_of_col(c));
      dst[(8 * q + order_map(i)) * nw] = v;
    }
  if (chunk == 0 && qz) {
    const uint32_t z = *reinterpret_cast<const uint32_t*>(unit + kMoeZeroOffset + 4 * w);
    uint32_t v = 0u;
#pragma unroll
    for (int c = 0; c < 8; ++c) v |= (z >> (4 * c) & 15u) << (4 * slot_of_col(c));
    qz[((int64_t)e * groups + g) * nw + col / 8] = v;
  } else if (chunk == 1) {
    *reinterpret_cast<uint4*>(sc + ((int64_t)e * groups + g) * N + col) =
        *reinterpret_cast<const uint4*>(unit + kMoeScaleOffset + 16 * w);
  }
}

dim3 unit_grid(int experts, int64_t K, int64_t N, bool gated) {
  return dim3((unsigned)(K / 128), (unsigned)moe_tiles(N, gated), (unsigned)experts);
}

}  // namespace

cudaError_t launch_moe_prepack(const uint32_t* qw, const uint32_t* qz, const uint16_t* sc, int experts, int64_t K, int64_t N,
                               bool gated, uint8_t* packed, cudaStream_t s) {
  moe_prepack_kernel<<<unit_grid(experts, K, N, gated), 128, 0, s>>>(qw, qz, sc, K, N, gated, packed);
  return cudaGetLastError();
}

cudaError_t launch_moe_unprepack(const uint8_t* packed, int experts, int64_t K, int64_t N, bool gated, uint32_t* qw,
                                 uint32_t* qz, uint16_t* sc, cudaStream_t s) {
  moe_unprepack_kernel<<<unit_grid(experts, K, N, gated), 128, 0, s>>>(packed, K, N, gated, qw, qz, sc);
  return cudaGetLastError();
}

}  // namespace awq
